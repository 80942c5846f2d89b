// A paged KV cache held in 4 bits (the format: fp4.cuh): quantising new tokens into it, and reading cached
// tokens back as the packed 16-bit cache.
//
// A row is the d values of one (token, key/value head) of K or of V.  Of each block of sixteen, with
// a = max |x_c|, the scale is a / 6 rounded to the scale's type and the codes are x_c / scale rounded to
// theirs, both to nearest even (a scale that rounds down makes the largest value saturate, by half a step
// of the scale at most).  The quotient is the correctly rounded one, x r + (x - s x r) r with r = 1 / s
// rounded, so that halves between two codes are told from their neighbours.  A block with a value that is
// not finite is stored as NaN: a code has none, and a finite one would hide it.  Reading back is exact in
// both 16-bit types.
//
// The pools are [page, head, token, d / 2] and [.., d / 16]: a head's rows of a page side by side, since
// a 64-byte row (32 at d = 64) is shorter than what memory moves best, and the attention kernels read one
// head's.  The writer takes its tokens' places as a slot map; a thread takes one block, the threads of a
// warp the blocks of one head's consecutive tokens, which are neighbours in the pool too.
//
// Bound by memory, of which the writer takes 5.5 TB/s and the reader 5.6-6.4 (a copy 6.8); the writer issues in
// four of five cycles beside it.  77k tokens (Hkv=8
// d=128) into 16-token pages 74 us and back out 72, 440k out of 32-token pages 357 us; 64 sequences' single
// tokens are launch and latency.  The reader's threads take eight values of each half of a row, so that their
// 16-byte stores lie side by side (sixteen together: 79 us; with streaming stores 75 -> 72); the same in the
// writer doubles the scales' arithmetic (92 us).  Four rows loaded ahead of the first conversion: 87.
#include "attn_cache.cuh"
#include "fp4.cuh"

namespace attn {

namespace {

struct Cache4Params {
  uint16_t* k;  // [total, Hkv, d] (written by the reader)
  uint16_t* v;
  CacheFp4 c;
  const int32_t* slots;  // [total] (writer)
  const int32_t* cu;     // [B + 1] (reader)
  const int32_t* starts;  // [B] or null: first token read of each sequence (reader)
  int* status;
  int total, B, Hkv, page_log2, run;
};

// Row `row` of a block's n x Hkv rows, token fastest: its token and head, advanced without a division.
struct HeadRow {
  int tok, h, dt, dh, n;
  __device__ __forceinline__ HeadRow(int u, int step, int n_)
      : tok(u % n_), h(u / n_), dt(step % n_), dh(step / n_), n(n_) {}
  __device__ __forceinline__ void advance() {
    tok += dt;
    h += dh;
    if (tok >= n) {
      tok -= n;
      ++h;
    }
  }
};

// Place of (page, head, slot in the page) among the pools' rows.
__device__ __forceinline__ size_t pool_row(int at, int h, int Hkv, int page_log2) {
  return (((static_cast<size_t>(at >> page_log2) * Hkv) + h) << page_log2) + (at & ((1 << page_log2) - 1));
}

}  // namespace

template <int D, bool BF16>
__global__ void __launch_bounds__(kCacheThreads) cache_write_fp4_kernel(const Cache4Params p) {
  constexpr int kLanes = D / kFp4Block;  // threads of a row
  constexpr int kStep = kCacheThreads / kLanes;
  __shared__ int slot[kMaxRun];
  const int i0 = blockIdx.x * p.run;
  const int n = min(p.run, p.total - i0);
  const int rows = n * p.Hkv;
  const int lane = threadIdx.x % kLanes;
  const bool is_v = blockIdx.y != 0;
  const uint16_t* src0 = (is_v ? p.v : p.k) + static_cast<size_t>(i0) * p.Hkv * D + lane * kFp4Block;
  uint8_t* codes = is_v ? p.c.v_codes : p.c.k_codes;
  uint8_t* scales = is_v ? p.c.v_scales : p.c.k_scales;
  for (int r = threadIdx.x; r < n; r += kCacheThreads) {
    const int at = p.slots[i0 + r];
    const bool good = at >= 0 && (at >> p.page_log2) < p.c.num_pages;
    if (!good && at != -1) latch_status(p.status, kStatusBadLengths);
    slot[r] = good ? at : -1;
  }
  HeadRow next(threadIdx.x / kLanes, kStep, n);  // rows are loaded two steps ahead
  uint4 ahead[2][2] = {};
  auto load = [&](uint4 (&w)[2], int u) {
    if (u < rows) {
      const uint4* src =
          reinterpret_cast<const uint4*>(src0 + (static_cast<size_t>(next.tok) * p.Hkv + next.h) * D);
      w[0] = __ldcs(src);
      w[1] = __ldcs(src + 1);
    }
    next.advance();
  };
  const int u_first = threadIdx.x / kLanes;
  HeadRow rr = next;
  load(ahead[0], u_first);
  load(ahead[1], u_first + kStep);
  __syncthreads();
#pragma unroll 2
  for (int u = u_first, b = 0; u < rows; u += kStep, b ^= 1) {
    const int at = slot[rr.tok];
    const int h = rr.h;
    rr.advance();
    uint32_t w[8] = {ahead[b][0].x, ahead[b][0].y, ahead[b][0].z, ahead[b][0].w,
                     ahead[b][1].x, ahead[b][1].y, ahead[b][1].z, ahead[b][1].w};
    load(ahead[b], u + 2 * kStep);
    if (at < 0) continue;
    uint32_t m2 = 0;
#pragma unroll
    for (int c = 0; c < 8; ++c) m2 = max_abs2<BF16>(m2, w[c]);
    float pair[8], x[16];
    unpack8<BF16>(make_uint4(m2, 0, 0, 0), pair);
    const float amax = fmaxf(pair[0], pair[1]);
    uint32_t byte = kFp4Nan;
    uint2 out = make_uint2(0, 0);
    if (pair[0] <= 3.402823466e38f && pair[1] <= 3.402823466e38f) {  // else the block is NaN
      byte = fp4_scale_byte(amax);
      if (byte != 0) {  // else every value is zero
        unpack8<BF16>(make_uint4(w[0], w[1], w[2], w[3]), x);
        unpack8<BF16>(make_uint4(w[4], w[5], w[6], w[7]), x + 8);
        const float s = fp4_scale(byte), r = __frcp_rn(s);
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          const float y = x[c] * r;
          x[c] = fmaf(fmaf(-s, y, x[c]), r, y);
        }
        out = make_uint2(fp4_codes8(x), fp4_codes8(x + 8));
      }
    }
    const size_t row = pool_row(at, h, p.Hkv, p.page_log2);
    *reinterpret_cast<uint2*>(codes + row * (D / 2) + lane * 8) = out;
    scales[row * kLanes + lane] = static_cast<uint8_t>(byte);
  }
}

// Two f16 pairs (exact in both types) -> the pairs of the output type.
template <bool BF16>
__device__ __forceinline__ uint32_t f16x2_out(uint32_t w) {
  if constexpr (!BF16) return w;
  float lo, hi;
  asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(lo), "=f"(hi)
      : "r"(w));
  return pack2<true>(lo, hi);
}

template <int D, bool BF16>
__global__ void __launch_bounds__(kCacheThreads) cache_read_fp4_kernel(const Cache4Params p) {
  constexpr int kLanes = D / kFp4Block;
  constexpr int kStep = kCacheThreads / kLanes;
  __shared__ int slot[kMaxRun];
  const int i0 = blockIdx.x * p.run;
  const int n = min(p.run, p.total - i0);
  const int rows = n * p.Hkv;
  const int lane = threadIdx.x % kLanes;
  const bool is_v = blockIdx.y != 0;
  uint16_t* dst0 = (is_v ? p.v : p.k) + static_cast<size_t>(i0) * p.Hkv * D;
  const uint8_t* codes = is_v ? p.c.v_codes : p.c.k_codes;
  const uint8_t* scales = is_v ? p.c.v_scales : p.c.k_scales;
  for (int r = threadIdx.x; r < n; r += kCacheThreads) {
    const int i = i0 + r;
    int at = -1;
    if (i >= p.cu[0] && i < p.cu[p.B]) {
      const int b = find_sequence(p.cu, p.B, i);
      const int first = p.cu[b], start = p.starts ? p.starts[b] : 0;
      const long long t = static_cast<long long>(start) + (i - first);
      int page = -1;
      if (first <= i && start >= 0 && (t >> p.page_log2) < p.c.max_pages)
        page = p.c.block_table[static_cast<size_t>(b) * p.c.max_pages + (t >> p.page_log2)];
      if (page >= 0 && page < p.c.num_pages)
        at = (page << p.page_log2) + static_cast<int>(t & ((1 << p.page_log2) - 1));
      else
        latch_status(p.status, kStatusBadLengths);
    }
    slot[r] = at;
  }
  __syncthreads();
  HeadRow rr(threadIdx.x / kLanes, kStep, n);
  for (int u = threadIdx.x / kLanes; u < rows; u += kStep, rr.advance()) {
    const int at = slot[rr.tok];
    if (at < 0) continue;
    const size_t row = pool_row(at, rr.h, p.Hkv, p.page_log2);
    // eight values of each half of the row, so that a row's threads store side by side
    uint4* dst = reinterpret_cast<uint4*>(dst0 + (static_cast<size_t>(rr.tok) * p.Hkv + rr.h) * D);
    uint32_t w[2], s[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      w[i] = __ldcs(reinterpret_cast<const uint32_t*>(codes + row * (D / 2)) + lane + i * kLanes);
      s[i] = __ldcs(scales + row * kLanes + (lane + i * kLanes) / 2);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint32_t v[4];
      fp4_values8(w[i], fp4_scale_pair(s[i]), v);
      __stcs(dst + lane + i * kLanes, make_uint4(f16x2_out<BF16>(v[0]), f16x2_out<BF16>(v[1]),
                                                 f16x2_out<BF16>(v[2]), f16x2_out<BF16>(v[3])));
    }
  }
}

static int cache4_params(Cache4Params& p, const CacheFp4& c, const void* k, const void* v, int total, int Hkv) {
  p.k = static_cast<uint16_t*>(const_cast<void*>(k));
  p.v = static_cast<uint16_t*>(const_cast<void*>(v));
  p.c = c;
  p.total = total;
  p.Hkv = Hkv;
  while ((1 << p.page_log2) < c.page_size) ++p.page_log2;
  p.status = device_status_ptr();
  p.run = cache_run(total);
  return p.status ? 0 : -5;
}

int launch_cache_write_fp4(const CacheFp4& c, const void* k, const void* v, const int32_t* slots, int total,
                           int Hkv, int d, bool bf16, cudaStream_t stream) {
  Cache4Params p = {};
  const int st = cache4_params(p, c, k, v, total, Hkv);
  if (st != 0) return st;
  p.slots = slots;
  const dim3 grid((total + p.run - 1) / p.run, 2);
  auto kern = d == 128 ? (bf16 ? cache_write_fp4_kernel<128, true> : cache_write_fp4_kernel<128, false>)
                       : (bf16 ? cache_write_fp4_kernel<64, true> : cache_write_fp4_kernel<64, false>);
  kern<<<grid, kCacheThreads, 0, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? 0 : -5;
}

int launch_cache_read_fp4(const CacheFp4& c, void* k, void* v, const int32_t* cu_k, const int32_t* starts,
                          int total, int B, int Hkv, int d, bool bf16, cudaStream_t stream) {
  Cache4Params p = {};
  const int st = cache4_params(p, c, k, v, total, Hkv);
  if (st != 0) return st;
  p.cu = cu_k;
  p.starts = starts;
  p.B = B;
  const dim3 grid((total + p.run - 1) / p.run, 2);
  auto kern = d == 128 ? (bf16 ? cache_read_fp4_kernel<128, true> : cache_read_fp4_kernel<128, false>)
                       : (bf16 ? cache_read_fp4_kernel<64, true> : cache_read_fp4_kernel<64, false>);
  kern<<<grid, kCacheThreads, 0, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? 0 : -5;
}

}  // namespace attn
