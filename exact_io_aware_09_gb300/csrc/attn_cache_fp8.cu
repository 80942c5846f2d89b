// A paged KV cache held in 8 bits: quantising new tokens as they are written, and reading cached
// tokens back as the packed 16-bit cache.
//
// A row is the d values of one (token, key/value head) of K or of V.  With a = max |x_c| over the
// row's finite values, e is the smallest integer (at least -126; 0 when a = 0) with
// a <= 448 * 2^e, 448 being E4M3's largest value; the row is stored as the codes E4M3(x_c 2^-e),
// nearest even, and the scale 2^e.  A power of two makes both directions exact multiplies: the
// only rounding is E4M3's, and none on the way back but for values outside the type's range
// (saturated to its largest finite value, or rounded into its subnormals).  A value that is not
// finite takes no part in a and is stored as the NaN code: E4M3 has no infinity, and a finite
// code would hide it.
//
// Both kernels are bound by memory; the writer's ALU is 45% busy beside it (amax, scale and conversion of
// every value).  Hkv=8 d=128: 77k prompt tokens into 16-token pages 82 us (499 MB, 6.1 TB/s), 440k cached
// tokens back out of 32-token pages 413 us (2.73 GB, 6.6 TB/s, a copy's rate); 64 sequences' single tokens
// 9 us on the device, launch and latency.  A block takes a run of packed tokens: its threads find their
// sequences and cache rows first (one token each, a binary search of the packed offsets), then the block
// streams the run's rows, d / 16 lanes per row with 32 bytes of 16-bit values and 16 bytes of codes each.
// Packed rows are consecutive, and so are cache rows inside a page, so every access of a warp is whole
// lines but for the scales.
#include "attn_cache.cuh"

namespace attn {

namespace {

struct CacheParams {
  const uint16_t* k;  // [total, Hkv, d] (written by the reader)
  const uint16_t* v;
  CacheFp8 c;
  const int32_t* cu;       // [B + 1]
  const int32_t* seqlens;  // [B] cached tokens, the new ones included (writer)
  int* status;
  int total, B, Hkv, page_log2, run;
};

// Exponent e of a row's scale: the smallest with amax <= 448 * 2^e.  With amax = (1 + M/2^23)
// 2^(E-127), amax <= 1.75 * 2^(8+e) holds from e = E - 135 when the mantissa is at most 0.75
// (1.75 = 448 / 2^8), from e = E - 134 otherwise.
__device__ __forceinline__ int row_scale_exp(float amax) {
  if (!(amax > 0.0f)) return 0;
  const uint32_t b = __float_as_uint(amax);
  const int E = static_cast<int>(b >> 23);
  const int e = ((b & 0x7fffffu) <= 0x600000u) ? E - 135 : E - 134;
  return e < -126 ? -126 : e;
}

__device__ __forceinline__ float pow2i(int e) {  // 2^e for -126 <= e <= 127
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// Two values -> a 16-bit pair, nearest even, saturating at the largest finite value (NaN stays).
template <bool BF16>
__device__ __forceinline__ uint32_t pack2_sat(float lo, float hi) {
  uint32_t r;
  if constexpr (BF16)
    asm("cvt.rn.satfinite.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Four E4M3 codes -> floats (exact).
__device__ __forceinline__ void codes4(uint32_t w, float* v) {
  uint32_t lo, hi;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
  asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(v[0]), "=f"(v[1])
      : "r"(lo));
  asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(v[2]), "=f"(v[3])
      : "r"(hi));
}

// The (page, slot) of each token of the block's run as one pool row (page * page_size + slot), or
// -1 for a packed row outside the sequences or a token whose position or page is out of bounds
// (reported).  WRITE: the packed rows are the last tokens of their sequences, else the first.
template <bool WRITE>
__device__ __forceinline__ void locate_run(const CacheParams& p, int i0, int n, int* slot) {
  for (int r = threadIdx.x; r < n; r += kCacheThreads) {
    const int i = i0 + r;
    int at = -1;
    if (i >= p.cu[0] && i < p.cu[p.B]) {
      const int b = find_sequence(p.cu, p.B, i);
      const int first = p.cu[b];
      int t = i - first;
      if (WRITE) t += p.seqlens[b] - (p.cu[b + 1] - first);
      int page = -1;
      if (first <= i && t >= 0 && (t >> p.page_log2) < p.c.max_pages)
        page = p.c.block_table[static_cast<size_t>(b) * p.c.max_pages + (t >> p.page_log2)];
      if (page >= 0 && page < p.c.num_pages)
        at = (page << p.page_log2) + (t & ((1 << p.page_log2) - 1));
      else
        latch_status(p.status, kStatusBadLengths);
    }
    slot[r] = at;
  }
}

// (token, head) of row u of a block's run, advanced by a fixed number of rows without a division.
struct RunRow {
  int tok, h, dt, dh, Hkv;
  __device__ __forceinline__ RunRow(int u, int step, int Hkv_)
      : tok(u / Hkv_), h(u % Hkv_), dt(step / Hkv_), dh(step % Hkv_), Hkv(Hkv_) {}
  __device__ __forceinline__ void advance() {
    tok += dt;
    h += dh;
    if (h >= Hkv) {
      h -= Hkv;
      ++tok;
    }
  }
};

}  // namespace

template <int D, bool BF16>
__global__ void __launch_bounds__(kCacheThreads) cache_write_fp8_kernel(const CacheParams p) {
  constexpr int kLanes = D / 16;  // lanes of a row
  __shared__ int slot[kMaxRun];
  constexpr int kStep = kCacheThreads / kLanes;  // rows of the block at a time
  const int i0 = blockIdx.x * p.run;
  const int n = min(p.run, p.total - i0);
  const int lane = threadIdx.x % kLanes;
  const int rows = n * p.Hkv;
  const bool is_v = blockIdx.y != 0;
  const uint16_t* src0 = (is_v ? p.v : p.k) + static_cast<size_t>(i0) * p.Hkv * D + lane * 16;
  uint8_t* codes = is_v ? p.c.v_pages : p.c.k_pages;
  float* scales = is_v ? p.c.v_scales : p.c.k_scales;
  // Rows are loaded two steps ahead: the first two while the run's cache rows are looked up.
  uint4 ahead[2][2] = {};
  auto load = [&](uint4 (&w)[2], int u) {
    if (u >= rows) return;
    const uint4* src = reinterpret_cast<const uint4*>(src0 + static_cast<size_t>(u) * D);
    w[0] = __ldcs(src);
    w[1] = __ldcs(src + 1);
  };
  const int u_first = threadIdx.x / kLanes;
  load(ahead[0], u_first);
  load(ahead[1], u_first + kStep);
  locate_run<true>(p, i0, n, slot);
  __syncthreads();
  RunRow rr(u_first, kStep, p.Hkv);
#pragma unroll 2
  for (int u0 = 0, b = 0; u0 < rows; u0 += kStep, b ^= 1) {
    const int u = u0 + u_first;  // every lane stays for the row's reductions
    const int at = u < rows ? slot[rr.tok] : -1;
    const int h = rr.h;
    rr.advance();
    float x[16];
    unpack8<BF16>(ahead[b][0], x);
    unpack8<BF16>(ahead[b][1], x + 8);
    // the row's largest magnitude, in 16-bit pairs (exact): the kernel is near the ALU's rate
    uint32_t m2 = 0;
    {
      const uint32_t w[8] = {ahead[b][0].x, ahead[b][0].y, ahead[b][0].z, ahead[b][0].w,
                             ahead[b][1].x, ahead[b][1].y, ahead[b][1].z, ahead[b][1].w};
#pragma unroll
      for (int c = 0; c < 8; ++c) m2 = max_abs2<BF16>(m2, w[c]);
    }
#pragma unroll
    for (int sh = kLanes / 2; sh > 0; sh >>= 1)
      m2 = max_abs2<BF16>(m2, __shfl_xor_sync(0xffffffffu, m2, sh));
    load(ahead[b], u + 2 * kStep);
    float pair[8];
    unpack8<BF16>(make_uint4(m2, 0, 0, 0), pair);
    float amax = fmaxf(pair[0], pair[1]);
    const bool odd = !(pair[0] <= 3.402823466e38f) || !(pair[1] <= 3.402823466e38f);
    if (__any_sync(0xffffffffu, odd)) {
      // a value that is not finite: it becomes the NaN code and takes no part in the maximum
      amax = 0.0f;
#pragma unroll
      for (int c = 0; c < 16; ++c) {
        const float a = fabsf(x[c]);
        if (a <= 3.402823466e38f)
          amax = fmaxf(amax, a);
        else
          x[c] = __uint_as_float(0x7fffffffu);
      }
#pragma unroll
      for (int sh = kLanes / 2; sh > 0; sh >>= 1)
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, sh));
    }
    if (at < 0) continue;
    const int e = row_scale_exp(amax);
    const float inv = pow2i(-e);
    uint4 w;
    w.x = pack4_e4m3(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv);
    w.y = pack4_e4m3(x[4] * inv, x[5] * inv, x[6] * inv, x[7] * inv);
    w.z = pack4_e4m3(x[8] * inv, x[9] * inv, x[10] * inv, x[11] * inv);
    w.w = pack4_e4m3(x[12] * inv, x[13] * inv, x[14] * inv, x[15] * inv);
    *reinterpret_cast<uint4*>(codes + (static_cast<size_t>(at) * p.Hkv + h) * D + lane * 16) = w;
    if (lane == 0) {
      const int page = at >> p.page_log2;
      scales[((static_cast<size_t>(page) * p.Hkv + h) << p.page_log2) +
             (at & ((1 << p.page_log2) - 1))] = pow2i(e);
    }
  }
}

template <int D, bool BF16>
__global__ void __launch_bounds__(kCacheThreads) cache_read_fp8_kernel(const CacheParams p) {
  constexpr int kLanes = D / 16;
  __shared__ int slot[kMaxRun];
  const int i0 = blockIdx.x * p.run;
  const int n = min(p.run, p.total - i0);
  locate_run<false>(p, i0, n, slot);
  __syncthreads();
  const int lane = threadIdx.x % kLanes;
  const int rows = n * p.Hkv;
  const bool is_v = blockIdx.y != 0;
  uint16_t* dst0 = const_cast<uint16_t*>(is_v ? p.v : p.k) + static_cast<size_t>(i0) * p.Hkv * D;
  const uint8_t* codes = is_v ? p.c.v_pages : p.c.k_pages;
  const float* scales = is_v ? p.c.v_scales : p.c.k_scales;
  for (int u = threadIdx.x / kLanes; u < rows; u += kCacheThreads / kLanes) {
    const int at = slot[u / p.Hkv];
    if (at < 0) continue;
    const int h = u % p.Hkv;
    const int page = at >> p.page_log2;
    const float sc = scales[((static_cast<size_t>(page) * p.Hkv + h) << p.page_log2) +
                            (at & ((1 << p.page_log2) - 1))];
    const uint4 w = *reinterpret_cast<const uint4*>(
        codes + (static_cast<size_t>(at) * p.Hkv + h) * D + lane * 16);
    float x[16];
    codes4(w.x, x);
    codes4(w.y, x + 4);
    codes4(w.z, x + 8);
    codes4(w.w, x + 12);
    uint32_t o[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) o[c] = pack2_sat<BF16>(x[2 * c] * sc, x[2 * c + 1] * sc);
    uint4* dst = reinterpret_cast<uint4*>(dst0 + static_cast<size_t>(u) * D + lane * 16);
    dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
    dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
  }
}

static int cache_params(CacheParams& p, const CacheFp8& c, const void* k, const void* v,
                        const int32_t* cu, const int32_t* seqlens, int total, int B, int Hkv) {
  p.k = static_cast<const uint16_t*>(k);
  p.v = static_cast<const uint16_t*>(v);
  p.c = c;
  p.cu = cu;
  p.seqlens = seqlens;
  p.total = total;
  p.B = B;
  p.Hkv = Hkv;
  p.page_log2 = 0;
  while ((1 << p.page_log2) < c.page_size) ++p.page_log2;
  p.status = device_status_ptr();
  if (!p.status) return -5;
  p.run = cache_run(total);
  return 0;
}

int launch_cache_write_fp8(const CacheFp8& c, const void* k, const void* v, const int32_t* cu_q,
                           const int32_t* seqlens, int total, int B, int Hkv, int d, bool bf16,
                           cudaStream_t stream) {
  CacheParams p;
  const int st = cache_params(p, c, k, v, cu_q, seqlens, total, B, Hkv);
  if (st != 0) return st;
  const dim3 grid((total + p.run - 1) / p.run, 2);
  auto kern = d == 128 ? (bf16 ? cache_write_fp8_kernel<128, true> : cache_write_fp8_kernel<128, false>)
                       : (bf16 ? cache_write_fp8_kernel<64, true> : cache_write_fp8_kernel<64, false>);
  kern<<<grid, kCacheThreads, 0, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? 0 : -5;
}

int launch_cache_read_fp8(const CacheFp8& c, void* k, void* v, const int32_t* cu_k, int total,
                          int B, int Hkv, int d, bool bf16, cudaStream_t stream) {
  CacheParams p;
  const int st = cache_params(p, c, k, v, cu_k, nullptr, total, B, Hkv);
  if (st != 0) return st;
  const dim3 grid((total + p.run - 1) / p.run, 2);
  auto kern = d == 128 ? (bf16 ? cache_read_fp8_kernel<128, true> : cache_read_fp8_kernel<128, false>)
                       : (bf16 ? cache_read_fp8_kernel<64, true> : cache_read_fp8_kernel<64, false>);
  kern<<<grid, kCacheThreads, 0, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? 0 : -5;
}

}  // namespace attn
