// A chunk of new tokens of each sequence over a paged cache held in 4 bits (fp4.cuh), with more rows per
// key/value head than the few-row kernel (attn_paged_fp4.cu) takes.
//
// The kernel is that of chunks over the 16-bit cache (attn_fwd_two.cuh: two blocks an SM, 64-key steps,
// products on the tensor cores), with f16 operands: code * scale is exact in f16, so nothing but the weights
// is rounded before a product.  The codes become operands in one of two ways:
//
//   few query tiles a chunk: four more warps of each block convert its codes into shared memory, so that
//     the cache is read as it is: 1.4 us a 64-key step at two blocks an SM, against 0.9 over 16 bits.  32
//     sequences of 16k tokens, 4 or 16 new ones each (Hq=64 Hkv=8 d=128 bf16): 287 and 302 us, as long as
//     over the 16-bit cache (310, its bytes); 64 of 3-8 tokens over 1k-32k 688 us (736).  Without the
//     conversions' arithmetic it takes as long, without the exponentials too: what counts is the chain of a
//     step through copies, converting warps, both products and the softmax, at 96 KB of shared-memory traffic
//     a step.  Asking for the codes in L2 2 to 8 steps ahead: 338-347 us.
//   many: every tile would convert the same codes again.  They are converted once, into an f16 copy in the
//     workspace that the kernel reads as it reads a 16-bit cache.  2 x 2,048 tokens over 12k-16k in 16-token
//     pages: 1,290-1,320 us with the copy's 27 (1,360-1,390 TFLOP/s), by codes 2,000.
#include "attn_paged.cuh"

namespace attn {

namespace {

// From this many query tiles on the copy, while it is not larger than kCopyBytes.  Four chunks over 8,192
// tokens (Hq=64 Hkv=8 d=128), us by codes / with the copy: 4 tiles 94 / 115, 8 tiles 156 / 148, 16 tiles
// 302 / 247, 32 tiles 539 / 440; d = 64, 4 x 256 tokens over 4,096 (4 tiles) 48 / 52.
constexpr int kCopyTiles = 8;
constexpr size_t kCopyBytes = size_t(1) << 30;

int copy_rows(int max_k) { return (max_k + kWN - 1) / kWN * kWN; }

size_t copy_bytes(int B, int Hkv, int max_k, int d) {  // of K and V
  return static_cast<size_t>(B) * copy_rows(max_k) * Hkv * d * 2 * 2;
}

bool takes_copy(int B, int Hkv, int max_k, int d, int n_qtiles) {
  // (one sequence's bytes fit 64 bits whatever the bounds, all sequences' need not)
  return n_qtiles >= kCopyTiles && Hkv <= 32767 && copy_bytes(1, Hkv, max_k, d) <= kCopyBytes / B;
}

struct CopyParams {
  CacheFp4 c;
  const int32_t* cu_q;
  const int32_t* seqlens;
  uint16_t* k;  // [B, copy_rows, Hkv, d]
  uint16_t* v;
  int* status;
  int page_log2, Hkv, max_q, max_k, rows, window, sinks;
};

constexpr int kCopyThreads = 256;

// One 64-key step of a sequence, K (y even) or V of one head.  A thread takes blocks of sixteen codes; those of
// four (d = 64: eight) consecutive tokens lie side by side in the pool.  Steps that no new token sees, and
// sequences whose lengths are refused (the attention kernel reports them), stay as they were.  The attention
// kernel does not look at the table: entries outside the pool are reported here, and their tokens zeros.
template <int D>
__global__ void __launch_bounds__(kCopyThreads) attn_fp4_copy_kernel(const CopyParams p) {
  constexpr int kLanes = D / kFp4Block, kUnits = kWN * kLanes;
  const int j = blockIdx.x, h = blockIdx.y >> 1, b = blockIdx.z;
  const bool is_v = blockIdx.y & 1;
  const int n = p.cu_q[b + 1] - p.cu_q[b], len = p.seqlens[b];
  if (n <= 0 || n > p.max_q || len < n || len > p.max_k || ((len - 1) >> p.page_log2) >= p.c.max_pages) return;
  const int t0 = j * kWN;
  if (t0 >= len) return;
  if (p.window >= 0 && t0 >= p.sinks && t0 + kWN <= len - n - p.window) return;
  const uint8_t* codes = is_v ? p.c.v_codes : p.c.k_codes;
  const uint8_t* scales = is_v ? p.c.v_scales : p.c.k_scales;
  uint16_t* out = is_v ? p.v : p.k;
  uint2 w[kUnits / kCopyThreads];
  uint32_t s[kUnits / kCopyThreads];
#pragma unroll
  for (int i = 0; i < kUnits / kCopyThreads; ++i) {
    const int u = threadIdx.x + i * kCopyThreads, t = t0 + u / kLanes, lane = u % kLanes;
    if (t >= len) {
      s[i] = 0x100;  // nothing to copy
      continue;
    }
    const int pg = p.c.block_table[static_cast<size_t>(b) * p.c.max_pages + (t >> p.page_log2)];
    if (pg < 0 || pg >= p.c.num_pages) {
      latch_status(p.status, kStatusBadLengths);
      w[i] = make_uint2(0, 0);
      s[i] = 0;
      continue;
    }
    const size_t row = ((static_cast<size_t>(pg) * p.Hkv + h) << p.page_log2) + (t & ((1 << p.page_log2) - 1));
    w[i] = __ldcs(reinterpret_cast<const uint2*>(codes + row * (D / 2)) + lane);
    s[i] = __ldcs(scales + row * kLanes + lane);
    // a token that no new one sees becomes zeros, whatever it holds
    if (p.window >= 0 && t < len - n - p.window && t >= p.sinks) s[i] = 0;
  }
#pragma unroll
  for (int i = 0; i < kUnits / kCopyThreads; ++i) {
    if (s[i] > 0xff) continue;
    const int u = threadIdx.x + i * kCopyThreads, t = t0 + u / kLanes, lane = u % kLanes;
    const uint32_t f = fp4_scale_pair(s[i]);
    uint32_t lo[4], hi[4];
    fp4_values8(w[i].x, f, lo);
    fp4_values8(w[i].y, f, hi);
    uint4* dst = reinterpret_cast<uint4*>(
        out + ((static_cast<size_t>(b) * p.rows + t) * p.Hkv + h) * D + lane * kFp4Block);
    dst[0] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    dst[1] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
  }
}

template <int D, bool BF16>
int launch_copy(const PagedArgs& a, const CacheFp4& c, cudaStream_t stream) {
  CopyParams p = {};
  p.c = c;
  p.cu_q = a.cu_q;
  p.seqlens = a.seqlens;
  p.rows = copy_rows(a.max_k);
  const size_t half = copy_bytes(a.B, a.Hkv, a.max_k, D) / 2;
  p.k = static_cast<uint16_t*>(a.workspace);
  p.v = p.k + half / 2;
  while ((1 << p.page_log2) < c.page_size) ++p.page_log2;
  p.Hkv = a.Hkv;
  p.max_q = a.max_q;
  p.max_k = a.max_k;
  p.status = device_status_ptr();
  if (!p.status) return -5;
  p.window = a.window;
  p.sinks = a.sinks;
  attn_fp4_copy_kernel<D><<<dim3(p.rows / kWN, 2 * a.Hkv, a.B), kCopyThreads, 0, stream>>>(p);
  if (cudaGetLastError() != cudaSuccess) return -5;
  PagedArgs b = a;
  b.k_pages = p.k;
  b.v_pages = p.v;
  b.workspace = static_cast<char*>(a.workspace) + 2 * half;  // the parts of split rows, if any
  return launch_paged_variant<D, BF16, kKvCopy>(b, nullptr, p.rows, stream);
}

template <int D, bool BF16>
int launch_chunk(const PagedArgs& a, const CacheFp4& c, cudaStream_t stream) {
  const PagedSplit sp = paged_split(a.B, a.Hq, a.Hkv, a.max_q, a.max_k, a.window, a.sinks, D);
  return takes_copy(a.B, a.Hkv, a.max_k, D, sp.n_qtiles)
             ? launch_copy<D, BF16>(a, c, stream)
             : launch_paged_variant<D, BF16, kKvCodes>(a, &c, 0, stream);
}

}  // namespace

int launch_attn_fp4_chunk(const PagedArgs& a, const CacheFp4& c, cudaStream_t stream) {
  if (a.d == 64)
    return a.bf16 ? launch_chunk<64, true>(a, c, stream) : launch_chunk<64, false>(a, c, stream);
  return a.bf16 ? launch_chunk<128, true>(a, c, stream) : launch_chunk<128, false>(a, c, stream);
}

size_t fp4_chunk_workspace_bytes(int total_q, int B, int Hq, int Hkv, int max_q, int max_k, int window,
                                 int sinks, int d) {
  const PagedSplit sp = paged_split(B, Hq, Hkv, max_q, max_k, window, sinks, d);
  const size_t parts = sp.n_splits == 1 ? 0 : paged_parts_bytes(total_q, Hq, sp.n_splits, d);
  return parts + (takes_copy(B, Hkv, max_k, d, sp.n_qtiles) ? copy_bytes(B, Hkv, max_k, d) : 0);
}

}  // namespace attn
