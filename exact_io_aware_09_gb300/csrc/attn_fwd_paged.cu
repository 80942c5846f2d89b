// A chunk of new tokens of each sequence over a paged KV cache: causal attention of the last
// positions of every sequence, with or without a sliding window and sinks.
//
// The kernel with two blocks on an SM (attn_fwd_two.cuh) runs it.  A query tile's 128 rows are (token,
// query head) pairs of one key/value head, 128 / G tokens of the G heads that share it, so that a tile
// reads each cache row once for all its heads and a chunk of a few tokens still fills the tile: the
// number of products is that of one head per tile, the diagonal takes G times fewer masked steps.  When
// the chunks give fewer tiles than keep the SMs evenly busy, an item's keys are split and the parts'
// normalised rows merged with the (m, l) rule by a second kernel.
//
// Bound by the tensor cores for long chunks, by the cache's bytes for a few tokens.  Hq=64 Hkv=8 d=128
// bf16: two chunks of 2,048 tokens, both over 16,384 cached ones, 1,330-1,380 us in 16-token pages (1,500-1,550
// TFLOP/s, tensor pipe 67% busy) and 1,300-1,410 in 64-token pages, the contiguous prefill of the same
// 1,320-1,480, box by box (on the prefill kernel, one block an SM: 1,750 and 1,400, its producers' 16 copies
// a tile being as long as the tile); over 12k-16k 1,260-1,280; 64 sequences of 3-8 tokens over 1k-32k 736 us (6.5 TB/s).
// Calls of at most 16 rows per key/value head go to attn_paged_few.cu.
#include "attn_paged.cuh"

namespace attn {

namespace {

size_t parts_o_bytes(size_t parts, int d) {
  return (parts * d * 4 + 255) & ~static_cast<size_t>(255);
}

}  // namespace

size_t paged_workspace_bytes(int total_q, int B, int Hq, int Hkv, int max_q, int max_k, int window,
                             int sinks, int d) {
  if (total_q <= 0 || B <= 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv || Hq / Hkv > kWM ||
      max_q <= 0 || max_k <= 0 || d <= 0)
    return 0;
  PagedArgs a = {};
  a.B = B;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.max_q = max_q;
  int n_splits;
  if (paged_few_rows(a)) {
    int stages;
    paged_few_split(B, Hkv, max_q, max_k, window, sinks, d, n_splits, stages);
    if (n_splits <= kMaxCluster) return 0;
  } else {
    n_splits = paged_split(B, Hq, Hkv, max_q, max_k, window, sinks, d).n_splits;
    if (n_splits == 1) return 0;
  }
  return paged_parts_bytes(total_q, Hq, n_splits, d);
}

size_t paged_parts_bytes(int total_q, int Hq, int n_splits, int d) {
  const size_t parts = static_cast<size_t>(total_q) * Hq * n_splits;
  return parts_o_bytes(parts, d) + parts * 8;
}

void paged_parts(const PagedArgs& a, int d, int n_splits, float*& ws_o, float*& ws_ml) {
  const size_t parts = static_cast<size_t>(a.total_q) * a.Hq * n_splits;
  ws_o = static_cast<float*>(a.workspace);
  ws_ml = reinterpret_cast<float*>(static_cast<char*>(a.workspace) + parts_o_bytes(parts, d));
}

// One warp per row: the merge of its splits' (m, l, o).  A split without a visible key has
// (m, l) = (-inf, 0) and no row of its own.  Rows outside the packed sequences are left alone.
constexpr int kMergeWarps = 4;

template <int D, bool BF16>
__global__ void __launch_bounds__(kMergeWarps * 32)
    attn_paged_merge_kernel(const float* ws_o, const float* ws_ml, const int32_t* cu_q, int B,
                            int Hq, size_t rows, int n_splits, uint16_t* out, float* lse) {
  constexpr int kC = D / 32;  // channels per lane
  griddep_wait();
  const int lane = threadIdx.x & 31;
  const size_t row = static_cast<size_t>(blockIdx.x) * kMergeWarps + (threadIdx.x >> 5);
  if (row >= rows) return;
  if (cu_q) {  // (null: one token of each sequence)
    const long long tok = static_cast<long long>(row / Hq);
    if (tok < cu_q[0] || tok >= cu_q[B]) return;
  }
  const float2* ml = reinterpret_cast<const float2*>(ws_ml) + row * n_splits;
  float m = -INFINITY;
  for (int s = lane; s < n_splits; s += 32) m = fmaxf(m, ml[s].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  float acc[kC] = {}, l = 0.0f;
  for (int s0 = 0; s0 < n_splits; s0 += 32) {
    float w_lane = 0.0f;
    if (s0 + lane < n_splits) {
      const float2 v = ml[s0 + lane];
      w_lane = v.x == -INFINITY ? v.y : ex2(v.x - m) * v.y;
    }
    const int n = min(32, n_splits - s0);
    for (int s = 0; s < n; ++s) {
      const float w = __shfl_sync(0xffffffffu, w_lane, s);
      if (w == 0.0f) continue;
      l += w;
      const float* src = ws_o + (row * n_splits + s0 + s) * D + lane * kC;
      float v[kC];
      if constexpr (kC == 4)
        *reinterpret_cast<float4*>(v) = *reinterpret_cast<const float4*>(src);
      else
        *reinterpret_cast<float2*>(v) = *reinterpret_cast<const float2*>(src);
#pragma unroll
      for (int c = 0; c < kC; ++c) acc[c] = fmaf(w, v[c], acc[c]);
    }
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  uint32_t* dst = reinterpret_cast<uint32_t*>(out + row * D + lane * kC);
#pragma unroll
  for (int c = 0; c < kC; c += 2) dst[c / 2] = pack2<BF16>(acc[c] * inv, acc[c + 1] * inv);
  if (lane == 0) lse[row] = l == 0.0f ? -INFINITY : (m + lg2(l)) * 0.69314718055994531f;
}

template <int D, bool BF16>
static int launch_merge_variant(const PagedArgs& a, int n_splits, cudaStream_t stream) {
  float *ws_o, *ws_ml;
  paged_parts(a, D, n_splits, ws_o, ws_ml);
  const size_t rows = static_cast<size_t>(a.total_q) * a.Hq;
  const uint64_t blocks = (rows + kMergeWarps - 1) / kMergeWarps;
  if (blocks > 0x7fffffffull) return -2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(kMergeWarps * 32);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, attn_paged_merge_kernel<D, BF16>, static_cast<const float*>(ws_o),
                         static_cast<const float*>(ws_ml), a.cu_q, a.B, a.Hq, rows, n_splits,
                         static_cast<uint16_t*>(a.o), a.lse) != cudaSuccess)
    return -5;
  return cudaGetLastError() == cudaSuccess ? 0 : -5;
}

int launch_paged_merge(const PagedArgs& a, int n_splits, cudaStream_t stream) {
  if (a.d == 64)
    return a.bf16 ? launch_merge_variant<64, true>(a, n_splits, stream)
                  : launch_merge_variant<64, false>(a, n_splits, stream);
  return a.bf16 ? launch_merge_variant<128, true>(a, n_splits, stream)
                : launch_merge_variant<128, false>(a, n_splits, stream);
}

int launch_attn_fwd_paged(const PagedArgs& a, cudaStream_t stream) {
  if (paged_few_rows(a)) return launch_attn_paged_few(a, stream);
  if (a.d == 64)
    return a.bf16 ? launch_paged_variant<64, true, kKvRows>(a, nullptr, 0, stream) : launch_paged_variant<64, false, kKvRows>(a, nullptr, 0, stream);
  if (a.d == 128)
    return a.bf16 ? launch_paged_variant<128, true, kKvRows>(a, nullptr, 0, stream) : launch_paged_variant<128, false, kKvRows>(a, nullptr, 0, stream);
  return -2;
}

}  // namespace attn
