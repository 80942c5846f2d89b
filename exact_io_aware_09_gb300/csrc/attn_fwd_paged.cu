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
#include "attn_fwd_two.cuh"
#include "attn_rows.cuh"

namespace attn {

namespace {

constexpr int kSms = 152;  // SMs of a GB300, two blocks each
constexpr int kMaxSplits = 128;
// Measured, us: a 64-key step and a block's start and end with two blocks on an SM, with one alone; the
// merge's launch, and its bytes (written and read) per us.
constexpr double kStepTwo = 0.88, kItemTwo = 4.0, kStepOne = 0.6, kItemOne = 3.5;
constexpr double kMerge = 4.0, kMergeBytes = 5e6;

struct PagedSplit {
  int tile_tokens, n_qtiles, n_splits, split_steps;
};

// How a call's work is cut.  An item is one query tile of one key/value head of a sequence; its 64-key
// steps are cut into the number of splits that is estimated to finish first: rounds of blocks over the
// SMs, two on each, a last round of few blocks running one on an SM, and the merge.  (The lengths are
// the caller's bounds: what the sequences really hold is on the device.)
PagedSplit paged_split(int B, int Hq, int Hkv, int max_q, int max_k, int window, int sinks, int d) {
  PagedSplit s;
  s.tile_tokens = kWM / (Hq / Hkv);
  s.n_qtiles = (max_q + s.tile_tokens - 1) / s.tile_tokens;
  long long steps = (static_cast<long long>(max_k) + kWN - 1) / kWN;
  if (window >= 0) {
    const long long near = (static_cast<long long>(window) + s.tile_tokens) / kWN + 2 +
                           (static_cast<long long>(sinks) + kWN - 1) / kWN;
    if (near < steps) steps = near;
  }
  const long long items = static_cast<long long>(B) * Hkv * s.n_qtiles;
  const double part_bytes = 2.0 * 4.0 * d * B * static_cast<double>(max_q) * Hq;
  s.n_splits = 1;
  s.split_steps = static_cast<int>(steps);
  double best = -1.0;
  for (int n = 1; n <= kMaxSplits && n <= steps; ++n) {
    const long long per = (steps + n - 1) / n, blocks = items * n;
    const double two = per * kStepTwo + kItemTwo, one = per * kStepOne + kItemOne;
    const long long left = blocks % (2 * kSms);
    double cost = static_cast<double>(blocks / (2 * kSms)) * two + (left == 0 ? 0.0 : left <= kSms ? one : two);
    if (n > 1) cost += kMerge + n * part_bytes / kMergeBytes;
    if (best < 0 || cost < best) {
      best = cost;
      s.split_steps = static_cast<int>(per);
      s.n_splits = static_cast<int>((steps + per - 1) / per);
    }
  }
  return s;
}

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
  const size_t tok = row / Hq;
  if (static_cast<long long>(tok) < cu_q[0] || static_cast<long long>(tok) >= cu_q[B]) return;
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

template <int D, bool BF16>
static int launch_paged_variant(const PagedArgs& a, cudaStream_t stream) {
  using L = WinLayout<D>;
  const PagedSplit sp = paged_split(a.B, a.Hq, a.Hkv, a.max_q, a.max_k, a.window, a.sinks, D);
  const int G = a.Hq / a.Hkv;
  const uint64_t row = static_cast<uint64_t>(D) * 2;
  const uint64_t tokens = static_cast<uint64_t>(a.num_pages) * a.page_size;
  const uint32_t box = static_cast<uint32_t>(a.page_size < kWN ? a.page_size : kWN);
  CUtensorMap tq, tk, tv, to;
  if (!make_tmap_3d(&tq, a.q, BF16, D, a.Hq, a.total_q, row, row * a.Hq, 64, G, sp.tile_tokens) ||
      !make_tmap_3d(&to, a.o, BF16, D, a.Hq, a.total_q, row, row * a.Hq, 64, G, sp.tile_tokens) ||
      !make_tmap_3d(&tk, a.k_pages, BF16, D, a.Hkv, tokens, row, row * a.Hkv, 64, 1, box) ||
      !make_tmap_3d(&tv, a.v_pages, BF16, D, a.Hkv, tokens, row, row * a.Hkv, 64, 1, box))
    return -5;
  PagedParams p = {};
  p.o = a.o;
  p.lse = a.lse;
  p.status = device_status_ptr();
  if (!p.status) return -5;
  p.Hq = a.Hq;
  p.Hkv = a.Hkv;
  p.n_qtiles = sp.n_qtiles;
  p.G = G;
  p.window = a.window;
  p.sinks = a.sinks;
  const uint64_t planes = static_cast<uint64_t>(a.B) * a.Hkv;
  if (planes > 0x7fffffffull) return -2;
  p.BH = static_cast<int>(planes);
  {
    // planes whose cache fills about half of L2 walk their query tiles together
    uint64_t group = (64ull << 20) / (2ull * a.max_k * D * 2);
    if (group < 1) group = 1;
    if (group > planes) group = planes;
    p.head_group = static_cast<int>(group);
  }
  p.sl2 = a.scale * 1.4426950408889634f;
  p.block_table = a.block_table;
  p.cu_q = a.cu_q;
  p.seqlens = a.seqlens;
  while ((1 << p.page_log2) < a.page_size) ++p.page_log2;
  p.max_pages = a.max_pages;
  p.num_pages = a.num_pages;
  p.total_q = a.total_q;
  p.max_q = a.max_q;
  p.max_k = a.max_k;
  p.tile_tokens = sp.tile_tokens;
  p.n_splits = sp.n_splits;
  p.split_steps = sp.split_steps;
  if (sp.n_splits > 1) paged_parts(a, D, sp.n_splits, p.ws_o, p.ws_ml);
  auto kern = sp.n_qtiles == 1 ? attn_fwd_two_kernel<D, BF16, true, true> : attn_fwd_two_kernel<D, BF16, true>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kBytes) !=
      cudaSuccess)
    return -5;
  const uint64_t blocks = planes * sp.n_qtiles * sp.n_splits;
  if (blocks > 0x7fffffffull) return -2;
  kern<<<static_cast<unsigned>(blocks), two_threads(true), L::kBytes, stream>>>(tq, tk, tv, to, p);
  if (cudaGetLastError() != cudaSuccess) return -5;
  return sp.n_splits == 1 ? 0 : launch_paged_merge(a, sp.n_splits, stream);
}

int launch_attn_fwd_paged(const PagedArgs& a, cudaStream_t stream) {
  if (paged_few_rows(a)) return launch_attn_paged_few(a, stream);
  if (a.d == 64)
    return a.bf16 ? launch_paged_variant<64, true>(a, stream) : launch_paged_variant<64, false>(a, stream);
  if (a.d == 128)
    return a.bf16 ? launch_paged_variant<128, true>(a, stream) : launch_paged_variant<128, false>(a, stream);
  return -2;
}

}  // namespace attn
