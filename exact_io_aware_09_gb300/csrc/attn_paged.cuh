// How the work of a chunk over a paged cache is cut, and its launch: for the 16-bit cache
// (attn_fwd_paged.cu) and the 4-bit one (attn_paged_fp4_chunk.cu).
#pragma once
#include "attn_fwd_two.cuh"

namespace attn {

constexpr int kPagedSms = 152;  // SMs of a GB300, two blocks each
constexpr int kPagedMaxSplits = 128;
// Measured over the 16-bit cache, us: a 64-key step and a block's start and end with two blocks on an SM, with one alone; the
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
inline PagedSplit paged_split(int B, int Hq, int Hkv, int max_q, int max_k, int window, int sinks, int d) {
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
  for (int n = 1; n <= kPagedMaxSplits && n <= steps; ++n) {
    const long long per = (steps + n - 1) / n, blocks = items * n;
    const double two = per * kStepTwo + kItemTwo, one = per * kStepOne + kItemOne;
    const long long left = blocks % (2 * kPagedSms);
    double cost = static_cast<double>(blocks / (2 * kPagedSms)) * two + (left == 0 ? 0.0 : left <= kPagedSms ? one : two);
    if (n > 1) cost += kMerge + n * part_bytes / kMergeBytes;
    if (best < 0 || cost < best) {
      best = cost;
      s.split_steps = static_cast<int>(per);
      s.n_splits = static_cast<int>((steps + per - 1) / per);
    }
  }
  return s;
}

// The chunk over a 16-bit cache (kKvRows), over a 4-bit cache's codes c (kKvCodes) or over its f16 copy
// (kKvCopy: a.k_pages and v_pages [B, copy_rows, Hkv, d]).
template <int D, bool BF16, int KV>
static int launch_paged_variant(const PagedArgs& a, const CacheFp4* c, int copy_rows, cudaStream_t stream) {
  using L = WinLayout<D, KV == kKvCodes>;
  const PagedSplit sp = paged_split(a.B, a.Hq, a.Hkv, a.max_q, a.max_k, a.window, a.sinks, D);
  const int G = a.Hq / a.Hkv;
  const uint64_t row = static_cast<uint64_t>(D) * 2;
  const bool copy = KV == kKvCopy;
  const uint64_t tokens = copy ? static_cast<uint64_t>(a.B) * copy_rows
                               : static_cast<uint64_t>(a.num_pages) * a.page_size;
  const uint32_t box = static_cast<uint32_t>(a.page_size < kWN && !copy ? a.page_size : kWN);
  CUtensorMap tq, tk = {}, tv = {}, to;
  if (!make_tmap_3d(&tq, a.q, BF16, D, a.Hq, a.total_q, row, row * a.Hq, 64, G, sp.tile_tokens) ||
      !make_tmap_3d(&to, a.o, BF16, D, a.Hq, a.total_q, row, row * a.Hq, 64, G, sp.tile_tokens))
    return -5;
  if (KV != kKvCodes &&
      (!make_tmap_3d(&tk, a.k_pages, BF16 && !copy, D, a.Hkv, tokens, row, row * a.Hkv, 64, 1, box) ||
       !make_tmap_3d(&tv, a.v_pages, BF16 && !copy, D, a.Hkv, tokens, row, row * a.Hkv, 64, 1, box)))
    return -5;
  typename TwoOf<true, KV>::Params p = {};
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
    uint64_t group = (64ull << 20) / (2ull * a.max_k * (KV == kKvCodes ? D / 2 + D / 16 : D * 2));
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
  if constexpr (KV == kKvCodes) {
    p.k_codes = c->k_codes;
    p.v_codes = c->v_codes;
    p.k_scales = c->k_scales;
    p.v_scales = c->v_scales;
  }
  if constexpr (KV == kKvCopy) p.copy_rows = copy_rows;
  auto kern = attn_fwd_two_kernel<D, BF16, true, false, KV>;
  if constexpr (KV != kKvCopy) {
    if (sp.n_qtiles == 1) kern = attn_fwd_two_kernel<D, BF16, true, true, KV>;
  }
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kBytes) !=
      cudaSuccess)
    return -5;
  const uint64_t blocks = planes * sp.n_qtiles * sp.n_splits;
  if (blocks > 0x7fffffffull) return -2;
  kern<<<static_cast<unsigned>(blocks), two_threads(true, KV), L::kBytes, stream>>>(tq, tk, tv, to, p);
  if (cudaGetLastError() != cudaSuccess) return -5;
  return sp.n_splits == 1 ? 0 : launch_paged_merge(a, sp.n_splits, stream);
}

}  // namespace attn
