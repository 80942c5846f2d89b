// Declarations shared by the split-KV decode kernels (16-bit and quantised cache).
#pragma once
#include "internal.h"
#include "ptx.cuh"

namespace attn {

constexpr int kDecTok = 64;      // tokens per ring stage
constexpr int kDecWarps = 4;     // compute warps, 16 tokens of each stage apiece
constexpr int kDecThreads = 160;  // + one producer warp
constexpr int kDecStages = 3;
constexpr int kMaxGroup = 16;    // query heads per key/value head (rows of the m16 tile)

struct DecParams {
  const uint16_t* q;   // [B, Hq, D]
  const int32_t* cu;   // [B + 1] (packed cache)
  const int32_t* block_table;  // [B, max_pages] (paged cache) or null
  const int32_t* seqlens;      // [B] (paged cache)
  int page_size, page_log2, max_pages, num_pages;
  int box_log2;        // log2 of the rows of one TMA box: min(page_size, 64); 64 when packed
  float* ws_o;         // [B * Hq * max_splits, D]  normalised partial outputs
  float* ws_ml;        // [B * Hq * max_splits, 2]  (m in log2 units, l)
  int* status;
  int Hq, Hkv, G, capacity, max_seqlen, split, max_splits;
  float sl2;
};

__device__ __forceinline__ bool dec_warp_wait(uint32_t bar, uint32_t parity, volatile int* abort,
                                              int* status) {
  const bool ok = wait_bounded(bar, parity, abort, status);
  return __all_sync(0xffffffffu, ok);
}

__device__ __forceinline__ bool lengths_ok(const DecParams& p, int t_start, int t_stop) {
  const int len = t_stop - t_start;
  return t_start >= 0 && len >= 0 && len <= p.max_seqlen && t_stop <= p.capacity;
}

// Sequence b's tokens: rows [t_start, t_stop) of the packed cache, or logical positions
// [0, seqlens[b]) of a paged one.  False for lengths the caller's bounds do not allow.
__device__ __forceinline__ bool seq_bounds(const DecParams& p, int b, int& t_start, int& t_stop) {
  if (p.block_table) {
    t_start = 0;
    t_stop = p.seqlens[b];
    return t_stop >= 0 && t_stop <= p.max_seqlen &&
           ((t_stop + p.page_size - 1) >> p.page_log2) <= p.max_pages;
  }
  t_start = p.cu[b];
  t_stop = p.cu[b + 1];
  return lengths_ok(p, t_start, t_stop);
}

// Launches the merge of the partial states a split kernel writes (attn_decode.cu) as a programmatic
// dependent of that kernel; p as the split kernel's.  Returns 0 or an attn_status_t value.
int launch_decode_merge(const DecParams& p, int d, bool bf16, int B, void* o, float* lse,
                        cudaStream_t stream);

}  // namespace attn
