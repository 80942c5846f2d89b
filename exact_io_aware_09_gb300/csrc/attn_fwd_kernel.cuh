// Prefill forward: exact attention, one fused persistent kernel per call, sm_103a.
//
// Schedule (the FA-2 loop of "FlashAttention and GPU Data Movement", section 2): a work item is
// one 128-row query tile of one (batch, query head); its 128-key K/V tiles stream through shared
// memory and the online-softmax state stays on chip until O and the log-sum-exp are written once
// at the end.  The grid has one block per work item, but only one block fits on an SM: a running
// block takes over the items of blocks that have not started yet (cluster launch control), so
// each SM runs one long-lived block whose pipelines run on from one item into the next — the
// next item's Q/K/V loads and first score MMAs overlap the current item's last tiles and
// epilogue.  Items are taken in launch order: the query heads of one key/value head adjacent (the
// K/V tiles they share stay in L2) and, inside a head, the longest query tiles first (under the
// causal mask a tile's key range grows with its row index), which keeps the tail of the grid short.
//
// Roles inside a thread block (384 threads):
//   warps 0-7  softmax, two warpgroups taking alternate K/V tiles of the block's tile sequence;
//              thread r of a warpgroup owns query row r.  Reads S_j from tensor memory, applies
//              the scale, the causal/ragged mask and the online-softmax update ("FlashAttention
//              and GPU Data Movement", section 3.1), writes P_j back to tensor memory as 16-bit
//              pairs and rescales the accumulator when the row maximum moved.  The warpgroup that
//              ran an item's last tile runs its epilogue O = a / l, L = m + ln l, with the other
//              warpgroup's partial row sum handed over through shared memory.
//   warp 8     work scheduler (cluster launch control) and TMA producer of Q and the K ring.
//   warp 11    TMA producer of the V ring.
//   warp 9     tcgen05 issuer of S_j = Q K_j^T (both operands in shared memory, fp32 result in
//              tensor memory); allocates and frees the 512 tensor-memory columns.
//   warp 10    tcgen05 issuer of O += P_j V_j (P from tensor memory, V from shared memory, fp32
//              accumulator in tensor memory).
// Tensor memory: S buffers at columns 0 and 128 (double-buffered so Q K_{j+1}^T runs while the
// softmax of tile j runs), the output accumulator at column 256, two P buffers after it.  A
// softmax releases its S buffer as soon as it has read it, so the score MMAs run ahead.
//
// Every barrier phase is counted over the block's whole tile sequence (all items), so the rings,
// buffers and hand-offs need no reset between items.
//
// Variants.  FP8: E4M3 operands (attn_fp8.cu).  SINKS: the first keys stay visible outside the
// sliding window; an item's key tiles are those that hold sinks, then the window's.  PAGED: a chunk
// of new tokens of each sequence over a paged cache (attn_fwd_paged.cu).  A masked score of the last
// two is replaced by bits, so that a NaN of a key no row sees does not spread; the dense variants add
// -inf, which costs one operation less per score.
//
// Departures from the pages' kernels (prior art for A100/H100/B200): accumulators live in tensor
// memory instead of registers, P is handed to the second MMA through tensor memory instead of
// shared memory or registers, exponentials are base 2 with the scale folded into one FMA, and the
// accumulator is rescaled only when a row maximum rises by more than 2^8 (the final division uses
// the same stale maximum in l, so the result is unchanged: "FlashAttention Explained", section on
// FlashAttention-4, conditional rescaling).
#pragma once
#include <cstdio>

#include "internal.h"
#include "ptx.cuh"

namespace attn {

// Optional per-tile timestamps for schedule analysis; compiled in only when ATTN_FWD_TRACE is
// defined (never in the library build).
#ifdef ATTN_FWD_TRACE
__device__ unsigned long long g_fwd_trace[8][80][28];
#define FWD_TRACE(j, ev)                                                                      \
  do {                                                                                        \
    if (trace_slot >= 0 && (j) < 80) {                                                        \
      unsigned long long t_;                                                                  \
      asm volatile("mov.u64 %0, %%clock64;" : "=l"(t_));                                      \
      g_fwd_trace[trace_slot][(j)][(ev)] = t_;                                                \
    }                                                                                         \
  } while (0)
#else
#define FWD_TRACE(j, ev) \
  do {                   \
  } while (0)
#endif

constexpr int kBlockM = 128;
constexpr int kBlockN = 128;
constexpr int kFwdThreads = 384;  // warps 0-7 softmax, 8 and 11 TMA, 9-10 MMA issue
constexpr int kSoftmaxThreads = 128;  // one softmax warpgroup (thread = query row)
constexpr int kProducerWarp = 8, kQkWarp = 9, kPvWarp = 10, kVProducerWarp = 11;
// Readers of the work-item ring: lane 0 of warps 9, 10, 11 and of each softmax warp.
constexpr uint32_t kItemReaders = 3 + 8;
constexpr uint32_t kTmemCols = 512;
// Registers per thread after the rebalancing at the role split (launched with 168).
constexpr uint32_t kRegsSoftmax = 184, kRegsIssue = 136;
static_assert(2 * 128 * kRegsSoftmax + 128 * kRegsIssue <= kFwdThreads * 168, "register split");
constexpr uint32_t kColS0 = 0, kColS1 = 128, kColO = 256;
// P buffers follow O: columns 256 + d and 256 + d + 64 (16-bit pairs, 64 columns each).
template <int D>
struct PCols {
  static constexpr uint32_t kP0 = kColO + D, kP1 = kColO + D + 64;
  static_assert(kP1 + 64 <= kTmemCols, "tensor memory budget");
};
constexpr float kRescaleThreshold = 8.0f;  // log2 units: rescale only if the max rises by > 2^8
// FP8: P enters the P V product as 2^kPShift8 P in E4M3.  The maximum moves whenever it rises by
// more than 2^kRescaleThreshold8, so P <= 2^3.8 and 2^5 P <= 2^8.8 < 448, inside E4M3's range;
// the row sum carries the same factor, which the epilogue removes.  (A lower threshold keeps
// more of P's small values out of E4M3's subnormal range but makes the rescale of O, which
// waits for the previous P V, frequent: on N(0,1) inputs a warp of 32 rows rescales on 43% of
// its tiles at 2^1 and on 0.3% at 2^3.8.)
constexpr float kRescaleThreshold8 = 3.8f;
constexpr int kPShift8 = 5;
constexpr uint32_t kSubTile = 128 * 128;   // bytes of one 64-column, 128-row swizzled sub-tile
constexpr uint64_t kDrainLimitNs = 100000000ull;

struct FwdParams {
  void* o;
  float* lse;
  int* status;
  int Hq, Hkv, N_q, N_kv;
  int n_qtiles, group, causal;
  int BH;           // batch * Hq
  int head_group;   // query heads walked together, longest query tiles first (see decode_item)
  int window;       // sliding window, keys behind the diagonal (-1: none)
  int n_kvtiles;    // key tiles of the sequence (row length of block_mask)
  const uint8_t* block_mask;  // [query tile][key tile], nonzero = compute; null: every tile
  // FP8 operands: E4M3 block scales of Q [B*Hq][query tile], K [B*Hkv][key tile], V [B*Hkv]
  const float* q_scale;
  const float* k_scale;
  const float* v_scale;
  float sl2;  // scale * log2(e)
};

// Parameters of the variants whose first `sinks` keys stay visible outside the window.
struct FwdParamsSinks : FwdParams {
  int sinks;
};

// Parameters of the variant that runs chunks of new tokens over a paged cache.  Here n_qtiles,
// BH and head_group count query tiles of the longest chunk and (sequence, key/value head)
// planes.
struct FwdParamsPaged : FwdParamsSinks {
  const int32_t* block_table;  // [B, max_pages]
  const int32_t* cu_q;         // [B + 1] packed rows of each sequence's new tokens
  const int32_t* seqlens;      // [B] cached tokens, the new ones included
  int page_log2, max_pages, num_pages;
  int total_q, max_q, max_k;
  int tile_tokens;             // tokens of one query tile: 128 / group
  int n_splits, split_tiles;   // key tiles of one split (n_splits == 1: the whole item)
  float* ws_o;                 // [total_q * Hq, n_splits, D] normalised partial outputs
  float* ws_ml;                // [total_q * Hq, n_splits, 2] (m in log2 units, l)
};

template <bool SINKS, bool PAGED>
struct FwdParamsOf {
  using T = FwdParams;
};
template <>
struct FwdParamsOf<true, false> {
  using T = FwdParamsSinks;
};
template <>
struct FwdParamsOf<true, true> {
  using T = FwdParamsPaged;
};

// Barriers (8 bytes each), in this order after the K/V rings.
enum FwdBar : uint32_t {
  kBarQFull = 0,       // Q tile landed (TMA)
  kBarQEmpty = 1,      // the item's last score MMA finished: Q may be replaced
  kBarS = 2,           // [2] S buffer written (MMA commit)
  kBarSFree = 4,       // [2] S buffer read by the softmax (128 arrivals)
  kBarP = 6,           // [2] P buffer written, O rescaled (128 arrivals)
  kBarO = 8,           // [2] P V of a tile of that parity finished (MMA commit)
  kBarM = 10,          // [2][4] running maximum of a tile of that parity published, one barrier
                       // per warp (lane quarter): its 32 rows are all the partner warp needs
  kBarLFull = 18,      // [2] partial row sum handed to the epilogue (128 arrivals), by item parity
  kBarLEmpty = 20,     // [2] ... and read (128 arrivals)
  kBarItemFull = 22,   // [2] work-item ring slot written
  kBarItemEmpty = 24,  // [2] ... and read by every role (kItemReaders arrivals)
  kBarOStageFull = 26, // O of an item written to the staging buffer (128 arrivals)
  kBarClc = 27,        // cluster-launch-control answer landed
  kBarDrain = 28,      // both issuers' MMAs finished (two commits)
  kBarOStage = 29,     // the TMA store of the previous epilogue has read the O staging buffer
  kBarRagged = 29,     // paged cache (no staging buffer): a sequence's last V tile landed
  kNumFixedBars = 30
};

template <int D, int KS, int VS, bool FP8 = false>
struct FwdLayout {
  static constexpr uint32_t kElem = FP8 ? 1 : 2;  // bytes per Q/K/V element
  static constexpr uint32_t kQBytes = kBlockM * D * kElem;
  static constexpr uint32_t kKVBytes = kBlockN * D * kElem;
  static constexpr uint32_t kOBytes = kBlockM * D * 2;  // O is written in 16 bits
  static constexpr uint32_t kQ = 0;
  static constexpr uint32_t kK = kQ + kQBytes;          // K ring, KS slots
  static constexpr uint32_t kV = kK + KS * kKVBytes;    // V ring, VS slots
  static constexpr uint32_t kOst = kV + VS * kKVBytes;  // O staging for the TMA store
  // k_full[KS], k_empty[KS], v_full[VS], v_empty[VS], then the FwdBar barriers
  static constexpr uint32_t kBar = kOst + kOBytes;
  static constexpr uint32_t kFixedBar = kBar + 2 * (KS + VS) * 8;
  static constexpr uint32_t kMisc = kFixedBar + kNumFixedBars * 8;  // tmem slot, abort, ring[2]
  static constexpr uint32_t kClc = (kMisc + 16 + 15) & ~15u;        // 16-byte answer
  // running row maximum handed from one softmax warpgroup to the other: [row]
  static constexpr uint32_t kMrow = kClc + 16;
  // partial row sums handed to the epilogue warpgroup: [item parity][row]
  static constexpr uint32_t kLpart = kMrow + kBlockM * 4;
  // per softmax warp: the owed epilogue's item index, first row, (batch, head), last tile
  static constexpr uint32_t kEpState = kLpart + 2 * kBlockM * 4;
  static constexpr uint32_t kBytes = kEpState + 8 * 4 * 4 + 1024;  // + alignment slack
  // paged cache: O goes out without staging, and its room holds the work-item ring (two decoded
  // items) and the owed epilogues' data, 8 words per softmax warp
  static constexpr uint32_t kItems = kOst;
  static constexpr uint32_t kEpPaged = kOst + 256;
  static_assert(kBytes <= 232448, "shared memory per block");
};

// One work item: a 128-row query tile of one (batch, query head).
struct FwdItem {
  int bh;            // batch * Hq + query head
  int q0;            // first query row
  int kv_plane;      // batch * Hkv + key/value head
  int n_tiles;       // K/V tiles the rows of this tile see (those of the block pattern)
  int j_begin;       // first key tile of the span
  int lo_masked;     // key tiles below this need the window's lower-edge mask
  int first_masked;  // key tiles from this on need the causal or ragged-edge mask
  const uint8_t* pattern;  // this query tile's row of the block pattern, or null
};

// Work item of the sinks variant: the key tiles that hold the sinks come first, then those of
// the window; tile i of the item is key tile kv_tile_at(it, i).
struct FwdItemSinks : FwdItem {
  int sink_tiles;  // tiles before j_begin that hold sinks
  int i0;          // first tile of this item's part of that sequence
};

// Work item of the paged variant: the query tile's rows are (token, query head of the group)
// pairs, token major, of one key/value head; bh is the sequence.
struct FwdItemPaged : FwdItemSinks {
  int id;      // launch index; -1: no more work
  int tok0;    // packed row of the tile's first token (q0 is its index inside the chunk)
  int n_rows;  // rows that belong to the chunk
  int pos0;    // cache position of the first token
  int len;     // cached tokens of the sequence
  int split;
};
static_assert(sizeof(FwdItemPaged) <= 128, "item ring slot");

template <bool SINKS, bool PAGED>
struct FwdItemOf {
  using T = FwdItem;
};
template <>
struct FwdItemOf<true, false> {
  using T = FwdItemSinks;
};
template <>
struct FwdItemOf<true, true> {
  using T = FwdItemPaged;
};

__device__ __forceinline__ int kv_tile_at(const FwdItemSinks& it, int i) {
  const int idx = it.i0 + i;
  return idx < it.sink_tiles ? idx : it.j_begin + idx - it.sink_tiles;
}

// Key tiles of an item in order: j_begin, j_begin + 1, ... skipping those the block pattern
// leaves out.  Every role walks the same sequence.
__device__ __forceinline__ int next_kv_tile(const FwdItem& it, int j) {
  if (it.pattern)
    while (!it.pattern[j]) ++j;
  return j;
}

// Work item `id` in launch order.  The (batch, query head) pairs are cut into groups of
// head_group consecutive ones (the query heads of one key/value head are consecutive, and
// head_group is a multiple of their number) whose K/V planes fill about half of L2; a group's
// items run longest query tile first across all its heads (under the causal mask a tile's key
// range grows with its row index), so that the last items of the grid are short ones while the
// K/V tiles in use stay in L2.
__device__ __forceinline__ FwdItem decode_item(int id, const FwdParams& p) {
  FwdItem it;
  const int span = p.head_group * p.n_qtiles;  // items per group
  const int g = id / span;
  const int r = id - g * span;
  const int h0 = g * p.head_group;
  const int gh = min(p.head_group, p.BH - h0);  // heads in this group (the last may be short)
  const int qt = p.n_qtiles - 1 - r / gh;
  it.bh = h0 + r % gh;
  it.q0 = qt * kBlockM;
  const int h = it.bh % p.Hq;
  const int b = it.bh / p.Hq;
  it.kv_plane = b * p.Hkv + h / p.group;
  int j_end;
  kv_tile_span(qt, kBlockM, kBlockN, p.N_q, p.N_kv, p.causal, p.window, it.j_begin, j_end,
               it.lo_masked, it.first_masked);
  it.pattern = nullptr;
  it.n_tiles = j_end - it.j_begin;
  if (p.block_mask) {
    it.pattern = p.block_mask + static_cast<size_t>(qt) * p.n_kvtiles;
    int n = 0;
    for (int j = it.j_begin; j < j_end; ++j) n += it.pattern[j] ? 1 : 0;
    it.n_tiles = n;
  }
  return it;
}

// The sinks variant: the same item with the key tiles that hold the first `sinks` keys in front
// of the window's.  A tile below j_begin lies wholly before every row's window, so of it every
// row sees the sinks and nothing else.
__device__ __forceinline__ FwdItemSinks decode_item(int id, const FwdParamsSinks& p) {
  FwdItemSinks it;
  static_cast<FwdItem&>(it) = decode_item(id, static_cast<const FwdParams&>(p));
  it.sink_tiles = min((p.sinks + kBlockN - 1) / kBlockN, it.j_begin);
  it.i0 = 0;
  it.n_tiles += it.sink_tiles;
  return it;
}

// The paged variant: launch index -> (plane, query tile, split), planes grouped and walked longest
// query tile first as above, a tile's splits side by side.  The grid covers the longest chunk the
// caller announced; items past a sequence's own chunk have no rows.
__device__ __forceinline__ FwdItemPaged decode_item(int id, const FwdParamsPaged& p) {
  FwdItemPaged it;
  it.id = id;
  it.pattern = nullptr;
  it.split = id % p.n_splits;
  const int u = id / p.n_splits;
  const int span = p.head_group * p.n_qtiles;
  const int g = u / span;
  const int r = u - g * span;
  const int h0 = g * p.head_group;
  const int gh = min(p.head_group, p.BH - h0);
  const int plane = h0 + r % gh;
  const int b = plane / p.Hkv;
  it.bh = b;
  it.kv_plane = plane - b * p.Hkv;
  it.q0 = (p.n_qtiles - 1 - r / gh) * p.tile_tokens;
  it.n_tiles = 0;
  it.n_rows = 0;
  it.j_begin = it.lo_masked = it.first_masked = it.sink_tiles = it.i0 = 0;
  const int c0 = p.cu_q[b], n = p.cu_q[b + 1] - c0;
  const int len = p.seqlens[b];
  it.tok0 = c0 + it.q0;
  it.len = len;
  it.pos0 = len - n + it.q0;
  if (c0 < 0 || n < 0 || n > p.max_q || n > p.total_q - c0 || len < n || len > p.max_k ||
      ((len - 1) >> p.page_log2) >= p.max_pages) {
    latch_status(p.status, kStatusBadLengths);
    return it;
  }
  if (it.q0 >= n) return it;
  const int n_tok = min(p.tile_tokens, n - it.q0);
  it.n_rows = n_tok * p.group;
  const int pos1 = it.pos0 + n_tok - 1;  // position of the tile's last token
  const int j_end = pos1 / kBlockN + 1;
  it.first_masked = min((it.pos0 + 1) / kBlockN, j_end);
  if (p.window >= 0) {
    it.j_begin = max(it.pos0 - p.window, 0) / kBlockN;
    it.lo_masked = (max(pos1 - p.window, 0) + kBlockN - 1) / kBlockN;
    it.sink_tiles = min((p.sinks + kBlockN - 1) / kBlockN, it.j_begin);
  }
  const int all = it.sink_tiles + j_end - it.j_begin;
  it.i0 = it.split * p.split_tiles;
  it.n_tiles = min(max(all - it.i0, 0), p.split_tiles);
  return it;
}

__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort,
                                          int* status) {
  const bool ok = wait_bounded(bar, parity, abort, status);
  return __all_sync(0xffffffffu, ok);
}

// The pages of a 128-key tile as a producer warp loads them: lane i the i-th, `rows` rows each
// (the whole tile from one page when a page holds 128 tokens or more).
struct PagedTile {
  int lane, rows, rows_log2;
  __device__ __forceinline__ PagedTile(const FwdParamsPaged& p, int lane_) : lane(lane_) {
    rows_log2 = min(p.page_log2, 7);
    rows = 1 << rows_log2;
  }
  // This lane's block-table entry for tile kt; -1 where the lane has no page of it that holds
  // tokens.
  __device__ __forceinline__ int entry(const FwdParamsPaged& p, const FwdItemPaged& it,
                                       int kt) const {
    const int t = kt * kBlockN + (lane << rows_log2);
    if ((lane << rows_log2) >= kBlockN || t >= it.len) return -1;
    return p.block_table[static_cast<size_t>(it.bh) * p.max_pages + (t >> p.page_log2)];
  }
  // The pool row the lane's load starts at; -1: no load.  An entry outside the pool is reported.
  __device__ __forceinline__ int row(const FwdParamsPaged& p, const FwdItemPaged& it, int kt,
                                     int entry, bool report) const {
    const int t = kt * kBlockN + (lane << rows_log2);
    if ((lane << rows_log2) >= kBlockN || t >= it.len) return -1;
    if (entry < 0 || entry >= p.num_pages) {
      if (report) latch_status(p.status, kStatusBadLengths);
      return -1;
    }
    return (entry << p.page_log2) + (t & ((1 << p.page_log2) - 1));
  }
};

// Epilogue of one item for the softmax thread of row r (its warpgroup did not run the item's
// last tile; that P V has finished): adds the partial sum handed over by the other warpgroup to
// its own, writes O = a / l (the accumulator row read from tensor memory 32 columns at a time)
// to the staging buffer of the TMA store (128-byte-swizzled sub-tiles of 64 columns), and
// L = m + ln l to global memory.  m_fin is the item's final maximum and (l_own, m_own) this
// warpgroup's partial sum and the maximum it refers to.
template <int D, bool BF16, bool FP8 = false, bool SINKS = false>
__device__ __forceinline__ bool run_epilogue(uint32_t o_tmem, float m_fin, float l_own,
                                             float m_own, int item, int q0, int bh, int r,
                                             uint32_t fbars, const float* lpart, uint8_t* staging,
                                             const FwdParams& p, volatile int* abort_flag) {
  // Handover slot item % 2; this is its (item / 2)-th use.
  const uint32_t slot = item & 1;
  if (!warp_wait(fbars + 8u * (kBarLFull + slot), (item >> 1) & 1, abort_flag, p.status))
    return false;
  float l_row = lpart[slot * kBlockM + r];
  mbar_arrive(fbars + 8u * (kBarLEmpty + slot));
  if (m_own != -INFINITY) l_row += l_own * ex2(m_own - m_fin);
  // FP8: the accumulator holds sum_j (2^5 p_j)_E4M3 v8_j with V = v8 * v_scale
  float out_scale = 1.0f;
  if constexpr (FP8) out_scale = p.v_scale[(bh / p.Hq) * p.Hkv + (bh % p.Hq) / p.group];
  const float inv_l = (l_row > 0.0f) ? out_scale / l_row : 0.0f;
  if (item >= 1 && !warp_wait(fbars + 8u * kBarOStage, (item - 1) & 1, abort_flag, p.status))
    return false;
#pragma unroll 1
  for (int c = 0; c < D / 32; ++c) {
    uint32_t o[32];
    tmem_ld32(o_tmem + c * 32, o);
    tmem_wait_ld();
#pragma unroll
    for (int q4 = 0; q4 < 4; ++q4) {
      uint4 w;
      w.x = pack2<BF16>(__uint_as_float(o[q4 * 8 + 0]) * inv_l,
                        __uint_as_float(o[q4 * 8 + 1]) * inv_l);
      w.y = pack2<BF16>(__uint_as_float(o[q4 * 8 + 2]) * inv_l,
                        __uint_as_float(o[q4 * 8 + 3]) * inv_l);
      w.z = pack2<BF16>(__uint_as_float(o[q4 * 8 + 4]) * inv_l,
                        __uint_as_float(o[q4 * 8 + 5]) * inv_l);
      w.w = pack2<BF16>(__uint_as_float(o[q4 * 8 + 6]) * inv_l,
                        __uint_as_float(o[q4 * 8 + 7]) * inv_l);
      const uint32_t chunk = c * 4 + q4;  // 16-byte chunk of the row
      *reinterpret_cast<uint4*>(staging + (chunk >> 3) * kSubTile + sw128(r, chunk & 7)) = w;
    }
  }
  fence_proxy_async_smem();
  mbar_arrive(fbars + 8u * kBarOStageFull);  // the P V issuer sends the TMA store
  const int row = q0 + r;
  if (row < p.N_q) {
    const float mu = (m_fin == -INFINITY) ? 0.0f : m_fin;
    const float shift = FP8 ? static_cast<float>(kPShift8) : 0.0f;
    p.lse[static_cast<size_t>(bh) * p.N_q + row] =
        (l_row > 0.0f || (SINKS && l_row != 0.0f))  // a NaN sum stays one
            ? (mu + lg2(l_row) - shift) * 0.69314718055994531f
            : -INFINITY;
  }
  return true;
}

// The same for the paged variant, whose rows go straight to global memory (a tile may end with
// the sequence, and the rows behind it belong to the next one): O in 16 bits and L, or with
// several splits the normalised fp32 row and its (m, l) for the merge.  ep: the owed epilogue's
// data (item index, packed row of the first token, key/value head, last tile, rows, split).
template <int D, bool BF16>
__device__ __forceinline__ bool paged_epilogue(uint32_t o_tmem, float m_fin, float l_own,
                                               float m_own, const volatile int* ep, int r,
                                               uint32_t fbars, const float* lpart,
                                               const FwdParamsPaged& p, volatile int* abort_flag) {
  const int item = ep[0];
  const uint32_t slot = item & 1;
  if (!warp_wait(fbars + 8u * (kBarLFull + slot), (item >> 1) & 1, abort_flag, p.status))
    return false;
  float l_row = lpart[slot * kBlockM + r];
  mbar_arrive(fbars + 8u * (kBarLEmpty + slot));
  if (m_own != -INFINITY) l_row += l_own * ex2(m_own - m_fin);
  const float inv_l = (l_row > 0.0f) ? 1.0f / l_row : (l_row == 0.0f ? 0.0f : l_row);
  const bool store = r < ep[4];
  const size_t row = static_cast<size_t>(ep[1] + r / p.group) * p.Hq + ep[2] * p.group + r % p.group;
  const size_t part = p.n_splits == 1 ? row : row * p.n_splits + ep[5];
#pragma unroll 1
  for (int c = 0; c < D / 32; ++c) {
    uint32_t o[32];
    tmem_ld32(o_tmem + c * 32, o);
    tmem_wait_ld();
    if (!store) continue;
    if (p.n_splits == 1) {
      uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.o) + part * D + c * 32);
#pragma unroll
      for (int q4 = 0; q4 < 4; ++q4)
        dst[q4] = make_uint4(pack2<BF16>(__uint_as_float(o[q4 * 8 + 0]) * inv_l,
                                         __uint_as_float(o[q4 * 8 + 1]) * inv_l),
                             pack2<BF16>(__uint_as_float(o[q4 * 8 + 2]) * inv_l,
                                         __uint_as_float(o[q4 * 8 + 3]) * inv_l),
                             pack2<BF16>(__uint_as_float(o[q4 * 8 + 4]) * inv_l,
                                         __uint_as_float(o[q4 * 8 + 5]) * inv_l),
                             pack2<BF16>(__uint_as_float(o[q4 * 8 + 6]) * inv_l,
                                         __uint_as_float(o[q4 * 8 + 7]) * inv_l));
    } else {
      float4* dst = reinterpret_cast<float4*>(p.ws_o + part * D + c * 32);
#pragma unroll
      for (int q4 = 0; q4 < 8; ++q4)
        dst[q4] = make_float4(__uint_as_float(o[q4 * 4 + 0]) * inv_l,
                              __uint_as_float(o[q4 * 4 + 1]) * inv_l,
                              __uint_as_float(o[q4 * 4 + 2]) * inv_l,
                              __uint_as_float(o[q4 * 4 + 3]) * inv_l);
    }
  }
  if (store) {
    const float mu = (m_fin == -INFINITY) ? 0.0f : m_fin;
    if (p.n_splits == 1)
      p.lse[row] = l_row == 0.0f ? -INFINITY : (mu + lg2(l_row)) * 0.69314718055994531f;
    else
      reinterpret_cast<float2*>(p.ws_ml)[part] = make_float2(m_fin, l_row);
  }
  return true;
}

template <int D, bool BF16, int KS, int VS, bool FP8 = false, bool SINKS = false,
          bool PAGED = false>
__global__ void __launch_bounds__(kFwdThreads, 1)
    attn_fwd_kernel(const __grid_constant__ CUtensorMap tm_q,
                    const __grid_constant__ CUtensorMap tm_k,
                    const __grid_constant__ CUtensorMap tm_v,
                    const __grid_constant__ CUtensorMap tm_o,
                    const typename FwdParamsOf<SINKS, PAGED>::T p) {
  static_assert(SINKS || !PAGED, "the paged variant takes the sinks variant's tile order");
  using L = FwdLayout<D, KS, VS, FP8>;
  using Item = typename FwdItemOf<SINKS, PAGED>::T;
  // 128-byte swizzled column chunks of a Q/K tile row: 64 16-bit or 128 8-bit elements
  constexpr int kChunks = FP8 ? 1 : D / 64;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);

  const uint32_t sQ = base + L::kQ;
  const uint32_t sK = base + L::kK;
  const uint32_t sV = base + L::kV;
  const uint32_t sOst = base + L::kOst;
  const uint32_t bars = base + L::kBar;
  const uint32_t fbars = base + L::kFixedBar;
#define BAR_K(s) (bars + 8u * (s))
#define BAR_KE(s) (bars + 8u * (KS + (s)))
#define BAR_V(s) (bars + 8u * (2u * KS + (s)))
#define BAR_VE(s) (bars + 8u * (2u * KS + VS + (s)))
#define FBAR(i) (fbars + 8u * (i))
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + L::kMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(gbase + L::kMisc + 4);
  volatile int* ring = reinterpret_cast<volatile int*>(gbase + L::kMisc + 8);  // [2] item ids
  const uint32_t clc_resp = base + L::kClc;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
#ifdef ATTN_FWD_TRACE
  const int trace_slot = (blockIdx.x < 8) ? static_cast<int>(blockIdx.x) : -1;
#endif

  if (threadIdx.x == 0) FWD_TRACE(79, 0);
  if (threadIdx.x == 0) {
    for (int s = 0; s < KS; ++s) {
      mbar_init(BAR_K(s), 1);
      mbar_init(BAR_KE(s), 1);
    }
    for (int s = 0; s < VS; ++s) {
      mbar_init(BAR_V(s), 1);
      mbar_init(BAR_VE(s), 1);
    }
    mbar_init(FBAR(kBarQFull), 1);
    mbar_init(FBAR(kBarQEmpty), 1);
    for (int b = 0; b < 2; ++b) {
      mbar_init(FBAR(kBarS + b), 1);
      mbar_init(FBAR(kBarSFree + b), kSoftmaxThreads);
      mbar_init(FBAR(kBarP + b), kSoftmaxThreads);
      mbar_init(FBAR(kBarO + b), 1);
      for (int q = 0; q < 4; ++q) mbar_init(FBAR(kBarM + b * 4 + q), 32);
      mbar_init(FBAR(kBarItemFull + b), 1);
      mbar_init(FBAR(kBarItemEmpty + b), kItemReaders);
      mbar_init(FBAR(kBarLFull + b), kSoftmaxThreads);
      mbar_init(FBAR(kBarLEmpty + b), kSoftmaxThreads);
    }
    mbar_init(FBAR(kBarOStageFull), kSoftmaxThreads);
    mbar_init(FBAR(kBarClc), 1);
    mbar_init(FBAR(kBarDrain), 2);  // one commit from each issuer
    mbar_init(FBAR(kBarOStage), 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == kQkWarp) {
    tmem_alloc(smem_u32(tmem_slot), kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  // Work item k of this block from the ring (single-thread readers; -1 = no more work).  The
  // paged variant's ring holds the decoded items, since decoding one reads global memory.
  [[maybe_unused]] volatile int* item_ring = reinterpret_cast<volatile int*>(gbase + L::kItems);
  constexpr int kItemWords = sizeof(FwdItemPaged) / 4;
  [[maybe_unused]] auto read_item = [&](int k) {
    union {
      FwdItemPaged it;
      int w[kItemWords];
    } u;
#pragma unroll
    for (int i = 0; i < kItemWords; ++i) u.w[i] = item_ring[(k & 1) * 32 + i];
    return u.it;
  };
  [[maybe_unused]] auto take_paged = [&](int k, FwdItemPaged& it) -> bool {
    if (!wait_bounded(FBAR(kBarItemFull + (k & 1)), (k >> 1) & 1, abort_flag, p.status))
      return false;
    it = read_item(k);
    mbar_arrive(FBAR(kBarItemEmpty + (k & 1)));
    return it.id >= 0;
  };
  auto take_item = [&](int k, int& id) -> bool {
    if (!wait_bounded(FBAR(kBarItemFull + (k & 1)), (k >> 1) & 1, abort_flag, p.status))
      return false;
    id = ring[k & 1];
    mbar_arrive(FBAR(kBarItemEmpty + (k & 1)));
    return true;
  };

  if (warp >= kProducerWarp) {
    // Warps 8-11 (one warpgroup) need few registers; the softmax warpgroups take the rest of
    // the 168 per thread the block was launched with: 2 x 128 x 184 + 128 x 136 = 384 x 168.
    setmaxnreg_dec<kRegsIssue>();
  if (warp == kProducerWarp) {
    // ----------------------------------------------------------------- scheduler + Q/K producer
    // Publishes the block's work items (its own first, then those of pending blocks it cancels)
    // and loads, per item, K_0, Q and then K_1, K_2, ...: a K slot is refilled as soon as its
    // score MMA finished, and Q once the previous item's last score MMA finished.  The next
    // item is requested when an item starts; as soon as the answer is in, its Q tile is pulled
    // into L2, so that the Q load at the item boundary is short.
    if constexpr (PAGED) {
      // The same by a whole warp: lane i loads the i-th page of a tile (its block-table entry is
      // read one tile ahead, while the previous tile waits for its slot), lane 0 does the rest.
      if (lane == 0) {
        prefetch_tmap(&tm_q);
        prefetch_tmap(&tm_k);
      }
      // Rows of the query tile that no token fills stay zero.
      const int rows_filled = p.tile_tokens * p.group;
      for (int i = lane; i < (kBlockM - rows_filled) * kChunks * 8; i += 32) {
        const int row = rows_filled + i / (kChunks * 8), c = i % (kChunks * 8);
        *reinterpret_cast<uint4*>(gbase + L::kQ + (c >> 3) * kSubTile + row * 128 + (c & 7) * 16) =
            make_uint4(0, 0, 0, 0);
      }
      fence_proxy_async_smem();
      __syncwarp();
      const uint32_t q_bytes = static_cast<uint32_t>(rows_filled) * D * 2;
      int id = static_cast<int>(blockIdx.x);
      bool clc_live = true, clc_pending = false;
      uint32_t clc_uses = 0;
      int T = 0, kq = 0;
      const PagedTile pages(p, lane);
      for (int k = 0;; ++k) {
        bool ok = true;
        if (lane == 0 && k >= 2)
          ok = wait_bounded(FBAR(kBarItemEmpty + (k & 1)), ((k >> 1) - 1) & 1, abort_flag, p.status);
        if (!__shfl_sync(0xffffffffu, ok, 0)) break;
        union {
          FwdItemPaged it;
          int w[kItemWords];
        } u;
        u.it.id = -1;
        if (id >= 0) u.it = decode_item(id, p);
        const FwdItemPaged& it = u.it;
        if (lane == 0) {
#pragma unroll
          for (int i = 0; i < kItemWords; ++i) item_ring[(k & 1) * 32 + i] = u.w[i];
          mbar_arrive(FBAR(kBarItemFull + (k & 1)));
        }
        if (id < 0) break;
        // The next item is asked for with this one's last K tile, as above.
        auto request_next = [&]() {
          if (!clc_live) return;
          if (lane == 0) {
            mbar_arrive_expect_tx(FBAR(kBarClc), 16);
            clc_try_cancel(clc_resp, FBAR(kBarClc));
          }
          clc_pending = true;
        };
        if (it.n_tiles == 0) request_next();
        int entry = it.n_tiles > 0 ? pages.entry(p, it, kv_tile_at(it, 0)) : -1;
        for (int j = 0; j < it.n_tiles; ++j) {
          const int kt = kv_tile_at(it, j);
          const int s = T % KS;
          if (j == it.n_tiles - 1) request_next();
          const int row = pages.row(p, it, kt, entry, true);
          if (j + 1 < it.n_tiles) entry = pages.entry(p, it, kv_tile_at(it, j + 1));
          if (lane == 0 && T >= KS)
            ok = wait_bounded(BAR_KE(s), ((T / KS) - 1) & 1, abort_flag, p.status);
          if (!__shfl_sync(0xffffffffu, ok, 0)) break;
          const uint32_t n_loads = __popc(__ballot_sync(0xffffffffu, row >= 0));
          if (lane == 0) mbar_arrive_expect_tx(BAR_K(s), n_loads * pages.rows * D * 2);
          __syncwarp();
          if (row >= 0) {
#pragma unroll
            for (int sub = 0; sub < kChunks; ++sub)
              tma_load_3d(sK + s * L::kKVBytes + sub * kSubTile + lane * pages.rows * 128, &tm_k,
                          BAR_K(s), sub * 64, it.kv_plane, row);
          }
          ++T;
          if (j == 0) {
            if (lane == 0) {
              if (kq >= 1) ok = wait_bounded(FBAR(kBarQEmpty), (kq - 1) & 1, abort_flag, p.status);
              if (ok) {
                mbar_arrive_expect_tx(FBAR(kBarQFull), q_bytes);
#pragma unroll
                for (int sub = 0; sub < kChunks; ++sub)
                  tma_load_3d(sQ + sub * kSubTile, &tm_q, FBAR(kBarQFull), sub * 64,
                              it.kv_plane * p.group, it.tok0);
              }
            }
            if (!__shfl_sync(0xffffffffu, ok, 0)) break;
            ++kq;
          }
        }
        if (!__shfl_sync(0xffffffffu, ok, 0)) break;
        int next_id = -1;
        if (clc_pending) {
          if (lane == 0) {
            ok = wait_bounded(FBAR(kBarClc), clc_uses & 1, abort_flag, p.status);
            int x;
            if (ok && clc_query(clc_resp, x)) next_id = x;
          }
          if (!__shfl_sync(0xffffffffu, ok, 0)) break;
          clc_pending = false;
          ++clc_uses;
          next_id = __shfl_sync(0xffffffffu, next_id, 0);
          clc_live = next_id >= 0;
        }
        id = next_id;
      }
      // Every asynchronous write into this block's shared memory lands before it may exit.
      if (lane == 0) {
        for (int t = (T > KS ? T - KS : 0); t < T; ++t)
          wait_bounded(BAR_K(t % KS), (t / KS) & 1, nullptr, p.status, kDrainLimitNs);
        if (kq >= 1)
          wait_bounded(FBAR(kBarQFull), (kq - 1) & 1, nullptr, p.status, kDrainLimitNs);
        if (clc_pending)
          wait_bounded(FBAR(kBarClc), clc_uses & 1, nullptr, p.status, kDrainLimitNs);
      }
    } else if (lane == 0) {
      prefetch_tmap(&tm_q);
      prefetch_tmap(&tm_k);
      int id = static_cast<int>(blockIdx.x);
      int next_id = -1;
      bool clc_live = true;     // no answer "nothing left" seen yet
      bool clc_pending = false;  // a request is in flight
      uint32_t clc_uses = 0;
      auto take_answer = [&]() {
        clc_pending = false;
        ++clc_uses;
        int x;
        if (clc_query(clc_resp, x)) {
          next_id = x;
          const Item nx = decode_item(x, p);
          if (nx.n_tiles > 0) {
#pragma unroll
            for (int sub = 0; sub < kChunks; ++sub) tma_prefetch_l2_3d(&tm_q, sub * 64, nx.q0, nx.bh);
          }
        } else {
          next_id = -1;
          clc_live = false;
        }
      };
      int T = 0, kq = 0;  // K tiles and Q tiles loaded so far
      bool ok = true;
      for (int k = 0; ok; ++k) {
        if (k >= 2 &&
            !wait_bounded(FBAR(kBarItemEmpty + (k & 1)), ((k >> 1) - 1) & 1, abort_flag, p.status)) {
          ok = false;
          break;
        }
        ring[k & 1] = id;
        mbar_arrive(FBAR(kBarItemFull + (k & 1)));
        if (id < 0) break;
        // The following item is asked for with this item's last K load (a few tiles before the
        // softmax finishes this item): late enough that a block does not hold on to work other
        // blocks could start, early enough to pull the next Q tile into L2 in time.
        auto request_next = [&]() {
          if (clc_live) {
            mbar_arrive_expect_tx(FBAR(kBarClc), 16);
            clc_try_cancel(clc_resp, FBAR(kBarClc));
            clc_pending = true;
          }
        };
        next_id = -1;
        const Item it = decode_item(id, p);
        if (it.n_tiles == 0) request_next();
        for (int j = 0, kt = it.j_begin; j < it.n_tiles; ++j, ++kt) {
          if constexpr (SINKS)
            kt = kv_tile_at(it, j);
          else
            kt = next_kv_tile(it, kt);
          const int s = T % KS;
          if (T >= KS && !wait_bounded(BAR_KE(s), ((T / KS) - 1) & 1, abort_flag, p.status)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(BAR_K(s), L::kKVBytes);
#pragma unroll
          for (int sub = 0; sub < kChunks; ++sub)
            tma_load_3d(sK + s * L::kKVBytes + sub * kSubTile, &tm_k, BAR_K(s), sub * 64,
                        kt * kBlockN, it.kv_plane);
          ++T;
          if (j == 0) {
            if (kq >= 1 && !wait_bounded(FBAR(kBarQEmpty), (kq - 1) & 1, abort_flag, p.status)) {
              ok = false;
              break;
            }
            mbar_arrive_expect_tx(FBAR(kBarQFull), L::kQBytes);
#pragma unroll
            for (int sub = 0; sub < kChunks; ++sub)
              tma_load_3d(sQ + sub * kSubTile, &tm_q, FBAR(kBarQFull), sub * 64, it.q0, it.bh);
            ++kq;
          }
          if (j == it.n_tiles - 1) request_next();
        }
        if (!ok) break;
        if (clc_pending) {
          if (!wait_bounded(FBAR(kBarClc), clc_uses & 1, abort_flag, p.status)) {
            ok = false;
            break;
          }
          take_answer();
        }
        id = next_id;
      }
      // Every asynchronous write into this block's shared memory lands before it may exit.
      for (int t = (T > KS ? T - KS : 0); t < T; ++t)
        wait_bounded(BAR_K(t % KS), (t / KS) & 1, nullptr, p.status, kDrainLimitNs);
      if (kq >= 1)
        wait_bounded(FBAR(kBarQFull), (kq - 1) & 1, nullptr, p.status, kDrainLimitNs);
      if (clc_pending)
        wait_bounded(FBAR(kBarClc), clc_uses & 1, nullptr, p.status, kDrainLimitNs);
    }
    __syncwarp();
  } else if (warp == kVProducerWarp) {
    // ----------------------------------------------------------------- V producer
    if constexpr (PAGED) {
      if (lane == 0) prefetch_tmap(&tm_v);
      const PagedTile pages(p, lane);
      int T = 0;
      uint32_t ragged = 0;  // ragged tiles so far
      bool live = true;     // the last stage's loads signal its own barrier
      for (int k = 0; live; ++k) {
        if (!warp_wait(FBAR(kBarItemFull + (k & 1)), (k >> 1) & 1, abort_flag, p.status)) break;
        const FwdItemPaged it = read_item(k);
        __syncwarp();
        if (lane == 0) mbar_arrive(FBAR(kBarItemEmpty + (k & 1)));
        if (it.id < 0) break;
        int entry = it.n_tiles > 0 ? pages.entry(p, it, kv_tile_at(it, 0)) : -1;
        for (int j = 0; j < it.n_tiles; ++j) {
          const int kt = kv_tile_at(it, j);
          const int s = T % VS;
          const int row = pages.row(p, it, kt, entry, false);
          if (j + 1 < it.n_tiles) entry = pages.entry(p, it, kv_tile_at(it, j + 1));
          bool ok = true;
          if (lane == 0 && T >= VS)
            ok = wait_bounded(BAR_VE(s), ((T / VS) - 1) & 1, abort_flag, p.status);
          if (!__shfl_sync(0xffffffffu, ok, 0)) {
            live = false;
            break;
          }
          // The tile that holds the sequence's end: its rows past the end hold other sequences'
          // or unwritten tokens, or were not loaded at all.  P is zero there, but 0 * V has to
          // stay 0: the rows are cleared once the loads have landed, and only then is the tile
          // handed on.  The same for pages that could not be loaded.
          const uint32_t n_loads = __popc(__ballot_sync(0xffffffffu, row >= 0));
          const int valid = it.len - kt * kBlockN;  // rows of the tile that hold tokens
          const bool last = valid < kBlockN || static_cast<int>(n_loads * pages.rows) < kBlockN;
          const uint32_t bar = last ? FBAR(kBarRagged) : BAR_V(s);
          if (lane == 0) mbar_arrive_expect_tx(bar, n_loads * pages.rows * D * 2);
          __syncwarp();
          if (row >= 0) {
#pragma unroll
            for (int sub = 0; sub < kChunks; ++sub)
              tma_load_3d(sV + s * L::kKVBytes + sub * kSubTile + lane * pages.rows * 128, &tm_v,
                          bar, sub * 64, it.kv_plane, row);
          }
          if (last) {
            ok = warp_wait(bar, ragged & 1, abort_flag, p.status);
            ++ragged;
            if (!ok) {
              live = false;
              break;
            }
            const uint32_t loaded = __ballot_sync(0xffffffffu, row >= 0);
            for (int i = lane; i < kBlockN * kChunks * 8; i += 32) {
              const int rr = i / (kChunks * 8), c = i % (kChunks * 8);
              if (rr >= valid || !((loaded >> (rr >> pages.rows_log2)) & 1u))
                *reinterpret_cast<uint4*>(gbase + L::kV + s * L::kKVBytes + (c >> 3) * kSubTile +
                                          rr * 128 + (c & 7) * 16) = make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(BAR_V(s));
          }
          ++T;
        }
      }
      // loads that nothing waited for land before the block may exit (an aborted ragged tile's
      // wait has already taken its limit)
      if (lane == 0)
        for (int t = (T > VS ? T - VS : 0); t < T; ++t)
          wait_bounded(BAR_V(t % VS), (t / VS) & 1, nullptr, p.status, kDrainLimitNs);
    } else if (lane == 0) {
      prefetch_tmap(&tm_v);
      int T = 0;
      bool ok = true;
      for (int k = 0; ok; ++k) {
        int id;
        if (!take_item(k, id)) break;
        if (id < 0) break;
        const Item it = decode_item(id, p);
        for (int j = 0, kt = it.j_begin; j < it.n_tiles; ++j, ++kt) {
          if constexpr (SINKS)
            kt = kv_tile_at(it, j);
          else
            kt = next_kv_tile(it, kt);
          const int s = T % VS;
          if (T >= VS && !wait_bounded(BAR_VE(s), ((T / VS) - 1) & 1, abort_flag, p.status)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(BAR_V(s), L::kKVBytes);
          if constexpr (FP8) {
            // V^T tile: d rows of 128 keys (the K-major B operand of the 8-bit P V product)
            tma_load_3d(sV + s * L::kKVBytes, &tm_v, BAR_V(s), kt * kBlockN, 0, it.kv_plane);
          } else {
#pragma unroll
            for (int sub = 0; sub < D / 64; ++sub)
              tma_load_3d(sV + s * L::kKVBytes + sub * kSubTile, &tm_v, BAR_V(s), sub * 64,
                          kt * kBlockN, it.kv_plane);
          }
          ++T;
        }
      }
      for (int t = (T > VS ? T - VS : 0); t < T; ++t)
        wait_bounded(BAR_V(t % VS), (t / VS) & 1, nullptr, p.status, kDrainLimitNs);
    }
    __syncwarp();
  } else if (warp == kQkWarp || warp == kPvWarp) {
    // ----------------------------------------------------------------- tcgen05 issuers
    // Warp 9 issues the score MMAs, warp 10 the P V MMAs.  The two streams touch disjoint tensor
    // memory (S buffers / O and P buffers) and disjoint shared memory (Q, K / V), so they need no
    // ordering between them beyond the barriers below, and each issuer's waits overlap the other
    // issuer's MMAs.
    if (lane == 0) {
      const bool qk_issuer = (warp == kQkWarp);
      // (FP8: kind::f8f6f4 with format code 0 = E4M3 for A and B; V^T is K-major)
      constexpr uint32_t idesc_qk = make_idesc_f16(BF16 && !FP8, kBlockM, kBlockN, false);
      constexpr uint32_t idesc_pv = make_idesc_f16(BF16 && !FP8, kBlockM, D, !FP8);
      // S_t = Q K_t^T into S buffer t % 2, once the softmax of tile t - 2 has read that buffer.
      auto issue_qk = [&](int t) -> bool {
        FWD_TRACE(t, 8);
        const int s = t % KS;
        if (t >= 2 &&
            !wait_bounded(FBAR(kBarSFree + (t & 1)), ((t >> 1) - 1) & 1, abort_flag, p.status))
          return false;
        FWD_TRACE(t, 15);
        if (!wait_bounded(BAR_K(s), (t / KS) & 1, abort_flag, p.status)) return false;
        FWD_TRACE(t, 9);
        tc_fence_after();
        const uint32_t s_col = tmem + ((t & 1) ? kColS1 : kColS0);
        if constexpr (FP8) {
          // 8-bit Q and K, K-major: 32 elements = 32 bytes per MMA in the one 128-byte row
#pragma unroll
          for (int kk = 0; kk < D / 32; ++kk) {
            const uint64_t adesc = make_sdesc_sw128(sQ + kk * 32, 16, 1024);
            const uint64_t bdesc = make_sdesc_sw128(sK + s * L::kKVBytes + kk * 32, 16, 1024);
            mma_ss_f8(s_col, adesc, bdesc, idesc_qk, kk > 0 ? 1u : 0u);
          }
        } else {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            // Q and K are K-major (d contiguous): 16 elements = 32 bytes per MMA inside the
            // 128-byte swizzle row; SBO = 1024 B between 8-row groups.
            const uint32_t off = (kk >> 2) * kSubTile + (kk & 3) * 32;
            const uint64_t adesc = make_sdesc_sw128(sQ + off, 16, 1024);
            const uint64_t bdesc = make_sdesc_sw128(sK + s * L::kKVBytes + off, 16, 1024);
            mma_ss(s_col, adesc, bdesc, idesc_qk, kk > 0 ? 1u : 0u);
          }
        }
        mma_commit(FBAR(kBarS + (t & 1)));
        mma_commit(BAR_KE(s));  // K slot free
        FWD_TRACE(t, 10);
        return true;
      };
      // O (+)= P_t V_t (P_t in P buffer t % 2, V_t in ring slot t % VS); the first tile of
      // an item overwrites the accumulator.
      auto issue_pv = [&](int t, bool first) -> bool {
        FWD_TRACE(t, 11);
        if (!wait_bounded(FBAR(kBarP + (t & 1)), (t >> 1) & 1, abort_flag, p.status)) return false;
        FWD_TRACE(t, 12);
        const int s = t % VS;
        if (!wait_bounded(BAR_V(s), (t / VS) & 1, abort_flag, p.status)) return false;
        FWD_TRACE(t, 13);
        tc_fence_after();
        const uint32_t p_col = tmem + ((t & 1) ? PCols<D>::kP1 : PCols<D>::kP0);
        if constexpr (FP8) {
          // P: E4M3 codes, four per tensor-memory column; V^T rows (d) of 128 keys, K-major:
          // 32 keys = 32 bytes per MMA in the 128-byte row
#pragma unroll
          for (int kk = 0; kk < kBlockN / 32; ++kk) {
            const uint64_t bdesc = make_sdesc_sw128(sV + s * L::kKVBytes + kk * 32, 16, 1024);
            mma_ts_f8(tmem + kColO, p_col + kk * 8, bdesc, idesc_pv, (!first || kk > 0) ? 1u : 0u);
          }
        } else {
#pragma unroll
          for (int kk = 0; kk < kBlockN / 16; ++kk) {
            // V is [keys, d] with d contiguous: the B operand is MN-major.  16 keys per MMA
            // (two 8-row groups, SBO = 1024 B apart); the two 64-column halves of d are
            // separate swizzled sub-tiles (LBO = one sub-tile).
            const uint64_t bdesc = make_sdesc_sw128(sV + s * L::kKVBytes + kk * 16 * 128,
                                                    kSubTile, 1024);
            mma_ts(tmem + kColO, p_col + kk * 8, bdesc, idesc_pv, (!first || kk > 0) ? 1u : 0u);
          }
        }
        mma_commit(FBAR(kBarO + (t & 1)));
        mma_commit(BAR_VE(s));  // V slot free
        FWD_TRACE(t, 14);
        return true;
      };
      // The score issuer runs up to two tiles ahead of the softmax (two S buffers), also into
      // the next item; the P V issuer follows the softmax tile by tile.  The P V issuer also
      // sends each item's O tile to global memory: the epilogue of item e fills the staging
      // buffer during the first tile of item e + 1, and the TMA store goes out from here while
      // item e + 1's MMAs run (at the latest after its last P V), so that no softmax warp ever
      // waits for a store.
      int T = 0, kq = 0;  // tiles and non-empty items issued so far
      int st_q0 = 0, st_bh = 0;  // the previous non-empty item, whose O is to be stored
      bool stored = true;        // ... and its store has been issued
      auto store_o = [&]() {
#pragma unroll
        for (int sub = 0; sub < D / 64; ++sub)
          tma_store_3d(&tm_o, sOst + sub * kSubTile, sub * 64, st_q0, st_bh);
        tma_store_commit();
        stored = true;
      };
      bool ok = true;
      for (int k = 0; ok; ++k) {
        Item it;
        if constexpr (PAGED) {
          if (!take_paged(k, it)) break;
        } else {
          int id;
          if (!take_item(k, id)) break;
          if (id < 0) break;
          it = decode_item(id, p);
        }
        if (it.n_tiles == 0) continue;
        if (qk_issuer) {
          if (!wait_bounded(FBAR(kBarQFull), kq & 1, abort_flag, p.status)) break;
          for (int j = 0; ok && j < it.n_tiles; ++j) ok = issue_qk(T + j);
          if (ok) mma_commit(FBAR(kBarQEmpty));  // Q free once these MMAs finished
        } else {
          for (int j = 0; ok && j < it.n_tiles; ++j) {
            ok = issue_pv(T + j, j == 0);
            if (!PAGED && !stored && mbar_test_wait(FBAR(kBarOStageFull), (kq - 1) & 1)) store_o();
          }
          if (!ok) break;
          if (!PAGED && kq >= 1) {
            // The staging buffer is free again once the store has read it.
            if (!stored) {
              if (!wait_bounded(FBAR(kBarOStageFull), (kq - 1) & 1, abort_flag, p.status)) break;
              store_o();
            }
            tma_store_wait_read0();
            mbar_arrive(FBAR(kBarOStage));
          }
          st_q0 = it.q0;
          st_bh = it.bh;
          stored = false;
        }
        T += it.n_tiles;
        ++kq;
      }
      if (!PAGED && !qk_issuer && ok && kq >= 1 && !stored &&
          wait_bounded(FBAR(kBarOStageFull), (kq - 1) & 1, abort_flag, p.status))
        store_o();
      if (!qk_issuer) tma_store_wait_all();  // every O tile written before the block exits
      // Every MMA this thread issued completes before the block frees tensor memory.
      if (T > 0)
        mma_commit(FBAR(kBarDrain));
      else
        mbar_arrive(FBAR(kBarDrain));
      wait_bounded(FBAR(kBarDrain), 0, nullptr, p.status, kDrainLimitNs);
    }
    __syncwarp();
  }
    tc_fence_before();
    __syncthreads();  // every tensor-memory access and MMA of the block has finished
    if (warp == kQkWarp) {
      tc_fence_after();
      tmem_dealloc(tmem, kTmemCols);
    }
  } else {
    setmaxnreg_inc<kRegsSoftmax>();
    // ----------------------------------------------------------------- softmax + epilogue
    // Two warpgroups share the rows: warpgroup w takes the tiles t of the block's tile sequence
    // with t % 2 == w (S buffer w, P buffer w); in both, thread r owns query row r and warp % 4
    // is its tensor-memory lane quarter.  The running maximum is the only state carried from
    // tile to tile: the warpgroup of tile t publishes m_t as soon as its row maxima are known
    // (kBarM, one barrier per warp: warp q of one warpgroup and warp q of the other own the same
    // 32 rows), and the other warpgroup, on tile t + 1, waits for it before its exponentials.
    // Each warpgroup keeps its own partial row sum, rescaled whenever the maximum moves.
    //
    // Epilogue of an item whose last tile is t_e: the warpgroup of t_e hands its partial sum
    // (relative to the final maximum m_{t_e}) over through shared memory and goes on; the other
    // warpgroup finishes the item during its next tile t_e + 1 (the first tile of the next
    // item): it reads m_{t_e} with the running maximum, reads the accumulator out of tensor
    // memory between storing P_{t_e+1} and releasing it (so before P V_{t_e+1} overwrites the
    // accumulator), then writes O = a / l to the staging buffer for the TMA store and the
    // log-sum-exp to global memory.
    const int wg = warp >> 2;
    const int quarter = warp & 3;
    const int r = quarter * 32 + lane;
    const uint32_t row_tmem = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    [[maybe_unused]] const bool tracer = (threadIdx.x & 127) == 0;  // timestamp hooks only
    const int off = p.N_kv - p.N_q;
    const float sl2 = p.sl2;
    // read once: the masked tiles' bounds (those tiles come once or twice an item, and their
    // parameter reads would otherwise be fetched cold)
    const int n_kv = p.N_kv, causal = p.causal, window = p.window;
    float* mrow = reinterpret_cast<float*>(gbase + L::kMrow);    // [row]
    float* lpart = reinterpret_cast<float*>(gbase + L::kLpart);  // [item parity][row]
    const uint32_t s_col = wg ? kColS1 : kColS0;
    const uint32_t p_col = wg ? PCols<D>::kP1 : PCols<D>::kP0;
    float m_own = -INFINITY;  // maximum (log2 units) this warpgroup's partial sum refers to
    float l = 0.0f;           // this warpgroup's partial sum of 2^(x - m_own)
    int T = 0;                // tiles of the block's sequence before the current item
    int kq = 0;               // items with at least one tile before the current one
    bool ok = true;
    bool s_ready = false;  // S of this warpgroup's next tile already seen complete
    // Epilogue this warpgroup owes: item index, first row, (batch, head), partial sum and
    // its maximum, and the item's last tile.
    // The owed epilogue's item data wait in shared memory (one copy per warp, written by its
    // lane 0 and read by the same warp), so that they take no registers across the
    // exponential loop.
    volatile int* ep_state = PAGED
                                 ? reinterpret_cast<volatile int*>(gbase + L::kEpPaged) + 8 * warp
                                 : reinterpret_cast<volatile int*>(gbase + L::kEpState) + 4 * warp;
    // paged: the token of the tile this row belongs to (a row past the tile's tokens follows the
    // last keys of the sequence and is not stored)
    int my_tok = 0;
    if constexpr (PAGED) my_tok = r / p.group;
    bool ep_pending = false;
    float ep_l = 0.0f, ep_m = -INFINITY;

    for (int k = 0; ok; ++k) {
      if (tracer) FWD_TRACE(T, 16 + wg * 4);
      if (!warp_wait(FBAR(kBarItemFull + (k & 1)), (k >> 1) & 1, abort_flag, p.status)) break;
      if (tracer) FWD_TRACE(T, 17 + wg * 4);
      Item it;
      if constexpr (PAGED) {
        it = read_item(k);
        __syncwarp();
        if (lane == 0) mbar_arrive(FBAR(kBarItemEmpty + (k & 1)));
        if (it.id < 0) break;
      } else {
        const int id = ring[k & 1];
        __syncwarp();
        if (lane == 0) mbar_arrive(FBAR(kBarItemEmpty + (k & 1)));
        if (id < 0) break;
        it = decode_item(id, p);
      }
      if (tracer) FWD_TRACE(T, 18 + wg * 4);
      const int n = it.n_tiles;
      const int row = it.q0 + r;
      if constexpr (PAGED) {
        // a split with no tile of its own: the merge gives it no weight
        if (n == 0) {
          if (wg == 0 && r < it.n_rows) {
            const size_t grow = static_cast<size_t>(it.tok0 + my_tok) * p.Hq +
                                it.kv_plane * p.group + (r - my_tok * p.group);
            reinterpret_cast<float2*>(p.ws_ml)[grow * p.n_splits + it.split] =
                make_float2(-INFINITY, 0.0f);
          }
          continue;
        }
      }
      if (n == 0) {
        // No key visible to any row of this tile: O = 0, L = -inf.
        if (wg == 0 && row < p.N_q) {
          const size_t row_index = static_cast<size_t>(it.bh) * p.N_q + row;
          uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.o) + row_index * D);
#pragma unroll
          for (int c = 0; c < D / 8; ++c) dst[c] = make_uint4(0, 0, 0, 0);
          p.lse[row_index] = -INFINITY;
        }
        continue;
      }
      const int T0 = T;
      const int T_last = T0 + n - 1;
      // FP8: the item's Q block scale (its K block scales are read per tile, before the wait
      // for the tile's scores, so that the loads are in flight during the wait)
      float q_sc = 1.0f;
      if constexpr (FP8) q_sc = p.q_scale[static_cast<size_t>(it.bh) * p.n_qtiles + it.q0 / kBlockM];
      for (int i = 0, j = it.j_begin; i < n; ++i, ++j) {
        if constexpr (SINKS)
          j = kv_tile_at(it, i);
        else
          j = next_kv_tile(it, j);  // key tile of the item's i-th tile
        const int t = T0 + i;
        if ((t & 1) != wg) continue;
        const int u = t >> 1;  // use index of this warpgroup's S and P buffers
        float k_sc = 1.0f;
        if constexpr (FP8) k_sc = p.k_scale[static_cast<size_t>(it.kv_plane) * p.n_kvtiles + j];
        if (tracer) FWD_TRACE(t, 0);
        if (!__all_sync(0xffffffffu, s_ready) &&
            !warp_wait(FBAR(kBarS + wg), u & 1, abort_flag, p.status)) {
          ok = false;
          break;
        }
        if (tracer) FWD_TRACE(t, 1);
        tc_fence_after();
        uint32_t sr[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(row_tmem + s_col + c * 32, sr[c]);
        tmem_wait_ld();
        tc_fence_before();
        mbar_arrive(FBAR(kBarSFree + wg));  // S buffer free for Q K_{t+2}^T
        if (tracer) FWD_TRACE(t, 2);
        // Early, non-blocking test of the barrier needed before P is written (P V_{t-2} read
        // this P buffer); its latency hides under the work below.
        const bool p_free = (t < 2) || mbar_test_wait(FBAR(kBarO + wg), (u - 1) & 1);
        float x[kBlockN];
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int e = 0; e < 32; ++e) x[c * 32 + e] = __uint_as_float(sr[c][e]);
        if (j >= it.first_masked || j < it.lo_masked) {
          // Visible columns [lo, hi] of this row in this tile: hi from the causal bound or the
          // ragged end, lo from the sliding window.  One code path for every masked tile, as
          // four 32-column bit masks and one test per column: masked tiles come once or twice
          // an item, so their code is fetched cold, and a short path costs less.
          int hi = kBlockN - 1, lo = 0;
          if constexpr (SINKS) {
            // ... and the sinks among the tile's columns
            int pos, last_key;
            if constexpr (PAGED) {
              pos = it.pos0 + my_tok;
              last_key = it.len - 1;
            } else {
              pos = row + off;
              last_key = n_kv - 1;
            }
            if (j >= it.first_masked) hi = min(min(pos, last_key) - j * kBlockN, kBlockN - 1);
            if (j < it.lo_masked) lo = max(pos - window - j * kBlockN, 0);
            const int sk = min(p.sinks - 1 - j * kBlockN, hi);  // last sink column
            uint32_t vis[kBlockN / 32];
#pragma unroll
            for (int g = 0; g < kBlockN / 32; ++g) {
              const int a = max(lo - 32 * g, 0), bb = min(hi - 32 * g, 31);
              const int ss = min(sk - 32 * g, 31);
              vis[g] = (a > bb) ? 0u : ((0xffffffffu >> (31 - bb)) & (0xffffffffu << a));
              vis[g] |= (ss < 0) ? 0u : (0xffffffffu >> (31 - ss));
            }
            // the score where visible, -inf where not: by bits, so that a NaN or infinite score
            // of a masked key (a row past the sequence's end) leaves no trace
#pragma unroll
            for (int c = 0; c < kBlockN; ++c) {
              const uint32_t keep =
                  static_cast<uint32_t>(static_cast<int32_t>(vis[c >> 5] << (31 - (c & 31))) >> 31);
              x[c] = __uint_as_float((__float_as_uint(x[c]) & keep) | (0xff800000u & ~keep));
            }
          } else {
            if (j >= it.first_masked) {
              int lim = causal ? row + off : n_kv - 1;  // last visible key of this row
              if (lim > n_kv - 1) lim = n_kv - 1;
              hi = min(lim - j * kBlockN, kBlockN - 1);
            }
            if (j < it.lo_masked) lo = max(row + off - window - j * kBlockN, 0);
            uint32_t vis[kBlockN / 32];
#pragma unroll
            for (int g = 0; g < kBlockN / 32; ++g) {
              const int a = max(lo - 32 * g, 0), bb = min(hi - 32 * g, 31);
              vis[g] = (a > bb) ? 0u : ((0xffffffffu >> (31 - bb)) & (0xffffffffu << a));
            }
            // x + 0 where visible, x + (-inf) where not: integer arithmetic, no per-column
            // condition (each of which could otherwise become a divergent branch)
#pragma unroll
            for (int c = 0; c < kBlockN; ++c)
              x[c] += __uint_as_float((((vis[c >> 5] >> (c & 31)) & 1u) - 1u) & 0xff800000u);
          }
        }
        // Row maximum of the tile: three-input max, sixteen independent chains.
        float mx[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) mx[e] = fmaxf(x[e], x[16 + e]);
#pragma unroll
        for (int c = 32; c < kBlockN; c += 32)
#pragma unroll
          for (int e = 0; e < 16; ++e) mx[e] = max3f(mx[e], x[c + e], x[c + 16 + e]);
#pragma unroll
        for (int e = 0; e < 8; ++e) mx[e] = fmaxf(mx[e], mx[e + 8]);
        const float tile_max = max3f(max3f(mx[0], mx[1], mx[2]), max3f(mx[3], mx[4], mx[5]),
                                     fmaxf(mx[6], mx[7]));
        // Running maximum after tile t - 1, from the other warpgroup (on the first tile of an
        // item: the previous item's final maximum, which an owed epilogue needs).  The wait also
        // orders this tile's write of mrow after the other warpgroup's read of it.
        float m_read = -INFINITY;
        if (tracer) FWD_TRACE(t, 24);
        if (t > 0) {
          if (!warp_wait(FBAR(kBarM + (wg ^ 1) * 4 + quarter), ((t - 1) >> 1) & 1, abort_flag,
                         p.status)) {
            ok = false;
            break;
          }
          m_read = mrow[r];
        }
        const float m_prev = (i > 0) ? m_read : -INFINITY;
        // Score scale of this tile: scale * log2(e), times the E4M3 block scales for FP8.
        float tsc = sl2;
        if constexpr (FP8) tsc = sl2 * q_sc * k_sc;
        // The maximum moves only when it rises by more than 2^8 (also for the first finite one);
        // FP8: by more than 2^3.8.
        float m_j = m_prev;
        float alpha = 1.0f;  // rescale of the accumulator O for this tile
        const float m_new = fmaxf(m_prev, tile_max * tsc);
        if (m_new - m_prev > (FP8 ? kRescaleThreshold8 : kRescaleThreshold)) {
          alpha = ex2(m_prev - m_new);
          m_j = m_new;
        }
        mrow[r] = m_j;
        mbar_arrive(FBAR(kBarM + wg * 4 + quarter));  // m_t published for tile t + 1
        if (tracer) FWD_TRACE(t, 25);
        if (m_j != m_own) {
          l = (m_own == -INFINITY) ? 0.0f : l * ex2(m_own - m_j);
          m_own = m_j;
        }
        const float neg_mu = ((m_j == -INFINITY) ? 0.0f : -m_j) + (FP8 ? kPShift8 : 0);
        // p = 2^(x * scale * log2(e) - m): one packed FMA per pair of scores and MUFU ex2, all
        // of them first (in place, so that consecutive ex2 depend on nothing but their own FMA),
        // then a packed add into four pair-accumulators for the row sum and the 16-bit pack for
        // P (FP8: 2^5 p, four E4M3 codes per word).
#pragma unroll
        for (int c = 0; c < kBlockN; c += 2) {
          float a0, a1;
          fma2(a0, a1, x[c], x[c + 1], tsc, tsc, neg_mu, neg_mu);
          x[c] = ex2(a0);
          x[c + 1] = ex2(a1);
        }
        float ps[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        uint32_t pk[2][32];
#pragma unroll
        for (int c = 0; c < kBlockN; c += 4) {
          const float p0 = x[c], p1 = x[c + 1], p2 = x[c + 2], p3 = x[c + 3];
          const int k2 = ((c >> 1) & 3) * 2;
          add2(ps[k2], ps[k2 + 1], p0, p1);
          add2(ps[k2 + 2], ps[k2 + 3], p2, p3);
          if constexpr (FP8) {
            pk[0][c >> 2] = pack4_e4m3(p0, p1, p2, p3);
          } else {
            pk[c >> 6][(c >> 1) & 31] = pack2<BF16>(p0, p1);
            pk[c >> 6][((c >> 1) & 31) + 1] = pack2<BF16>(p2, p3);
          }
        }
        l += ((ps[0] + ps[1]) + (ps[2] + ps[3])) + ((ps[4] + ps[5]) + (ps[6] + ps[7]));
        // Tile t + 2 is this warpgroup's next one, in this item or the next.
        s_ready = mbar_test_wait(FBAR(kBarS + wg), (u + 1) & 1);
        if (tracer) FWD_TRACE(t, 3);
        if (t >= 2) {
          if (!__all_sync(0xffffffffu, p_free) &&
              !warp_wait(FBAR(kBarO + wg), (u - 1) & 1, abort_flag, p.status)) {
            ok = false;
            break;
          }
          tc_fence_after();  // order the P store after the MMA that read the buffer
        }
        if (tracer) FWD_TRACE(t, 4);
        tmem_st32(row_tmem + p_col, pk[0]);
        if constexpr (!FP8) tmem_st32(row_tmem + p_col + 32, pk[1]);
        // Both cases below need P V_{t-1} finished: P V_t waits for this tile's P and P V_{t+1}
        // comes after it, so nothing else touches the accumulator meanwhile.
        const bool rescale = i > 0 && __any_sync(0xffffffffu, alpha != 1.0f);
        if (rescale || ep_pending) {
          if (!warp_wait(FBAR(kBarO + (wg ^ 1)), ((t - 1) >> 1) & 1, abort_flag, p.status)) {
            ok = false;
            break;
          }
          tc_fence_after();
        }
        if (rescale) {
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            uint32_t o[32];
            tmem_ld32(row_tmem + kColO + c * 32, o);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
            tmem_st32(row_tmem + kColO + c * 32, o);
          }
        }
        if (ep_pending) {
          // The first tile after the owed item's last one: its accumulator is read out before
          // this tile's P is released to P V_t, which overwrites it.
          if (tracer) FWD_TRACE(ep_state[3], 6);
          bool done;
          if constexpr (PAGED)
            done = paged_epilogue<D, BF16>(row_tmem + kColO, m_read, ep_l, ep_m, ep_state, r, fbars,
                                           lpart, p, abort_flag);
          else
            done = run_epilogue<D, BF16, FP8, SINKS>(row_tmem + kColO, m_read, ep_l, ep_m, ep_state[0],
                                              ep_state[1], ep_state[2], r, fbars, lpart,
                                              gbase + L::kOst, p, abort_flag);
          if (!done) {
            ok = false;
            break;
          }
          ep_pending = false;
          if (tracer) FWD_TRACE(ep_state[3], 7);
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(FBAR(kBarP + wg));
        if (tracer) FWD_TRACE(t, 5);
      }
      if (!ok) break;
      if (tracer) FWD_TRACE(T, 19 + wg * 4);
      // ------------------------------------------------------------- end of the item
      if ((T_last & 1) == wg) {
        // This warpgroup ran the last tile: its partial sum refers to the final maximum.  The
        // other warpgroup finishes the item.
        // Handover slot kq % 2, free once item kq - 2's epilogue has read it.
        const int slot = kq & 1;
        if (kq >= 2 &&
            !warp_wait(FBAR(kBarLEmpty + slot), ((kq >> 1) - 1) & 1, abort_flag, p.status))
          break;
        lpart[slot * kBlockM + r] = l;
        mbar_arrive(FBAR(kBarLFull + slot));
      } else {
        ep_pending = true;
        if (lane == 0) {
          ep_state[0] = kq;
          if constexpr (PAGED) {
            ep_state[1] = it.tok0;
            ep_state[2] = it.kv_plane;
            ep_state[4] = it.n_rows;
            ep_state[5] = it.split;
          } else {
            ep_state[1] = it.q0;
            ep_state[2] = it.bh;
          }
          ep_state[3] = T_last;
        }
        __syncwarp();
        ep_l = l;
        ep_m = m_own;
      }
      l = 0.0f;
      m_own = -INFINITY;
      T += n;
      ++kq;
    }
    if (ok && ep_pending) {
      // No tile follows the block's last item: finish it here.  A parity wait is only sound
      // while its barrier is at most one phase behind or ahead of the awaited one: tile t_e - 1
      // was this warpgroup's (its P-buffer wait saw P V_{t_e-3} finish), so P V_{t_e-1} is
      // awaited first on this warpgroup's barrier, which makes P V_{t_e-2} finished too and
      // P V_{t_e} the next phase of the other barrier.
      const int t_e = ep_state[3];
      bool done = true;
      if (t_e >= 1)
        done = warp_wait(FBAR(kBarO + ((t_e - 1) & 1)), ((t_e - 1) >> 1) & 1, abort_flag, p.status);
      done = done && warp_wait(FBAR(kBarO + (t_e & 1)), (t_e >> 1) & 1, abort_flag, p.status);
      if (done && warp_wait(FBAR(kBarM + (t_e & 1) * 4 + quarter), (t_e >> 1) & 1, abort_flag,
                            p.status)) {
        tc_fence_after();
        if constexpr (PAGED)
          paged_epilogue<D, BF16>(row_tmem + kColO, mrow[r], ep_l, ep_m, ep_state, r, fbars, lpart,
                                  p, abort_flag);
        else
          run_epilogue<D, BF16, FP8, SINKS>(row_tmem + kColO, mrow[r], ep_l, ep_m, ep_state[0],
                                     ep_state[1], ep_state[2], r, fbars, lpart, gbase + L::kOst,
                                     p, abort_flag);
      }
    }
    tc_fence_before();
    __syncthreads();  // the other warpgroup's matching barrier ends its branch
    if (threadIdx.x == 0) FWD_TRACE(79, 1);
  }
#undef BAR_K
#undef BAR_V
#undef BAR_KE
#undef BAR_VE
#undef FBAR
}

}  // namespace attn
