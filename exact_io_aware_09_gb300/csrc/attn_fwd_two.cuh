// Prefill with two blocks on an SM: the sliding window with sinks (attn_fwd_window.cu) and chunks over a
// paged cache (attn_fwd_paged.cu).
//
// The prefill kernel (attn_fwd.cu) runs one long-lived block on an SM and spends about 6 us per work
// item between the last tile of one and a full pipeline on the next, as much as nine 128-key tiles.
// This kernel takes one work item per block and runs two blocks on an SM, so that one block's start
// and end, and its waits, lie under the other's key loop.  What a block may hold is halved: 256
// tensor-memory columns, about 100 KB of shared memory (113 at most), 128 registers a thread.
//
// Keys go in steps of 64: S = Q K_t^T is 128 x 64 in a tensor-memory buffer that is free as soon as the
// softmax (one warpgroup, thread = query row) has read it; P_t goes as 16-bit pairs into one of two
// buffers of its own, and O += P_t V_t follows.  So S_{t+1} is made under the softmax of S_t, and
// nothing waits for P_t V_t but the step after the next (with P_t over the scores, as before, S_{t+2}
// had to: 278 us against 266 at the first shape below).  The finer steps also cut what the window's
// edges and a few sinks leave of a tile.  The running maximum is the thread's own; the accumulator is
// rescaled when it rises by more than 2^8, the division by the row sum at the end undoing the difference.
//
// P is rounded to V's 16-bit type for its product (the tensor cores multiply operands of one type), which
// moves each weight by at most half a step; the row sums take the unrounded weights, and scores, statistics
// and O are fp32 until O is stored.
//
// Roles: warps 0-3 softmax and epilogue; warp 4 TMA producer (paged: of Q and K, page by page, a page's
// copy issued by its own lane, the block-table entries read a step ahead); warp 5 tcgen05 issuer of S
// (it owns the tensor memory), warp 6 of P V (one thread for both: 268 us against 260); paged: warp 7
// producer of V.  Every wait on a barrier is bounded.
//
// Bound by the tensor pipe's 64-wide products and a step's chain at two blocks an SM.  B=1 Hq=64 Hkv=8
// N=8192 d=128 bf16, W=1024, 4 sinks: 250 us (1,030 TFLOP/s of visible products; tensor pipe 52% busy,
// 1.8 instructions a cycle), the prefill kernel 334; B=8 H=12 N=1024 d=64, W=256: 25 us.  Tried and
// slower: a persistent grid of two blocks an SM (321 us when this kernel took 282), the same with
// 128-key tiles (319); three blocks an SM at d=64 (27 us against 25).
#pragma once
#include "internal.h"
#include "ptx.cuh"

namespace attn {

constexpr int kWM = 128;        // query rows
constexpr int kWN = 64;         // keys of a step
constexpr uint32_t kWSubQ = kWM * 128;   // one 64-column sub-tile of Q
constexpr uint32_t kWSubKV = kWN * 128;  // ... of a K or V step
constexpr uint32_t kWTmemCols = 256;
constexpr uint32_t kWColP = 0, kWColS = 64;  // P buffers at 0 and 32; S buffers, then O
constexpr float kWRescale = 8.0f;  // log2 units
constexpr uint64_t kWDrainNs = 100000000ull;

struct WinParams {
  void* o;
  float* lse;
  int* status;
  int Hq, Hkv, G, N_q, N_kv, n_qtiles, BH, head_group, window, sinks;
  float sl2;
};

template <int D>
struct WinLayout {
  static constexpr int kKS = D == 128 ? 2 : 3, kVS = D == 128 ? 2 : 3;  // ring slots
  static constexpr int kNS = D == 128 ? 1 : 2;                          // S buffers
  static constexpr uint32_t kColO = kWColS + kNS * kWN;
  static_assert(kColO + D <= kWTmemCols, "tensor memory");
  static constexpr uint32_t kQBytes = kWM * D * 2;
  static constexpr uint32_t kStep = kWN * D * 2;
  static constexpr uint32_t kK = kQBytes;
  static constexpr uint32_t kV = kK + kKS * kStep;
  static constexpr uint32_t kBar = kV + kVS * kStep;
  // q_full, k_full, k_empty, v_full, v_empty, s_full[2], p_ready[2], pv_done[2], drain, s_free[2],
  // drain of the S issuer, a ragged V step's loads (paged)
  static constexpr uint32_t kNumBars = 1 + 2 * kKS + 2 * kVS + 11;
  static constexpr uint32_t kMisc = kBar + kNumBars * 8;
  static constexpr uint32_t kBytes = kMisc + 16 + 1024;  // + alignment
  static_assert(2 * (kBytes + 1024) <= 233472, "two blocks on an SM");
};

// One work item: a 128-row query tile of one (batch, query head).
struct WinItem {
  int qt, bh, kv_plane;
  int rows;                           // of the tile that exist
  int j_begin, lo_masked, hi_masked;  // first step of the window; steps below / from which on masked
  int sink_steps, n;                  // steps that hold sinks and lie before the window; all steps
  static constexpr bool full = true;  // (its store clips the rows past the end)
  __device__ __forceinline__ int key_step(int t) const {
    return t < sink_steps ? t : j_begin + t - sink_steps;
  }
};

// (batch, query head) pairs in groups whose K/V planes fill about half of L2, a group's items longest
// query tile first across its heads.
__device__ __forceinline__ WinItem two_item(int id, const WinParams& p) {
  WinItem it;
  const int span = p.head_group * p.n_qtiles;
  const int grp = id / span;
  const int rem = id - grp * span;
  const int h0 = grp * p.head_group;
  const int gh = min(p.head_group, p.BH - h0);
  it.qt = p.n_qtiles - 1 - rem / gh;
  it.bh = h0 + rem % gh;
  it.rows = min(p.N_q - it.qt * kWM, kWM);
  it.kv_plane = (it.bh / p.Hq) * p.Hkv + (it.bh % p.Hq) / p.G;
  int j_end;
  kv_tile_span(it.qt, kWM, kWN, p.N_q, p.N_kv, 1, p.window, it.j_begin, j_end, it.lo_masked,
               it.hi_masked);
  it.sink_steps = min((p.sinks + kWN - 1) / kWN, it.j_begin);
  it.n = it.sink_steps + j_end - it.j_begin;
  return it;
}


// A chunk of new tokens over a paged cache: n_qtiles, BH and head_group count query tiles of the longest
// chunk and (sequence, key/value head) planes.
struct PagedParams {
  void* o;
  float* lse;
  int* status;
  int Hq, Hkv, G, n_qtiles, BH, head_group, window, sinks;
  float sl2;
  const int32_t* block_table;  // [B, max_pages]
  const int32_t* cu_q;         // [B + 1] packed rows of each sequence's new tokens
  const int32_t* seqlens;      // [B] cached tokens, the new ones included
  int page_log2, max_pages, num_pages;
  int total_q, max_q, max_k;
  int tile_tokens;             // tokens of one query tile: 128 / G
  int n_splits, split_steps;   // 64-key steps of one split (n_splits == 1: the whole item)
  float* ws_o;                 // [total_q * Hq, n_splits, D] normalised partial outputs
  float* ws_ml;                // [total_q * Hq, n_splits, 2] (m in log2 units, l)
};

// One work item: a query tile of one (sequence, key/value head), or one split of its keys.  The tile's
// rows are (token, query head of the group) pairs, token major.
struct PagedItem {
  int b, kv_plane;  // sequence, key/value head
  int rows;         // that belong to the chunk
  bool full;        // ... and are all the tile's rows a store would write
  int tok0;         // packed row of the tile's first token
  int pos0, len;    // its cache position; cached tokens of the sequence
  int split;
  int j_begin, lo_masked, hi_masked;
  int sink_steps, i0, n;  // steps with sinks before the window; this split's first step; its steps
  __device__ __forceinline__ int key_step(int t) const {
    const int i = i0 + t;
    return i < sink_steps ? i : j_begin + i - sink_steps;
  }
};

// Planes grouped and walked longest query tile first as above, a tile's splits side by side.  The grid
// covers the longest chunk the caller announced; items past a sequence's own chunk have no rows.
__device__ __forceinline__ PagedItem two_item(int id, const PagedParams& p) {
  PagedItem it;
  it.split = id % p.n_splits;
  const int u = id / p.n_splits;
  const int span = p.head_group * p.n_qtiles;
  const int g = u / span;
  const int r = u - g * span;
  const int h0 = g * p.head_group;
  const int gh = min(p.head_group, p.BH - h0);
  const int plane = h0 + r % gh;
  const int q0 = (p.n_qtiles - 1 - r / gh) * p.tile_tokens;
  it.b = plane / p.Hkv;
  it.kv_plane = plane - it.b * p.Hkv;
  it.rows = it.n = 0;
  it.full = false;
  it.j_begin = it.lo_masked = it.hi_masked = it.sink_steps = it.i0 = 0;
  const int c0 = p.cu_q[it.b], n = p.cu_q[it.b + 1] - c0;
  const int len = p.seqlens[it.b];
  it.tok0 = c0 + q0;
  it.len = len;
  it.pos0 = len - n + q0;
  if (c0 < 0 || n < 0 || n > p.max_q || n > p.total_q - c0 || len < n || len > p.max_k ||
      ((len - 1) >> p.page_log2) >= p.max_pages) {
    latch_status(p.status, kStatusBadLengths);
    return it;
  }
  if (q0 >= n) return it;
  const int n_tok = min(p.tile_tokens, n - q0);
  it.rows = n_tok * p.G;
  it.full = n_tok == p.tile_tokens;
  const int pos1 = it.pos0 + n_tok - 1;  // position of the tile's last token
  const int j_end = pos1 / kWN + 1;
  it.hi_masked = min((it.pos0 + 1) / kWN, j_end);
  if (p.window >= 0) {
    it.j_begin = max(it.pos0 - p.window, 0) / kWN;
    it.lo_masked = (max(pos1 - p.window, 0) + kWN - 1) / kWN;
    it.sink_steps = min((p.sinks + kWN - 1) / kWN, it.j_begin);
  }
  const int all = it.sink_steps + j_end - it.j_begin;
  it.i0 = it.split * p.split_steps;
  it.n = min(max(all - it.i0, 0), p.split_steps);
  return it;
}

// The pages of a 64-key step as a producer warp loads them: lane i the i-th, `rows` rows each (the
// whole step from one page when a page holds 64 tokens or more).
struct PageBox {
  int log2, rows;
  __device__ __forceinline__ explicit PageBox(int page_log2) : log2(min(page_log2, 6)), rows(1 << log2) {}
};

// A page's copy; STREAM: with the policy that evicts its lines first.
template <bool STREAM>
__device__ __forceinline__ void load_page(uint32_t dst, const CUtensorMap* m, uint32_t bar, int x, int y,
                                          int z, uint64_t policy) {
  if constexpr (STREAM)
    tma_load_3d_hint(dst, m, bar, x, y, z, policy);
  else
    tma_load_3d(dst, m, bar, x, y, z);
}

// This lane's block-table entry for step j; -1 where the lane has no page of it that holds tokens.
__device__ __forceinline__ int page_entry(const PagedParams& p, const PagedItem& it, int j, int lane) {
  const int first = lane << min(p.page_log2, 6);
  const int t = j * kWN + first;
  if (first >= kWN || t >= it.len) return -1;
  return p.block_table[static_cast<size_t>(it.b) * p.max_pages + (t >> p.page_log2)];
}

// The pool row the lane's load starts at; -1: no load.  An entry outside the pool is reported.
__device__ __forceinline__ int page_row(const PagedParams& p, const PagedItem& it, int j, int lane,
                                        int entry, bool report) {
  const int first = lane << min(p.page_log2, 6);
  const int t = j * kWN + first;
  if (first >= kWN || t >= it.len) return -1;
  if (entry < 0 || entry >= p.num_pages) {
    if (report) latch_status(p.status, kStatusBadLengths);
    return -1;
  }
  return (entry << p.page_log2) + (t & ((1 << p.page_log2) - 1));
}

// Position of row r of an item's tile, keys of its sequence, and its row of o and lse.
__device__ __forceinline__ int two_position(const WinItem& it, const WinParams& p, int r) {
  return it.qt * kWM + r + p.N_kv - p.N_q;
}
__device__ __forceinline__ int two_position(const PagedItem& it, const PagedParams& p, int r) {
  return it.pos0 + r / p.G;
}
__device__ __forceinline__ int two_keys(const WinItem&, const WinParams& p) { return p.N_kv; }
__device__ __forceinline__ int two_keys(const PagedItem& it, const PagedParams&) { return it.len; }
__device__ __forceinline__ size_t two_row(const WinItem& it, const WinParams& p, int r) {
  return static_cast<size_t>(it.bh) * p.N_q + it.qt * kWM + r;
}
__device__ __forceinline__ size_t two_row(const PagedItem& it, const PagedParams& p, int r) {
  return static_cast<size_t>(it.tok0 + r / p.G) * p.Hq + it.kv_plane * p.G + r % p.G;
}

// Parts of a row (key splits), and a part's (m, l) and 32 of its normalised columns.
__device__ __forceinline__ int two_parts(const WinParams&) { return 1; }
__device__ __forceinline__ int two_parts(const PagedParams& p) { return p.n_splits; }
__device__ __forceinline__ void two_write_ml(const WinItem&, const WinParams&, size_t, float, float) {}
__device__ __forceinline__ void two_write_ml(const PagedItem& it, const PagedParams& p, size_t row, float m,
                                             float l) {
  reinterpret_cast<float2*>(p.ws_ml)[row * p.n_splits + it.split] = make_float2(m, l);
}
// (by a warp, whose 32 rows go through 4 KB of shared memory so that four whole lines leave at a time;
// r0: the warp's first row)
template <int D>
__device__ __forceinline__ void two_write_part(const PagedItem& it, const PagedParams& p, int r0, int c,
                                               const uint32_t (&o)[32], float inv_l, uint8_t* scratch) {
  const int lane = threadIdx.x & 31;
  __syncwarp();
#pragma unroll
  for (int q = 0; q < 8; ++q)
    *reinterpret_cast<float4*>(scratch + sw128(lane, q)) =
        make_float4(__uint_as_float(o[q * 4]) * inv_l, __uint_as_float(o[q * 4 + 1]) * inv_l,
                    __uint_as_float(o[q * 4 + 2]) * inv_l, __uint_as_float(o[q * 4 + 3]) * inv_l);
  __syncwarp();
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    const int rr = q * 4 + (lane >> 3);
    if (r0 + rr < it.rows)
      *reinterpret_cast<float4*>(p.ws_o + (two_row(it, p, r0 + rr) * p.n_splits + it.split) * D + c * 32 +
                                 (lane & 7) * 4) =
          *reinterpret_cast<const float4*>(scratch + sw128(rr, lane & 7));
  }
}

template <bool PAGED>
struct TwoOf {
  using Params = WinParams;
  using Item = WinItem;
};
template <>
struct TwoOf<true> {
  using Params = PagedParams;
  using Item = PagedItem;
};

// Threads of a block: softmax, producer, two issuers; the paged variant has a producer for V.
constexpr int two_threads(bool paged) { return paged ? 256 : 224; }

__device__ __forceinline__ bool win_wait(uint32_t bar, uint32_t parity, volatile int* abort,
                                         int* status) {
  const bool ok = wait_bounded(bar, parity, abort, status);
  return __all_sync(0xffffffffu, ok);
}

// STREAM (paged): a cache that only one query tile reads is streamed through L2.  64 x 3-8 tokens over
// 1k-32k (Hq=64 Hkv=8 d=128) 747 -> 736 us, 16 tokens over 32k 42.5 -> 39.2; an instantiation of its own,
// since a choice at every copy costs long chunks 2.5%.
template <int D, bool BF16, bool PAGED, bool STREAM = false>
__global__ void __launch_bounds__(two_threads(PAGED), 2)
    attn_fwd_two_kernel(const __grid_constant__ CUtensorMap tm_q,
                        const __grid_constant__ CUtensorMap tm_k,
                        const __grid_constant__ CUtensorMap tm_v,
                        const __grid_constant__ CUtensorMap tm_o,
                        const typename TwoOf<PAGED>::Params p) {
  using L = WinLayout<D>;
  constexpr int KS = L::kKS, VS = L::kVS, NS = L::kNS;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  const uint32_t bars = base + L::kBar;
  const uint32_t bar_q = bars;
#define K_FULL(s) (bars + 8u * (1 + (s)))
#define K_EMPTY(s) (bars + 8u * (1 + KS + (s)))
#define V_FULL(s) (bars + 8u * (1 + 2 * KS + (s)))
#define V_EMPTY(s) (bars + 8u * (1 + 2 * KS + VS + (s)))
  const uint32_t bar_b = bars + 8u * (1 + 2 * KS + 2 * VS);
#define S_FULL(b) (bar_b + 8u * (b))
#define P_READY(b) (bar_b + 8u * (2 + (b)))
#define PV_DONE(b) (bar_b + 8u * (4 + (b)))
  const uint32_t bar_drain = bar_b + 8u * 6;
#define S_FREE(b) (bar_b + 8u * (7 + (b)))
  const uint32_t bar_drain_s = bar_b + 8u * 9;
  [[maybe_unused]] const uint32_t bar_ragged = bar_b + 8u * 10;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + L::kMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(gbase + L::kMisc + 4);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  const typename TwoOf<PAGED>::Item it = two_item(static_cast<int>(blockIdx.x), p);
  const int n = it.n;
  [[maybe_unused]] auto load_k = [&](int t) {
    mbar_arrive_expect_tx(K_FULL(t % KS), L::kStep);
#pragma unroll
    for (int sub = 0; sub < D / 64; ++sub)
      tma_load_3d(base + L::kK + (t % KS) * L::kStep + sub * kWSubKV, &tm_k, K_FULL(t % KS), sub * 64,
                  it.key_step(t) * kWN, it.kv_plane);
  };
  [[maybe_unused]] auto load_v = [&](int t) {
    mbar_arrive_expect_tx(V_FULL(t % VS), L::kStep);
#pragma unroll
    for (int sub = 0; sub < D / 64; ++sub)
      tma_load_3d(base + L::kV + (t % VS) * L::kStep + sub * kWSubKV, &tm_v, V_FULL(t % VS), sub * 64,
                  it.key_step(t) * kWN, it.kv_plane);
  };

  if (warp == 4 && lane == 0) {
    prefetch_tmap(&tm_q);
    prefetch_tmap(&tm_k);
    prefetch_tmap(&tm_v);
    mbar_init(bar_q, 1);
    for (int s = 0; s < KS; ++s) {
      mbar_init(K_FULL(s), 1);
      mbar_init(K_EMPTY(s), 1);
    }
    for (int s = 0; s < VS; ++s) {
      mbar_init(V_FULL(s), 1);
      mbar_init(V_EMPTY(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(S_FULL(b), 1);
      mbar_init(P_READY(b), kWM);
      mbar_init(PV_DONE(b), 1);
      mbar_init(S_FREE(b), kWM);
    }
    mbar_init(bar_drain, 1);
    mbar_init(bar_drain_s, 1);
    if constexpr (PAGED) mbar_init(bar_ragged, 1);
    *abort_flag = 0;
    fence_barrier_init();
    if constexpr (!PAGED) {
      // the first loads go out before the block's setup is done
      if (n > 0) {
        mbar_arrive_expect_tx(bar_q, L::kQBytes);
#pragma unroll
        for (int sub = 0; sub < D / 64; ++sub)
          tma_load_3d(base + sub * kWSubQ, &tm_q, bar_q, sub * 64, it.qt * kWM, it.bh);
        for (int t = 0; t < KS && t < n; ++t) load_k(t);
        for (int t = 0; t < VS && t < n; ++t) load_v(t);
      }
    }
  }
  // paged: this lane's block-table entry of the next step
  [[maybe_unused]] int entry = -1;
  if constexpr (PAGED) {
    if ((warp == 4 || warp == 7) && n > 0) entry = page_entry(p, it, it.key_step(0), lane);
  }
  if (warp == 5) {
    tmem_alloc(smem_u32(tmem_slot), kWTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 4) {
    // ------------------------------------------------- TMA producer (paged: of Q and K)
    if constexpr (PAGED) {
      if (n > 0) {
        const PageBox box(p.page_log2);
        // Rows of the query tile that no token fills stay zero.
        const int rows_filled = p.tile_tokens * p.G;
        for (int i = lane; i < (kWM - rows_filled) * (D / 8); i += 32) {
          const int row = rows_filled + i / (D / 8), c = i % (D / 8);
          *reinterpret_cast<uint4*>(gbase + (c >> 3) * kWSubQ + row * 128 + (c & 7) * 16) =
              make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive_expect_tx(bar_q, static_cast<uint32_t>(rows_filled) * D * 2);
#pragma unroll
          for (int sub = 0; sub < D / 64; ++sub)
            tma_load_3d(base + sub * kWSubQ, &tm_q, bar_q, sub * 64, it.kv_plane * p.G, it.tok0);
        }
        [[maybe_unused]] const uint64_t policy = STREAM ? l2_policy_evict_first() : 0;
        int issued = 0;
        for (int t = 0; t < n; ++t) {
          const int s = t % KS;
          const int row = page_row(p, it, it.key_step(t), lane, entry, true);
          if (t + 1 < n) entry = page_entry(p, it, it.key_step(t + 1), lane);
          bool ok = true;
          if (lane == 0 && t >= KS)
            ok = wait_bounded(K_EMPTY(s), ((t / KS) - 1) & 1, abort_flag, p.status);
          if (!__shfl_sync(0xffffffffu, ok, 0)) break;
          const uint32_t n_loads = __popc(__ballot_sync(0xffffffffu, row >= 0));
          if (lane == 0) mbar_arrive_expect_tx(K_FULL(s), n_loads * box.rows * D * 2);
          __syncwarp();
          if (row >= 0) {
#pragma unroll
            for (int sub = 0; sub < D / 64; ++sub)
              load_page<STREAM>(base + L::kK + s * L::kStep + sub * kWSubKV + lane * box.rows * 128, &tm_k,
                        K_FULL(s), sub * 64, it.kv_plane, row, policy);
          }
          issued = t + 1;
        }
        // Every asynchronous write into this block's shared memory lands before it may exit.
        if (lane == 0) {
          wait_bounded(bar_q, 0, nullptr, p.status, kWDrainNs);
          for (int t = (issued > KS ? issued - KS : 0); t < issued; ++t)
            wait_bounded(K_FULL(t % KS), (t / KS) & 1, nullptr, p.status, kWDrainNs);
        }
      }
    } else if (lane == 0 && n > 0) {
      int issued_k = min(KS, n), issued_v = min(VS, n);
      static_assert(KS == VS, "one loop for both rings");
      for (int t = KS; t < n; ++t) {
        if (!wait_bounded(K_EMPTY(t % KS), ((t / KS) - 1) & 1, abort_flag, p.status)) break;
        load_k(t);
        issued_k = t + 1;
        if (!wait_bounded(V_EMPTY(t % VS), ((t / VS) - 1) & 1, abort_flag, p.status)) break;
        load_v(t);
        issued_v = t + 1;
      }
      // Every asynchronous write into this block's shared memory lands before it may exit.
      wait_bounded(bar_q, 0, nullptr, p.status, kWDrainNs);
      for (int t = (issued_k > KS ? issued_k - KS : 0); t < issued_k; ++t)
        wait_bounded(K_FULL(t % KS), (t / KS) & 1, nullptr, p.status, kWDrainNs);
      for (int t = (issued_v > VS ? issued_v - VS : 0); t < issued_v; ++t)
        wait_bounded(V_FULL(t % VS), (t / VS) & 1, nullptr, p.status, kWDrainNs);
    }
    __syncwarp();
  } else if (warp == 5) {
    // ----------------------------------------------------------------- tcgen05 issuer of S
    if (lane == 0 && n > 0) {
      constexpr uint32_t idesc_qk = make_idesc_f16(BF16, kWM, kWN, false);
      const uint64_t q_desc = make_sdesc_sw128(base, 16, 1024);
      if (wait_bounded(bar_q, 0, abort_flag, p.status)) {
        for (int t = 0; t < n; ++t) {  // S_t into buffer t % NS, once S_{t-NS} has been read
          const int s = t % KS, b = t % NS;
          if (!wait_bounded(K_FULL(s), (t / KS) & 1, abort_flag, p.status)) break;
          if (t >= NS && !wait_bounded(S_FREE(b), ((t / NS) - 1) & 1, abort_flag, p.status)) break;
          tc_fence_after();
          const uint64_t k_desc = make_sdesc_sw128(base + L::kK + s * L::kStep, 16, 1024);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            mma_ss(tmem + kWColS + b * kWN, q_desc + (((kk >> 2) * kWSubQ + (kk & 3) * 32) >> 4),
                   k_desc + (((kk >> 2) * kWSubKV + (kk & 3) * 32) >> 4), idesc_qk, kk > 0 ? 1u : 0u);
          mma_commit(S_FULL(b));
          mma_commit(K_EMPTY(s));
        }
      }
      // every MMA this thread issued completes before the block frees its tensor memory
      mma_commit(bar_drain_s);
      wait_bounded(bar_drain_s, 0, nullptr, p.status, kWDrainNs);
    }
    __syncwarp();
  } else if (PAGED && warp == 7) {
    // ----------------------------------------------------------------- V producer (paged)
    if constexpr (PAGED) {
      if (n > 0) {
        const PageBox box(p.page_log2);
        int issued = 0;
        [[maybe_unused]] const uint64_t policy = STREAM ? l2_policy_evict_first() : 0;
        uint32_t ragged = 0;  // ragged steps so far
        for (int t = 0; t < n; ++t) {
          const int s = t % VS, j = it.key_step(t);
          const int row = page_row(p, it, j, lane, entry, false);
          if (t + 1 < n) entry = page_entry(p, it, it.key_step(t + 1), lane);
          bool ok = true;
          if (lane == 0 && t >= VS)
            ok = wait_bounded(V_EMPTY(s), ((t / VS) - 1) & 1, abort_flag, p.status);
          if (!__shfl_sync(0xffffffffu, ok, 0)) break;
          // The step that holds the sequence's end: its rows past the end hold other sequences' or
          // unwritten tokens, or were not loaded at all.  P is zero there, but 0 * V has to stay 0:
          // the rows are cleared once the loads have landed, and only then is the step handed on.  The
          // same for pages that could not be loaded.
          const uint32_t loaded = __ballot_sync(0xffffffffu, row >= 0);
          const uint32_t bytes = __popc(loaded) * box.rows * D * 2;
          const int valid = it.len - j * kWN;  // rows of the step that hold tokens
          const bool clear = valid < kWN || bytes < L::kStep;
          const uint32_t bar = clear ? bar_ragged : V_FULL(s);
          if (lane == 0) mbar_arrive_expect_tx(bar, bytes);
          __syncwarp();
          if (row >= 0) {
#pragma unroll
            for (int sub = 0; sub < D / 64; ++sub)
              load_page<STREAM>(base + L::kV + s * L::kStep + sub * kWSubKV + lane * box.rows * 128, &tm_v, bar,
                        sub * 64, it.kv_plane, row, policy);
          }
          if (clear) {
            if (!win_wait(bar, ragged & 1, abort_flag, p.status)) break;
            ++ragged;
            for (int i = lane; i < kWN * (D / 8); i += 32) {
              const int rr = i / (D / 8), c = i % (D / 8);
              if (rr >= valid || !((loaded >> (rr >> box.log2)) & 1u))
                *reinterpret_cast<uint4*>(gbase + L::kV + s * L::kStep + (c >> 3) * kWSubKV + rr * 128 +
                                          (c & 7) * 16) = make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(V_FULL(s));
          }
          issued = t + 1;
        }
        // loads that nothing waited for land before the block may exit (an aborted ragged step's wait
        // has already taken its limit)
        if (lane == 0)
          for (int t = (issued > VS ? issued - VS : 0); t < issued; ++t)
            wait_bounded(V_FULL(t % VS), (t / VS) & 1, nullptr, p.status, kWDrainNs);
      }
    }
    __syncwarp();
  } else if (warp == 6) {
    // ----------------------------------------------------------------- tcgen05 issuer of O += P V
    if (lane == 0 && n > 0) {
      constexpr uint32_t idesc_pv = make_idesc_f16(BF16, kWM, D, true);
      for (int t = 0; t < n; ++t) {
        const int s = t % VS, b = t & 1;
        if (!wait_bounded(V_FULL(s), (t / VS) & 1, abort_flag, p.status)) break;
        if (!wait_bounded(P_READY(b), (t >> 1) & 1, abort_flag, p.status)) break;
        tc_fence_after();
        // V is [keys, d] with d contiguous: an MN-major operand, 16 keys per step of the product
        const uint64_t v_desc = make_sdesc_sw128(base + L::kV + s * L::kStep, kWSubKV, 1024);
#pragma unroll
        for (int kk = 0; kk < kWN / 16; ++kk)
          mma_ts(tmem + L::kColO, tmem + kWColP + b * (kWN / 2) + kk * 8, v_desc + ((kk * 16 * 128) >> 4),
                 idesc_pv, (t > 0 || kk > 0) ? 1u : 0u);
        mma_commit(PV_DONE(b));
        mma_commit(V_EMPTY(s));
      }
      mma_commit(bar_drain);
      wait_bounded(bar_drain, 0, nullptr, p.status, kWDrainNs);
    }
    __syncwarp();
  } else {
    // ----------------------------------------------------------------- softmax + epilogue
    const int r = warp * 32 + lane;
    const uint32_t row_tmem = tmem + (static_cast<uint32_t>(warp * 32) << 16);
    const float sl2 = p.sl2;
    const bool store = r < it.rows;
    const int pos = two_position(it, p, r);  // this row's position, and the last key it may see
    const int last = min(pos, two_keys(it, p) - 1);
    const size_t row_index = store ? two_row(it, p, r) : 0;  // of o and lse
    float m = -INFINITY, l = 0.0f;
    bool ok = true;
    for (int t = 0; t < n; ++t) {
      const int j = it.key_step(t);
      const int b = t & 1;
      if (!win_wait(S_FULL(t % NS), (t / NS) & 1, abort_flag, p.status)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const uint32_t s_addr = row_tmem + kWColS + (t % NS) * kWN;
      uint32_t sr[2][32];
      tmem_ld32(s_addr, sr[0]);
      tmem_ld32(s_addr + 32, sr[1]);
      tmem_wait_ld();
      tc_fence_before();
      mbar_arrive(S_FREE(t % NS));
      if (j >= it.hi_masked || j < it.lo_masked) {
        // visible columns: [lo, hi] and the sinks up to sk
        const int hi = min(last - j * kWN, kWN - 1);
        const int lo = j < it.lo_masked ? max(pos - p.window - j * kWN, 0) : 0;
        const int sk = min(p.sinks - 1 - j * kWN, hi);
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          const int a = max(lo - 32 * g, 0), bb = min(hi - 32 * g, 31);
          const int ss = min(sk - 32 * g, 31);
          uint32_t vis = (a > bb) ? 0u : ((0xffffffffu >> (31 - bb)) & (0xffffffffu << a));
          vis |= (ss < 0) ? 0u : (0xffffffffu >> (31 - ss));
          // the score where visible, -inf where not: by bits, so that a NaN or infinite score of a
          // masked key leaves no trace
#pragma unroll
          for (int c = 0; c < 32; ++c) sr[g][c] = (vis & (1u << c)) ? sr[g][c] : 0xff800000u;
        }
      }
      float mx[8];
#pragma unroll
      for (int e = 0; e < 8; ++e)
        mx[e] = fmaxf(__uint_as_float(sr[0][e]), __uint_as_float(sr[1][e]));
#pragma unroll
      for (int c = 8; c < 32; c += 8)
#pragma unroll
        for (int e = 0; e < 8; ++e)
          mx[e] = max3f(mx[e], __uint_as_float(sr[0][c + e]), __uint_as_float(sr[1][c + e]));
      const float tile_max = max3f(max3f(mx[0], mx[1], mx[2]), max3f(mx[3], mx[4], mx[5]),
                                   fmaxf(mx[6], mx[7]));
      // the maximum moves when it rises by more than 2^8 (and at the first finite one)
      const float m_new = fmaxf(m, tile_max * sl2);
      float alpha = 1.0f;
      if (m_new - m > kWRescale) {
        alpha = ex2(m - m_new);
        m = m_new;
        l *= alpha;
      }
      const float neg_mu = (m == -INFINITY) ? 0.0f : -m;
      uint32_t pk[32];
      float ps[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int g = 0; g < 2; ++g)
#pragma unroll
        for (int c = 0; c < 32; c += 2) {
          float a0, a1;
          fma2(a0, a1, __uint_as_float(sr[g][c]), __uint_as_float(sr[g][c + 1]), sl2, sl2, neg_mu,
               neg_mu);
          sr[g][c] = __float_as_uint(ex2(a0));
          sr[g][c + 1] = __float_as_uint(ex2(a1));
        }
#pragma unroll
      for (int g = 0; g < 2; ++g)
#pragma unroll
        for (int c = 0; c < 32; c += 2) {
          const float p0 = __uint_as_float(sr[g][c]), p1 = __uint_as_float(sr[g][c + 1]);
          const int k2 = c & 6;
          add2(ps[k2], ps[k2 + 1], p0, p1);
          pk[(g * 32 + c) >> 1] = pack2<BF16>(p0, p1);
        }
      l += ((ps[0] + ps[1]) + (ps[2] + ps[3])) + ((ps[4] + ps[5]) + (ps[6] + ps[7]));
      if (t > 0 && __any_sync(0xffffffffu, alpha != 1.0f)) {
        // P V_{t-1} done; P V_t waits for this step's P, so nothing else touches O meanwhile
        if (!win_wait(PV_DONE(b ^ 1), ((t - 1) >> 1) & 1, abort_flag, p.status)) {
          ok = false;
          break;
        }
        tc_fence_after();
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32];
          tmem_ld32(row_tmem + L::kColO + c * 32, o);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
          tmem_st32(row_tmem + L::kColO + c * 32, o);
        }
      }
      if (t > 1) {  // P V_{t-2} read this buffer
        if (!win_wait(PV_DONE(b), ((t - 2) >> 1) & 1, abort_flag, p.status)) {
          ok = false;
          break;
        }
        tc_fence_after();
      }
      tmem_st32(row_tmem + kWColP + b * (kWN / 2), pk);
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(P_READY(b));
    }
    const bool whole = !PAGED || two_parts(p) == 1;  // else the row is one of several parts
    if (n == 0) {
      // No key visible to any row of this tile: O = 0, L = -inf (of a part: no weight in the merge).
      if (store && !whole) {
        two_write_ml(it, p, row_index, -INFINITY, 0.0f);
      } else if (store) {
        uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.o) + row_index * D);
#pragma unroll
        for (int c = 0; c < D / 8; ++c) dst[c] = make_uint4(0, 0, 0, 0);
        p.lse[row_index] = -INFINITY;
      }
    } else {
      // O / l into Q's shared memory (its products are done) and out by one TMA store per 64 columns,
      // where the tile's rows are all the item's; a warp whose wait ran out still meets the others at the
      // barrier
      const bool staged = !PAGED || (whole && it.full);
      if (ok) ok = win_wait(PV_DONE((n - 1) & 1), ((n - 1) >> 1) & 1, abort_flag, p.status);
      if (ok) {
        tc_fence_after();
        const float inv_l = (l > 0.0f) ? 1.0f / l : (l == 0.0f ? 0.0f : l);  // a NaN sum stays one
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32];
          tmem_ld32(row_tmem + L::kColO + c * 32, o);
          tmem_wait_ld();
          if constexpr (PAGED) {
            if (!whole) {
              two_write_part<D>(it, p, warp * 32, c, o, inv_l, gbase + warp * 4096);
              continue;
            }
          }
#pragma unroll
          for (int q4 = 0; q4 < 4; ++q4) {
            const uint4 w = make_uint4(
                pack2<BF16>(__uint_as_float(o[q4 * 8 + 0]) * inv_l, __uint_as_float(o[q4 * 8 + 1]) * inv_l),
                pack2<BF16>(__uint_as_float(o[q4 * 8 + 2]) * inv_l, __uint_as_float(o[q4 * 8 + 3]) * inv_l),
                pack2<BF16>(__uint_as_float(o[q4 * 8 + 4]) * inv_l, __uint_as_float(o[q4 * 8 + 5]) * inv_l),
                pack2<BF16>(__uint_as_float(o[q4 * 8 + 6]) * inv_l, __uint_as_float(o[q4 * 8 + 7]) * inv_l));
            const uint32_t chunk = c * 4 + q4;
            if (staged)
              *reinterpret_cast<uint4*>(gbase + (chunk >> 3) * kWSubQ + sw128(r, chunk & 7)) = w;
            else if (store)
              reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.o) + row_index * D)[chunk] = w;
          }
        }
        if (store && !whole)
          two_write_ml(it, p, row_index, m, l);
        else if (store)
          p.lse[row_index] = (l == 0.0f) ? -INFINITY
                                         : ((m == -INFINITY ? 0.0f : m) + lg2(l)) * 0.69314718055994531f;
      }
      fence_proxy_async_smem();
      named_bar_sync(1, kWM);
      if (staged && threadIdx.x == 0 && *abort_flag == 0) {
#pragma unroll
        for (int sub = 0; sub < D / 64; ++sub) {
          if constexpr (PAGED)
            tma_store_3d(&tm_o, base + sub * kWSubQ, sub * 64, it.kv_plane * p.G, it.tok0);
          else
            tma_store_3d(&tm_o, base + sub * kWSubQ, sub * 64, it.qt * kWM, it.bh);
        }
        tma_store_commit();
        tma_store_wait_read0();  // the block's shared memory may go
      }
    }
  }
#undef K_FULL
#undef K_EMPTY
#undef V_FULL
#undef V_EMPTY
#undef S_FULL
#undef P_READY
#undef PV_DONE
#undef S_FREE
  tc_fence_before();
  __syncthreads();
  if (warp == 5) {
    tc_fence_after();
    tmem_dealloc(tmem, kWTmemCols);
  }
}

}  // namespace attn
