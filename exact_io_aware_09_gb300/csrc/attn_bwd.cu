// Backward pass of exact attention by recomputation, sm_103a.
//
// "FlashAttention Explained", section "Backward Pass: Recomputation Beats Storage": the forward
// pass saves O and one log-sum-exp L per row; the backward pass recomputes the score and
// probability tiles from Q, K and L (P = exp(S - L)) and forms
//     dV = P^T dO,  dP = dO V^T,  dS = P o (dP - D) with D_i = rowsum(dO_i o O_i),
//     dQ = scale dS K,  dK = scale dS^T Q.
// The pages note that accumulating dQ across key tiles with atomic adds makes the result
// nondeterministic.  Here every gradient is owned by exactly one thread block, so the result is
// deterministic by construction:
//   kernel 0  D and L log2(e) per query row (padded to whole 128-row tiles);
//   kernel 1  one block per 128-key tile of one (batch, key/value head): loops over the query
//             tiles of every query head that shares the key/value head and keeps dK and dV in
//             tensor memory (four MMAs per step: S^T, dP^T, dV += P^T dO, dK += dS^T Q);
//   kernel 2  one block per 128-row query tile: loops over the key tiles and keeps dQ in
//             tensor memory (three MMAs per step: S, dP, dQ += dS K).
// S and dP are recomputed in both kernels (seven MMAs per tile pair instead of five): the price
// of owning every output without atomics.
//
// The dK/dV kernel steps through 64 queries at a time (S^T and dP^T as 128 x 64 products,
// double-buffered, so one step's elementwise work overlaps the next step's products); the dQ
// kernel takes whole 128 x 128 tiles with single S and dP buffers that are released as soon as
// they have been read.  The two elementwise warpgroups take alternate steps in kernel 1 and
// split each tile's keys in kernel 2.  Probabilities and dS go back to tensor memory as 16-bit
// pairs (over the fp32 columns they came from, or into a buffer of their own) and feed the
// accumulating MMAs as their A operand.
//
// Roles inside a thread block (384 threads): warps 0-3 and 4-7 the elementwise warpgroups
// (thread = one row of the tensor-memory tiles: a key in kernel 1, a query in kernel 2), warp 8
// the TMA producer, warp 9 the issuer of the score products (S^T or S; it owns the
// tensor-memory allocation), warp 11 the issuer of dP^T or dP, warp 10 the issuer of the
// accumulations (dV and dK, or dQ).  Each issuing thread commits its own products; the
// hand-offs between them run through the elementwise warps' barriers.  Every wait on a barrier
// is bounded.
//
// Roundings.  P and dS enter their products in the operands' 16-bit type, since the tensor cores multiply
// operands of one type: each term of dV, dK and dQ is off by at most half a step (2^-8 of it in bf16,
// 2^-11 in fp16), about as much as rounding the gradients themselves; products with what the roundings
// leave would add three to the seven.  In fp16 both are held times powers of two that keep them within
// its normal numbers (grad_scale in attn_bwd.cuh; kernel 0 takes the ranges, which costs it a pass over V).
// D is formed from O as stored.  Sums, S, dP and the exponentials are fp32.
//
// The window variant (WINDOW; a sliding window whose first keys, the sinks, stay visible) walks only
// the tiles a row sees.  A key tile with sinks is seen by every later query row, many times what a
// tile of the window is: its query tiles are cut into parts, blocks of their own whose fp32 sums a
// last kernel adds in order (B=1 Hq=64 Hkv=8 N=8192 d=128, W=1024, 64 sinks: forward and gradients
// 1,788 -> 1,369 us).  The masks sit in a branch of their own: as tests per column inside the
// exponential loop they cost every tile (gradients 1,028 -> 882 us at 4 sinks).  The same shape now: D
// 42 us, dK/dV 437 (tensor pipe 70% busy), dQ 376 (56%: nine key tiles a block do not hide its start and
// end), sums 5.  At d = 64 calls of many short tiles take the kernels of attn_bwd_window.cu.
#include <algorithm>
#include <list>
#include <map>
#include <mutex>
#include <queue>
#include <tuple>
#include <vector>

#include "attn_bwd.cuh"

namespace attn {

namespace {

constexpr int kKvThreads = 384;    // three issuing warps in either kernel
constexpr int kQThreads = 384;
constexpr int kEwThreads = 128;     // one elementwise warpgroup (two of them: warps 0-3, 4-7)
// warp 9 issues the score products S^T or S (and owns the tensor-memory allocation), warp 11
// the dP^T or dP products, warp 10 the gradient accumulations.  Several issuing threads keep
// the tensor pipe's short queue fed while one of them waits on a barrier.
constexpr int kBwdProducerWarp = 8, kBwdIssuerWarp = 9, kBwdAccWarp = 10, kBwdDpWarp = 11;
constexpr uint32_t kBwdTmemCols = 512;

template <bool BF16>
__device__ __forceinline__ float half_to_f32(uint32_t h) {
  if constexpr (BF16) {
    return __uint_as_float(h << 16);
  } else {
    float f;
    asm("{\n\t.reg .f16 t;\n\tmov.b16 t, %1;\n\tcvt.f32.f16 %0, t;\n\t}" : "=f"(f) : "h"(static_cast<uint16_t>(h)));
    return f;
  }
}

}  // namespace

// ------------------------------------------------------------------------------------------
// kernel 0: -scale D = -scale rowsum(dO o O) and -L log2(e), d / 8 lanes per (padded) query row
// ------------------------------------------------------------------------------------------
// Bound by HBM: 4 d bytes a row.  Four rows a lane, all loaded before the first is summed: 42 us at B=1
// Hq=64 N=8192 d=128 (268 MB, 6.4 TB/s), one row a lane 50.
constexpr int kPreRows = 4;

// The largest of a block's values (none negative) into N words that start at 0.  (With a warp's each
// straight to the words the gradients of fp16 B=4 H=32 N=4096 d=128, W=256, take 700 us and not 633.)
template <int N>
__device__ __forceinline__ void block_max_to(uint32_t* word, const float (&v)[N]) {
  __shared__ uint32_t top[N][8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const uint32_t w = __reduce_max_sync(0xffffffffu, __float_as_uint(v[i]));
    if (lane == 0) top[i][warp] = w;
  }
  __syncthreads();
  if (warp < N) {
    const uint32_t w = __reduce_max_sync(0xffffffffu, lane < 8 ? top[warp][lane] : 0u);
    if (lane == 0 && w > __ldcg(word + warp)) atomicMax(word + warp, w);
  }
}

// fp16: also the ranges of each plane (grad_scale); the blocks from q_blocks on take the rows of V.  The
// ranges, their use and the words' clearing cost, W=256: B=8 H=12 N=1024 d=64 65 -> 68 us, B=1 Hq=64 Hkv=8
// N=8192 d=128 492 -> 508, B=4 H=32 N=4096 d=128 591 -> 633.
template <int D, bool BF16>
__global__ void __launch_bounds__(256)
    attn_bwd_pre_kernel(const uint16_t* o, const uint16_t* dout, const uint16_t* v, const float* lse,
                        float* lse2, float* dvec, uint32_t* range, int N_q, int nqp, int N_kv, int Hq,
                        int Hkv, long long rows, unsigned q_blocks, float scale) {
  // D / 8 lanes per row, 16-byte loads of O and dO
  constexpr int kLanes = D / 8;
  if (threadIdx.x == 0) griddep_launch_dependents();  // dK/dV's setup and first loads may start
  const int lane = threadIdx.x % kLanes;
  if constexpr (!BF16) {
    if (blockIdx.x >= q_blocks) {
      constexpr int kRows = 256 / kLanes * kPreRows;  // of a block
      const unsigned per = (static_cast<unsigned>(N_kv) + kRows - 1) / kRows;
      const unsigned vb = blockIdx.x - q_blocks;
      const int j0 = static_cast<int>(vb % per) * kRows + static_cast<int>(threadIdx.x / kLanes) * kPreRows;
      float top = 0.0f;
      uint4 a[kPreRows];
#pragma unroll
      for (int u = 0; u < kPreRows; ++u)
        a[u] = j0 + u < N_kv ? *reinterpret_cast<const uint4*>(
                                   v + (static_cast<size_t>(vb / per) * N_kv + j0 + u) * D + lane * 8)
                             : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int u = 0; u < kPreRows; ++u) {
        const uint32_t av[4] = {a[u].x, a[u].y, a[u].z, a[u].w};
        float sq = 0.0f;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const float lo = half_to_f32<BF16>(av[c] & 0xffffu), hi = half_to_f32<BF16>(av[c] >> 16);
          sq = fmaf(lo, lo, fmaf(hi, hi, sq));
        }
#pragma unroll
        for (int sh = kLanes / 2; sh > 0; sh >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, sh);
        top = fmaxf(top, sq);
      }
      block_max_to<1>(range + vb / per * 4 + 2, {sqrtf(top)});
      return;
    }
  }
  const long long w0 =
      (static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x) / kLanes * kPreRows;
  // the first row's (batch, query head) and index; nqp is a multiple of the rows a block takes
  const long long bh = w0 < rows ? w0 / nqp : 0;
  const int i0 = w0 < rows ? static_cast<int>(w0 - bh * nqp) : N_q;
  uint4 a[kPreRows], b[kPreRows];
#pragma unroll
  for (int u = 0; u < kPreRows; ++u) {
    a[u] = b[u] = make_uint4(0, 0, 0, 0);
    if (i0 + u < N_q) {
      const size_t base = (static_cast<size_t>(bh) * N_q + i0 + u) * D + lane * 8;
      a[u] = *reinterpret_cast<const uint4*>(o + base);
      b[u] = *reinterpret_cast<const uint4*>(dout + base);
    }
  }
  [[maybe_unused]] float top_do = 0.0f, top_d = 0.0f;
#pragma unroll
  for (int u = 0; u < kPreRows; ++u) {
    const uint32_t av[4] = {a[u].x, a[u].y, a[u].z, a[u].w}, bv[4] = {b[u].x, b[u].y, b[u].z, b[u].w};
    float acc = 0.0f;
    [[maybe_unused]] float sq = 0.0f;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const float lo = half_to_f32<BF16>(bv[c] & 0xffffu), hi = half_to_f32<BF16>(bv[c] >> 16);
      acc = fmaf(half_to_f32<BF16>(av[c] & 0xffffu), lo, acc);
      acc = fmaf(half_to_f32<BF16>(av[c] >> 16), hi, acc);
      if constexpr (!BF16) sq = fmaf(lo, lo, fmaf(hi, hi, sq));
    }
#pragma unroll
    for (int sh = kLanes / 2; sh > 0; sh >>= 1) {
      acc += __shfl_xor_sync(0xffffffffu, acc, sh);
      if constexpr (!BF16) sq += __shfl_xor_sync(0xffffffffu, sq, sh);
    }
    if constexpr (!BF16) {
      top_do = fmaxf(top_do, sq);
      top_d = fmaxf(top_d, fabsf(scale * acc));
    }
    if (w0 < rows && lane == 0) {
      // stored negated (and D times the scale), so that the elementwise steps are single FMAs:
      // s * scale log2(e) + (-L log2(e)) and dP * scale + (-scale D)
      const int i = i0 + u;
      dvec[w0 + u] = (i < N_q) ? -scale * acc : 0.0f;
      // a row that sees no key (L = -inf) takes part in nothing, as the padding rows
      const float L = (i < N_q) ? lse[bh * N_q + i] : -INFINITY;
      const float shift = BF16 ? 0.0f : static_cast<float>(kPShift);
      lse2[w0 + u] = (L == -INFINITY) ? -INFINITY : fmaf(-L, 1.4426950408889634f, shift);
    }
  }
  if constexpr (!BF16) {
    uint32_t* w = range + ((bh / Hq) * Hkv + (bh % Hq) / (Hq / Hkv)) * 4;
    block_max_to<2>(w, {sqrtf(top_do), top_d});
  }
}

// ------------------------------------------------------------------------------------------
// kernel 1: dK, dV of one 128-key tile
// ------------------------------------------------------------------------------------------
// The query tiles stream through a ring of shared-memory stages of 64 queries (Q, dO, and their
// L log2(e) and D), taken one stage per step: S^T and dP^T (128 keys x 64 queries) are
// double-buffered in tensor memory, and elementwise warpgroup w takes the steps of buffer w, so
// that the MMAs of one step run while the elementwise step of the other is computed.  Tensor
// memory: S^T[2] 0-127, dP^T[2] 128-255, dV 256-(256+d), dK after it; P^T and dS^T go back as
// 16-bit pairs over the first 32 columns of the buffers they came from.

// Dispatch order of the dK/dV kernel's blocks.  A block's work grows with the query tiles that
// see its key tile, and under the causal mask the longest blocks are long against a GPU's share
// of the whole (a 128-key tile of an 8192-token sequence with eight query heads: 1,024 64-query
// steps, against about 1,750 per SM): started longest first, the blocks leave a tail of about 7%.
// The launcher packs the blocks into one bin per SM (largest first, each into the fullest bin
// that stays under the average load) and lists them in the order in which SMs that free up in
// turn would take them; block i of the launch then runs job order.job[i].  n = 0: the default
// order (key tile major, job = block index).
constexpr int kMaxKvOrder = 2048;
struct KvOrder {
  int n;
  uint16_t job[kMaxKvOrder];
};

template <int D, int QS>
struct KvLayout {
  static constexpr uint32_t kTile = kBT * D * 2;             // K or V: 128 rows
  static constexpr uint32_t kHalf = kStepQ * D * 2;          // Q or dO: 64 rows
  static constexpr uint32_t kHalfSub = kStepQ * 128;         // one 64-column sub-tile of it
  static constexpr uint32_t kStage = (2 * kHalf + 512 + 1023) / 1024 * 1024;
  static constexpr uint32_t kK = 0;
  static constexpr uint32_t kV = kTile;
  static constexpr uint32_t kStages = 2 * kTile;
  static constexpr uint32_t kBar = kStages + QS * kStage;
  // kv_full, st_full[QS], st_empty[QS], s_full[2], dp_full[2], p_ready[2], drain,
  // p_free[2], ds_free[2], drain of the S^T issuer, ds_ready[2], drain of the dP^T issuer
  static constexpr uint32_t kNumBars = 1 + 2 * QS + 15;
  static constexpr uint32_t kMisc = kBar + kNumBars * 8;  // tmem slot, abort flag
  static constexpr uint32_t kBytes = kMisc + 16 + 1024;
  static constexpr uint32_t kColS = 0, kColDP = 128, kColDV = 256, kColDK = 256 + D;
  static_assert(kTile % 1024 == 0 && kHalf % 1024 == 0, "tile alignment");
  static_assert(kBytes <= 232448, "shared memory per block");
};

template <int D, bool BF16, int QS, bool WINDOW>
__global__ void __launch_bounds__(kKvThreads, 1)
    attn_bwd_dkdv_kernel(const __grid_constant__ CUtensorMap tm_q,
                         const __grid_constant__ CUtensorMap tm_k,
                         const __grid_constant__ CUtensorMap tm_v,
                         const __grid_constant__ CUtensorMap tm_do,
                         const __grid_constant__ CUtensorMap tm_dk,
                         const __grid_constant__ CUtensorMap tm_dv, const BwdParams p,
                         const __grid_constant__ KvOrder order) {
  using L = KvLayout<D, QS>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  const uint32_t bars = base + L::kBar;
  const uint32_t bar_kv = bars;
#define ST_FULL(s) (bars + 8u * (1 + (s)))
#define ST_EMPTY(s) (bars + 8u * (1 + QS + (s)))
  const uint32_t bar_b = bars + 8u * (1 + 2 * QS);
#define S_FULL(b) (bar_b + 8u * (b))           // S^T of buffer b written (MMA commit)
#define DP_FULL(b) (bar_b + 8u * (2 + (b)))     // dP^T of buffer b written (MMA commit)
#define P_READY(b) (bar_b + 8u * (4 + (b)))     // P^T of buffer b stored (128 arrivals)
#define DS_READY(b) (bar_b + 8u * (12 + (b)))   // dS^T of buffer b stored (128 arrivals)
#define P_FREE(b) (bar_b + 8u * (7 + (b)))      // dV product of buffer b done: S^T columns free
#define DS_FREE(b) (bar_b + 8u * (9 + (b)))     // dK product of buffer b done: dP^T columns free
  const uint32_t bar_drain = bar_b + 8u * 6;
  const uint32_t bar_drain_s = bar_b + 8u * 11;
  const uint32_t bar_drain_dp = bar_b + 8u * 14;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + L::kMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(gbase + L::kMisc + 4);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  // The dQ kernel needs nothing this one writes: its blocks may take the SMs this grid's
  // blocks leave, as soon as every block of this grid has started and kernel 0 has ended (dQ
  // reads its vectors too).
  if (threadIdx.x == 0) {
    griddep_wait();
    griddep_launch_dependents();
  }

  // job: key tile kt of (batch, key/value head) bkv, numbered key tile major; the launch order
  // is the packed one of KvOrder when the launcher gives one
  const int n_planes =
      static_cast<int>(gridDim.x) /
      (WINDOW ? p.n_kvtiles + p.sink_tiles * (p.sink_parts - 1) : p.n_kvtiles);
  int job = order.n ? static_cast<int>(order.job[blockIdx.x]) : static_cast<int>(blockIdx.x);
  // window variant: a key tile with sinks is seen by every later row, many times what a tile of
  // the window is; its query tiles are cut into sink_parts blocks (numbered first, part major)
  [[maybe_unused]] int part = 0;
  if constexpr (WINDOW) {
    const int n_sink = n_planes * p.sink_tiles;
    if (job < n_sink * p.sink_parts) {
      part = job / n_sink;
      job -= part * n_sink;
    } else {
      job -= n_sink * (p.sink_parts - 1);
    }
  }
  const int kt = job / n_planes;
  const int bkv = job % n_planes;
  const int b = bkv / p.Hkv;
  const int hk = bkv % p.Hkv;
  const int off = p.N_kv - p.N_q;
  int qt_lo = 0;
  if (p.causal) {
    const int first_row = kt * kBT - off;  // first query row that sees key kt * 128
    qt_lo = first_row > 0 ? first_row / kBT : 0;
  }
  int qt_hi = p.n_qtiles;
  if constexpr (WINDOW) window_q_tiles(kt, p.n_qtiles, off, p.window, p.sinks, qt_lo, qt_hi);
  const int nq_per = qt_hi - qt_lo;  // query tiles per query head
  int n = nq_per > 0 ? p.G * nq_per : 0;
  int tile0 = 0;                          // first (query head, query tile) pair of this block
  [[maybe_unused]] const bool partial = WINDOW && kt < p.sink_tiles && p.sink_parts > 1;
  if constexpr (WINDOW) {
    if (partial) {
      tile0 = static_cast<int>(static_cast<long long>(n) * part / p.sink_parts);
      n = static_cast<int>(static_cast<long long>(n) * (part + 1) / p.sink_parts) - tile0;
    }
  }
  const int n_steps = 2 * n;              // two 64-query steps per query tile
  auto load_stage = [&](int i) {
    const int s = i % QS;
    const int tile = tile0 + (i >> 1);
    const int g = tile / nq_per;
    const int q0 = (qt_lo + tile % nq_per) * kBT + (i & 1) * kStepQ;
    const int bhq = b * p.Hq + hk * p.G + g;
    const uint32_t st = base + L::kStages + s * L::kStage;
    mbar_arrive_expect_tx(ST_FULL(s), 2 * L::kHalf + 512);
#pragma unroll
    for (int sub = 0; sub < D / 64; ++sub) {
      tma_load_3d(st + sub * L::kHalfSub, &tm_q, ST_FULL(s), sub * 64, q0, bhq);
      tma_load_3d(st + L::kHalf + sub * L::kHalfSub, &tm_do, ST_FULL(s), sub * 64, q0, bhq);
    }
    if (i == 0) griddep_wait();  // kernel 0's vectors
    const size_t vec = static_cast<size_t>(bhq) * p.nqp + static_cast<size_t>(q0);
    bulk_load(st + 2 * L::kHalf, p.lse2 + vec, kStepQ * 4, ST_FULL(s));
    bulk_load(st + 2 * L::kHalf + 256, p.dvec + vec, kStepQ * 4, ST_FULL(s));
  };

  if (warp == kBwdProducerWarp && lane == 0) {
    mbar_init(bar_kv, 1);
    for (int s = 0; s < QS; ++s) {
      mbar_init(ST_FULL(s), 1);
      mbar_init(ST_EMPTY(s), 1);
    }
    for (int bb = 0; bb < 2; ++bb) {
      mbar_init(S_FULL(bb), 1);
      mbar_init(DP_FULL(bb), 1);
      mbar_init(P_READY(bb), kEwThreads);
      mbar_init(DS_READY(bb), kEwThreads);
      mbar_init(P_FREE(bb), 1);
      mbar_init(DS_FREE(bb), 1);
    }
    mbar_init(bar_drain, 1);
    mbar_init(bar_drain_s, 1);
    mbar_init(bar_drain_dp, 1);
    *abort_flag = 0;
    fence_barrier_init();
    // the first loads go out before the block's setup is done
    if (n > 0) {
      mbar_arrive_expect_tx(bar_kv, 2 * L::kTile);
#pragma unroll
      for (int sub = 0; sub < D / 64; ++sub) {
        tma_load_3d(base + L::kK + sub * kSub, &tm_k, bar_kv, sub * 64, kt * kBT, bkv);
        tma_load_3d(base + L::kV + sub * kSub, &tm_v, bar_kv, sub * 64, kt * kBT, bkv);
      }
      load_stage(0);
    }
  }
  if (warp == kBwdIssuerWarp) {
    tmem_alloc(smem_u32(tmem_slot), kBwdTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == kBwdProducerWarp) {
    if (lane == 0 && n > 0) {
      int issued = 1;
      for (int i = 1; i < n_steps; ++i) {
        if (i >= QS && !wait_bounded(ST_EMPTY(i % QS), ((i / QS) - 1) & 1, abort_flag, p.status)) break;
        load_stage(i);
        issued = i + 1;
      }
      wait_bounded(bar_kv, 0, nullptr, p.status, kBwdDrainNs);
      for (int i = (issued > QS ? issued - QS : 0); i < issued; ++i)
        wait_bounded(ST_FULL(i % QS), (i / QS) & 1, nullptr, p.status, kBwdDrainNs);
    }
    __syncwarp();
  } else if (warp == kBwdIssuerWarp || warp == kBwdDpWarp) {
    if (lane == 0 && n > 0) {
      // Step i in buffer i % 2.  Warp 9: S^T_i = K Q_i^T once step i - 2's dV product (which
      // reads P^T from the same columns) is done.  Warp 11: dP^T_i = V dO_i^T once step i - 2's
      // dK product (dS^T) is done.  Waiting for each product separately lets step i's products
      // start while step i - 2's are still in the pipe, and the two threads' waits overlap
      // each other's issue.
      const bool is_s = (warp == kBwdIssuerWarp);
      constexpr uint32_t idesc_s = make_idesc_f16(BF16, kBT, kStepQ, false);
      const uint64_t a_desc = make_sdesc_sw128(base + (is_s ? L::kK : L::kV), 16, 1024);
      const uint32_t col0 = is_s ? L::kColS : L::kColDP;
      const uint32_t b_off = is_s ? 0u : L::kHalf;  // Q or dO of the stage
      bool ok = wait_bounded(bar_kv, 0, abort_flag, p.status);
      for (int i = 0; ok && i < n_steps; ++i) {
        const int s = i % QS, bb = i & 1;
        if (!wait_bounded(ST_FULL(s), (i / QS) & 1, abort_flag, p.status)) break;
        if (i >= 2 && !wait_bounded(is_s ? P_FREE(bb) : DS_FREE(bb), ((i >> 1) - 1) & 1,
                                    abort_flag, p.status))
          break;
        tc_fence_after();
        const uint32_t st = base + L::kStages + s * L::kStage;
        mma_rows_rows_d<D, kSub, L::kHalfSub>(tmem + col0 + bb * kStepQ, a_desc,
                                               make_sdesc_sw128(st + b_off, 16, 1024), idesc_s);
        mma_commit(is_s ? S_FULL(bb) : DP_FULL(bb));
      }
      // this thread's products are complete before the block ends (after an abort as well)
      const uint32_t drain = is_s ? bar_drain_s : bar_drain_dp;
      mma_commit(drain);
      wait_bounded(drain, 0, nullptr, p.status, kBwdDrainNs);
    }
    __syncwarp();
  } else if (warp == kBwdAccWarp) {
    if (lane == 0 && n > 0) {
      // Once P^T_i is stored: dV += P^T_i dO_i (its commit frees the S^T columns); once dS^T_i
      // is stored: dK += dS^T_i Q_i (its commit frees the dP^T columns and the stage: step i's
      // score products are complete, the elementwise warps waited for them before storing).
      constexpr uint32_t idesc_acc = make_idesc_f16(BF16, kBT, D, true);
      for (int i = 0; i < n_steps; ++i) {
        const int s = i % QS, bb = i & 1;
        const uint32_t st = base + L::kStages + s * L::kStage;
        if (!wait_bounded(P_READY(bb), (i >> 1) & 1, abort_flag, p.status)) break;
        tc_fence_after();
        mma_tmem_rows_d<kStepQ>(tmem + L::kColDV, tmem + L::kColS + bb * kStepQ,
                                make_sdesc_sw128(st + L::kHalf, L::kHalfSub, 1024), idesc_acc,
                                i > 0);  // dV += P^T dO
        mma_commit(P_FREE(bb));
        if (!wait_bounded(DS_READY(bb), (i >> 1) & 1, abort_flag, p.status)) break;
        tc_fence_after();
        mma_tmem_rows_d<kStepQ>(tmem + L::kColDK, tmem + L::kColDP + bb * kStepQ,
                                make_sdesc_sw128(st, L::kHalfSub, 1024), idesc_acc,
                                i > 0);  // dK += dS^T Q
        mma_commit(ST_EMPTY(s));
        mma_commit(DS_FREE(bb));
      }
      mma_commit(bar_drain);
      wait_bounded(bar_drain, 0, nullptr, p.status, kBwdDrainNs);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ elementwise (thread = key)
    // Warpgroup w takes the steps of buffer w; thread r owns key row r (warp % 4 is its
    // tensor-memory lane quarter).
    const int wg = warp >> 2;
    const int quarter = warp & 3;
    const int r = quarter * 32 + lane;
    const int kr = kt * kBT + r;  // this thread's key
    const uint32_t row_tmem = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    if constexpr (!BF16) griddep_wait();  // kernel 0's ranges
    const GradScale gs = grad_scale<BF16>(p, bkv);
    const float sl2 = p.sl2, scale = p.scale * gs.u;
    const int q_first_visible = kr - off;  // the smallest query row that sees this key
    // window variant: the largest
    [[maybe_unused]] int q_last_visible = 0x7fffffff;
    if constexpr (WINDOW) {
      const long long last = static_cast<long long>(kr) - off + p.window;
      if (kr >= p.sinks && last < q_last_visible) q_last_visible = static_cast<int>(last);
    }
    const uint32_t s_col = L::kColS + wg * kStepQ, dp_col = L::kColDP + wg * kStepQ;
    bool ok = true;
    for (int i = wg; i < n_steps; i += 2) {
      const int s = i % QS;
      const int tile = tile0 + (i >> 1);
      const int q0 = (qt_lo + tile % nq_per) * kBT + (i & 1) * kStepQ;
      const float* lv = reinterpret_cast<const float*>(gbase + L::kStages + s * L::kStage +
                                                       2 * L::kHalf);
      const float* dvv = lv + kStepQ;
      if (!ew_wait(S_FULL(wg), (i >> 1) & 1, abort_flag, p.status)) {
        ok = false;
        break;
      }
      tc_fence_after();
      // P^T row of this key over the step's 64 queries, kept in registers for dS^T:
      // p = 2^(s scale log2(e) - L log2(e)), one packed FMA per pair; the causal test only
      // where some query of the 64 precedes this key
      float pv[kStepQ];
      uint32_t pp[kStepQ / 2];
      {
        uint32_t sv[2][32];
        tmem_ld32(row_tmem + s_col, sv[0]);
        tmem_ld32(row_tmem + s_col + 32, sv[1]);
        tmem_wait_ld();
        const bool full =
            WINDOW ? q0 >= q_first_visible && q0 + (kStepQ - 1) <= q_last_visible
                   : !p.causal || q0 >= q_first_visible;
        const bool all_full = __all_sync(0xffffffffu, full);
        if constexpr (WINDOW) {
          if (!all_full) {
            const int lo = max(q_first_visible, 0) - q0, hi = q_last_visible - q0;
            mask32(sv[0], 0, lo, hi, -1);
            mask32(sv[1], 32, lo, hi, -1);
          }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            const int col = h * 32 + e;
            const float4 l4 = *reinterpret_cast<const float4*>(lv + col);
            float a0, a1, a2, a3;
            fma2(a0, a1, __uint_as_float(sv[h][e]), __uint_as_float(sv[h][e + 1]), sl2, sl2, l4.x, l4.y);
            fma2(a2, a3, __uint_as_float(sv[h][e + 2]), __uint_as_float(sv[h][e + 3]), sl2, sl2, l4.z,
                 l4.w);
            if (!WINDOW && !all_full) {
              const int rel = q_first_visible - (q0 + col);  // columns below rel precede the key
              a0 = (0 >= rel) ? a0 : -INFINITY;
              a1 = (1 >= rel) ? a1 : -INFINITY;
              a2 = (2 >= rel) ? a2 : -INFINITY;
              a3 = (3 >= rel) ? a3 : -INFINITY;
            }
            pv[col] = ex2(a0);
            pv[col + 1] = ex2(a1);
            pv[col + 2] = ex2(a2);
            pv[col + 3] = ex2(a3);
            pp[col >> 1] = pack2<BF16>(pv[col], pv[col + 1]);
            pp[(col >> 1) + 1] = pack2<BF16>(pv[col + 2], pv[col + 3]);
          }
      }
      tmem_st32(row_tmem + s_col, pp);  // P^T over the S^T columns already read
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(P_READY(wg));  // dV += P^T dO may start while dS^T is formed
      if (!ew_wait(DP_FULL(wg), (i >> 1) & 1, abort_flag, p.status)) {
        ok = false;
        break;
      }
      tc_fence_after();
      uint32_t dpv[2][32];
      tmem_ld32(row_tmem + dp_col, dpv[0]);
      tmem_ld32(row_tmem + dp_col + 32, dpv[1]);
      tmem_wait_ld();
      // dS^T = P^T o (dP^T - D) scale = P^T o (dP^T scale + (-scale D)): two packed FMAs a pair
      uint32_t dd[kStepQ / 2];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
          const int col = h * 32 + e;
          float4 d4 = *reinterpret_cast<const float4*>(dvv + col);
          if constexpr (!BF16) {
            fma2(d4.x, d4.y, d4.x, d4.y, gs.u, gs.u, 0.0f, 0.0f);
            fma2(d4.z, d4.w, d4.z, d4.w, gs.u, gs.u, 0.0f, 0.0f);
          }
          float u0, u1, u2, u3, g0, g1, g2, g3;
          fma2(u0, u1, __uint_as_float(dpv[h][e]), __uint_as_float(dpv[h][e + 1]), scale, scale, d4.x, d4.y);
          fma2(u2, u3, __uint_as_float(dpv[h][e + 2]), __uint_as_float(dpv[h][e + 3]), scale, scale, d4.z,
               d4.w);
          fma2(g0, g1, pv[col], pv[col + 1], u0, u1, 0.0f, 0.0f);
          fma2(g2, g3, pv[col + 2], pv[col + 3], u2, u3, 0.0f, 0.0f);
          dd[col >> 1] = pack2<BF16>(g0, g1);
          dd[(col >> 1) + 1] = pack2<BF16>(g2, g3);
        }
      tmem_st32(row_tmem + dp_col, dd);  // dS^T over the dP^T columns already read
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(DS_READY(wg));
    }
    // epilogue: warpgroup 0 stores dV, warpgroup 1 dK, once the last MMA has finished
    if (ok && n > 0) ok = ew_wait(bar_drain, 0, abort_flag, p.status);
    if (ok) tc_fence_after();
    const uint32_t col = wg ? L::kColDK : L::kColDV;
    if (partial) {
      const size_t at = ((static_cast<size_t>(bkv) * p.sink_tiles + kt) * p.sink_parts + part) * 2 + wg;
      if (ok) store_part_row<D, BF16>(row_tmem + col, p.part + (at * kBT + r) * D, n > 0, wg ? gs.ds : gs.p);
    } else if (n > 0) {
      // dV over K, dK over V, whose products are done; each warpgroup its own
      const uint32_t tile = wg ? L::kV : L::kK;
      if (ok) stage_acc_row<BF16>(row_tmem + col, gbase + tile, r, 0, D, wg ? gs.ds : gs.p);
      fence_proxy_async_smem();
      named_bar_sync(1 + wg, kEwThreads);
      if (r == 0 && *abort_flag == 0) store_staged<D>(wg ? &tm_dk : &tm_dv, base + tile, kt * kBT, bkv);
    } else if (kr < p.N_kv) {
      store_zero_row<D>((wg ? p.dk : p.dv) + (static_cast<size_t>(bkv) * p.N_kv + kr) * D);
    }
  }
#undef ST_FULL
#undef ST_EMPTY
#undef S_FULL
#undef DP_FULL
#undef P_READY
#undef DS_READY
#undef P_FREE
#undef DS_FREE
  tc_fence_before();
  __syncthreads();
  if (warp == kBwdIssuerWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kBwdTmemCols);
  }
}

// ------------------------------------------------------------------------------------------
// kernel 2: dQ of one 128-row query tile
// ------------------------------------------------------------------------------------------
// Q stays in tensor memory as the A operand of S = Q K^T; dO (shared memory) is that of
// dP = dO V^T.  Tensor memory: Q 0-63, S 64-191, dP 192-319, dS 320-383, dQ 384-.  The two
// elementwise warpgroups split each tile's 128 keys and release S and dP as soon as they have
// read them, and dS has its own buffer, so that the tensor pipe takes, per tile, S_{t+1} and
// dP_{t+1} (issued while tile t's elementwise step runs) and then dQ += dS_t K_t: no product
// waits for another tile's dS.
template <int D, int KR, int VR>
struct QLayout {
  static constexpr uint32_t kTile = kBT * D * 2;
  static constexpr uint32_t kDO = 0;                 // dO tile
  static constexpr uint32_t kK = kTile;              // K ring, KR slots
  static constexpr uint32_t kV = kK + KR * kTile;    // V ring, VR slots
  static constexpr uint32_t kBar = kV + VR * kTile;
  // k_full[KR], k_empty[KR], v_full[VR], v_empty[VR], q_ready, do_full, s_full, s_free,
  // drain of the S issuer, dp_free, ds_ready[2], drain, ds_free[2], drain of the dP issuer;
  // dP written is the V slot's release barrier
  static constexpr uint32_t kNumBars = 2 * KR + 2 * VR + 12;
  static constexpr uint32_t kMisc = kBar + kNumBars * 8;
  static constexpr uint32_t kBytes = kMisc + 16 + 1024;
  static constexpr uint32_t kColQ = 0, kColS = 64, kColDP = 192, kColDS = 320, kColDQ = 384;
  static_assert(kBytes <= 232448, "shared memory per block");
};

// Half h of A [128 x 128] B: A in tensor memory as 16-bit pairs (64 columns), B [128 rows x D]
// in shared memory read MN-major; the product over A's columns and B's rows 64h .. 64h + 63:
// D[128 x D] (+)= A[:, 64h:64h+64] B[64h:64h+64, :].
__device__ __forceinline__ void mma_tmem_kt_half(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_smem,
                                                 uint32_t idesc, int h, bool accumulate) {
  const uint64_t b_desc = make_sdesc_sw128(b_smem, kSub, 1024);
#pragma unroll
  for (int k4 = 0; k4 < kBT / 32; ++k4) {
    const int kk = h * (kBT / 32) + k4;
    mma_ts(d_tmem, a_tmem + kk * 8, b_desc + ((kk * 16 * 128) >> 4), idesc,
           (accumulate || k4 > 0) ? 1u : 0u);
  }
}

// A [128 x D] in tensor memory as 16-bit pairs (D / 2 columns) times B^T, B [128 rows x D]
// K-major in shared memory (64-column sub-tiles kSub apart): D[128 x 128] = A B^T.
template <int D>
__device__ __forceinline__ void mma_tmem_rows_t(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_smem,
                                                uint32_t idesc) {
  const uint64_t b_desc = make_sdesc_sw128(b_smem, 16, 1024);
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk)
    mma_ts(d_tmem, a_tmem + kk * 8, b_desc + (((kk >> 2) * kSub + (kk & 3) * 32) >> 4), idesc,
           kk > 0 ? 1u : 0u);
}

// One row of a contiguous 16-bit [rows, D] tensor as D / 2 32-bit words (zeros for a row past
// the end), and those words into tensor memory, thread = lane row: two elements a column with
// the lower-indexed one in the low half (the A operand layout of tcgen05.mma kind::f16).  The
// load is issued before the block's setup, the store after it, so that the setup hides the
// load's latency.
template <int D>
__device__ __forceinline__ void row_load(const uint16_t* src, bool valid, uint4 (&w)[D / 8]) {
#pragma unroll
  for (int i = 0; i < D / 8; ++i)
    w[i] = valid ? reinterpret_cast<const uint4*>(src)[i] : make_uint4(0, 0, 0, 0);
}

template <int D>
__device__ __forceinline__ void row_to_tmem(uint32_t taddr, const uint4 (&w)[D / 8]) {
#pragma unroll
  for (int c = 0; c < D / 64; ++c) {
    uint32_t v[32];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[4 * i] = w[c * 8 + i].x;
      v[4 * i + 1] = w[c * 8 + i].y;
      v[4 * i + 2] = w[c * 8 + i].z;
      v[4 * i + 3] = w[c * 8 + i].w;
    }
    tmem_st32(taddr + c * 32, v);
  }
}

template <int D, bool BF16, int KR, int VR, bool WINDOW>
__global__ void __launch_bounds__(kQThreads, 1)
    attn_bwd_dq_kernel(const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v,
                       const __grid_constant__ CUtensorMap tm_do,
                       const __grid_constant__ CUtensorMap tm_dq, const BwdParams p) {
  using L = QLayout<D, KR, VR>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  const uint32_t bars = base + L::kBar;
#define K_FULL(s) (bars + 8u * (s))
#define K_EMPTY(s) (bars + 8u * (KR + (s)))
#define V_FULL(s) (bars + 8u * (2 * KR + (s)))
#define V_EMPTY(s) (bars + 8u * (2 * KR + VR + (s)))
  const uint32_t bar_q = bars + 8u * (2 * KR + 2 * VR);  // Q rows in tensor memory (128)
  const uint32_t bar_do = bar_q + 8;         // dO tile landed (TMA)
  const uint32_t bar_sfull = bar_q + 16;     // S_t written (MMA commit)
  const uint32_t bar_sfree = bar_q + 24;     // S_t read (256 arrivals)
  const uint32_t bar_drain_s = bar_q + 32;   // S issuer's products done (commit)
  const uint32_t bar_drain_dp = bar_q + 88;  // dP issuer's products done (commit)
  const uint32_t bar_dpfree = bar_q + 40;    // dP_t read (256 arrivals)
#define DS_READY(w) (bar_q + 48 + 8u * (w))       // warpgroup w's half of dS_t stored (128)
#define DS_FREE(w) (bar_q + 72 + 8u * (w))        // dQ's product over that half done (commit)
  const uint32_t bar_drain = bar_q + 64;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + L::kMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(gbase + L::kMisc + 4);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  // item: query tile qt of (batch, query head) bh.  Query-tile major, last tile first: under
  // the causal mask the longest items of every head start first and the grid ends on one-tile
  // items; the heads of one key/value head run side by side and share its K/V tiles in L2.
  const int n_bh = static_cast<int>(gridDim.x) / p.n_qtiles;
  const int qt = p.n_qtiles - 1 - static_cast<int>(blockIdx.x) / n_bh;
  const int bh = static_cast<int>(blockIdx.x) % n_bh;
  const int kv_plane = (bh / p.Hq) * p.Hkv + (bh % p.Hq) / p.G;
  int n, first_masked;
  // window variant: the key tiles that hold sinks, then those of the window
  [[maybe_unused]] int j_begin = 0, lo_masked = 0, sink_tiles = 0;
  if constexpr (WINDOW) {
    int j_end;
    kv_tile_span(qt, kBT, kBT, p.N_q, p.N_kv, 1, p.window, j_begin, j_end, lo_masked, first_masked);
    sink_tiles = min((p.sinks + kBT - 1) / kBT, j_begin);
    n = sink_tiles + j_end - j_begin;
  } else {
    kv_tile_range(qt, kBT, kBT, p.N_q, p.N_kv, p.causal, n, first_masked);
  }
  auto key_tile = [&](int t) {  // key tile of step t
    if constexpr (WINDOW) return t < sink_tiles ? t : j_begin + t - sink_tiles;
    return t;
  };
  // warpgroup 0 (thread = query row) starts loading the tile's Q rows now
  uint4 q_row[D / 8];
  if (n > 0 && threadIdx.x < kEwThreads) {
    const int qr = qt * kBT + static_cast<int>(threadIdx.x);
    row_load<D>(p.q + (static_cast<size_t>(bh) * p.N_q + (qr < p.N_q ? qr : 0)) * D, qr < p.N_q,
                q_row);
  }

  auto load_k = [&](int t) {
    mbar_arrive_expect_tx(K_FULL(t % KR), L::kTile);
#pragma unroll
    for (int sub = 0; sub < D / 64; ++sub)
      tma_load_3d(base + L::kK + (t % KR) * L::kTile + sub * kSub, &tm_k, K_FULL(t % KR), sub * 64,
                  key_tile(t) * kBT, kv_plane);
  };
  auto load_v = [&](int t) {
    mbar_arrive_expect_tx(V_FULL(t % VR), L::kTile);
#pragma unroll
    for (int sub = 0; sub < D / 64; ++sub)
      tma_load_3d(base + L::kV + (t % VR) * L::kTile + sub * kSub, &tm_v, V_FULL(t % VR), sub * 64,
                  key_tile(t) * kBT, kv_plane);
  };
  if (warp == kBwdProducerWarp && lane == 0) {
    for (int s = 0; s < KR; ++s) {
      mbar_init(K_FULL(s), 1);
      mbar_init(K_EMPTY(s), 1);
    }
    for (int s = 0; s < VR; ++s) {
      mbar_init(V_FULL(s), 1);
      mbar_init(V_EMPTY(s), 1);
    }
    mbar_init(bar_q, kEwThreads);
    mbar_init(bar_do, 1);
    mbar_init(bar_sfull, 1);
    mbar_init(bar_sfree, 2 * kEwThreads);
    mbar_init(bar_dpfree, 2 * kEwThreads);
    for (int w = 0; w < 2; ++w) {
      mbar_init(DS_READY(w), kEwThreads);
      mbar_init(DS_FREE(w), 1);
    }
    mbar_init(bar_drain, 1);
    mbar_init(bar_drain_s, 1);
    mbar_init(bar_drain_dp, 1);
    *abort_flag = 0;
    fence_barrier_init();
    // the first loads go out before the block's setup is done
    if (n > 0) {
      load_k(0);
      mbar_arrive_expect_tx(bar_do, L::kTile);
#pragma unroll
      for (int sub = 0; sub < D / 64; ++sub)
        tma_load_3d(base + L::kDO + sub * kSub, &tm_do, bar_do, sub * 64, qt * kBT, bh);
      load_v(0);
    }
  }
  if (warp == kBwdIssuerWarp) {
    tmem_alloc(smem_u32(tmem_slot), kBwdTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == kBwdProducerWarp) {
    if (lane == 0 && n > 0) {
      int issued_k = 1, issued_v = 1;
      for (int t = 1; t < n; ++t) {
        if (t >= KR && !wait_bounded(K_EMPTY(t % KR), ((t / KR) - 1) & 1, abort_flag, p.status)) break;
        load_k(t);
        issued_k = t + 1;
        if (t >= VR && !wait_bounded(V_EMPTY(t % VR), ((t / VR) - 1) & 1, abort_flag, p.status)) break;
        load_v(t);
        issued_v = t + 1;
      }
      wait_bounded(bar_do, 0, nullptr, p.status, kBwdDrainNs);
      for (int t = (issued_k > KR ? issued_k - KR : 0); t < issued_k; ++t)
        wait_bounded(K_FULL(t % KR), (t / KR) & 1, nullptr, p.status, kBwdDrainNs);
      for (int t = (issued_v > VR ? issued_v - VR : 0); t < issued_v; ++t)
        wait_bounded(V_FULL(t % VR), (t / VR) & 1, nullptr, p.status, kBwdDrainNs);
    }
    __syncwarp();
  } else if (warp == kBwdIssuerWarp) {
    if (lane == 0 && n > 0) {
      // S_t = Q K_t^T once S_{t-1} has been read
      constexpr uint32_t idesc_rr = make_idesc_f16(BF16, kBT, kBT, false);
      bool ok = wait_bounded(bar_q, 0, abort_flag, p.status);
      for (int t = 0; ok && t < n; ++t) {
        const int sk = t % KR;
        if (t > 0 && !wait_bounded(bar_sfree, (t - 1) & 1, abort_flag, p.status)) break;
        if (!wait_bounded(K_FULL(sk), (t / KR) & 1, abort_flag, p.status)) break;
        tc_fence_after();
        mma_tmem_rows_t<D>(tmem + L::kColS, tmem + L::kColQ, base + L::kK + sk * L::kTile, idesc_rr);
        mma_commit(bar_sfull);
      }
      // this thread's products are complete before the block ends (after an abort as well)
      mma_commit(bar_drain_s);
      wait_bounded(bar_drain_s, 0, nullptr, p.status, kBwdDrainNs);
    }
    __syncwarp();
  } else if (warp == kBwdDpWarp) {
    if (lane == 0 && n > 0) {
      // dP_t = dO V_t^T once dP_{t-1} has been read
      constexpr uint32_t idesc_rr = make_idesc_f16(BF16, kBT, kBT, false);
      const uint64_t do_desc = make_sdesc_sw128(base + L::kDO, 16, 1024);
      bool ok = wait_bounded(bar_do, 0, abort_flag, p.status);
      for (int t = 0; ok && t < n; ++t) {
        const int sv = t % VR;
        if (t > 0 && !wait_bounded(bar_dpfree, (t - 1) & 1, abort_flag, p.status)) break;
        if (!wait_bounded(V_FULL(sv), (t / VR) & 1, abort_flag, p.status)) break;
        tc_fence_after();
        mma_rows_rows_d<D, kSub, kSub>(tmem + L::kColDP, do_desc,
                                       make_sdesc_sw128(base + L::kV + sv * L::kTile, 16, 1024),
                                       idesc_rr);
        // one commit for both readers: the elementwise warps (dP_t written) and the producer
        // (V slot free) wait on the V slot's barrier
        mma_commit(V_EMPTY(sv));
      }
      mma_commit(bar_drain_dp);
      wait_bounded(bar_drain_dp, 0, nullptr, p.status, kBwdDrainNs);
    }
    __syncwarp();
  } else if (warp == kBwdAccWarp) {
    if (lane == 0 && n > 0) {
      // dQ += dS_t K_t in two halves over the keys, each once its warpgroup has stored its
      // half of dS_t; each half's commit frees that half of the dS buffer.  After both, the K
      // slot is free (S_t, read by the elementwise warps before they stored dS_t, is complete).
      constexpr uint32_t idesc_q = make_idesc_f16(BF16, kBT, D, true);
      bool ok = true;
      for (int t = 0; ok && t < n; ++t) {
        const uint32_t kslot = base + L::kK + (t % KR) * L::kTile;
        for (int w = 0; w < 2; ++w) {
          if (!wait_bounded(DS_READY(w), t & 1, abort_flag, p.status)) {
            ok = false;
            break;
          }
          tc_fence_after();
          mma_tmem_kt_half(tmem + L::kColDQ, tmem + L::kColDS, kslot, idesc_q, w,
                           t > 0 || w > 0);  // dQ += dS K over keys 64w .. 64w + 63
          mma_commit(DS_FREE(w));
        }
        if (ok) mma_commit(K_EMPTY(t % KR));
      }
      mma_commit(bar_drain);
      wait_bounded(bar_drain, 0, nullptr, p.status, kBwdDrainNs);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ elementwise (thread = query)
    // Warpgroup w takes keys c0 = 64w .. c0+63 of every key tile; thread r owns query row r.
    const int wg = warp >> 2;
    const int c0 = wg * 64;
    const int quarter = warp & 3;
    const int r = quarter * 32 + lane;
    const int row = qt * kBT + r;
    const uint32_t row_tmem = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const size_t vec = static_cast<size_t>(bh) * p.nqp + row;
    const GradScale gs = grad_scale<BF16>(p, kv_plane);
    const float nl2 = p.lse2[vec];         // -L log2(e)
    const float nsd = p.dvec[vec] * gs.u;  // -scale D
    const float sl2 = p.sl2, scale = p.scale * gs.u;
    int lim = p.causal ? row + (p.N_kv - p.N_q) : p.N_kv - 1;  // last visible key of this row
    if (lim > p.N_kv - 1) lim = p.N_kv - 1;
    [[maybe_unused]] int first_key = 0;  // first key of this row's window
    if constexpr (WINDOW) {
      const long long lo = static_cast<long long>(row) + (p.N_kv - p.N_q) - p.window;
      first_key = static_cast<int>(lo > 0 ? lo : 0);
    }
    bool ok = true;
    if (n > 0 && wg == 0) {
      // warpgroup 0 writes the Q rows it loaded before the setup
      row_to_tmem<D>(row_tmem + L::kColQ, q_row);
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(bar_q);
    }
    const uint32_t s_col = L::kColS + c0, dp_col = L::kColDP + c0, ds_col = L::kColDS + wg * 32;
    for (int t = 0; t < n; ++t) {
      const int j = key_tile(t);
      const bool masked = WINDOW ? j >= first_masked || j < lo_masked : j >= first_masked;
      const int rel = lim - (j * kBT + c0);  // last visible key, relative to this half tile
      if (!ew_wait(bar_sfull, t & 1, abort_flag, p.status)) {
        ok = false;
        break;
      }
      tc_fence_after();
      uint32_t sv[2][32];
      tmem_ld32(row_tmem + s_col, sv[0]);
      tmem_ld32(row_tmem + s_col + 32, sv[1]);
      tmem_wait_ld();
      tc_fence_before();
      mbar_arrive(bar_sfree);  // S_{t+1} may overwrite
      if constexpr (WINDOW) {
        if (masked) {
          // the first key of the window and the last sink, relative to this half tile
          const int lo = max(first_key - (j * kBT + c0), 0);
          const int sk = min(p.sinks - 1 - (j * kBT + c0), rel);
          mask32(sv[0], 0, lo, rel, sk);
          mask32(sv[1], 32, lo, rel, sk);
        }
      }
      // p = 2^(s scale log2(e) - L log2(e)), one packed FMA a pair; the mask only on the tiles
      // that need it (the same for every row of the tile)
      float pv[64];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          const int col = h * 32 + e;
          float a0, a1;
          fma2(a0, a1, __uint_as_float(sv[h][e]), __uint_as_float(sv[h][e + 1]), sl2, sl2, nl2, nl2);
          if (!WINDOW && masked) {
            a0 = (col <= rel) ? a0 : -INFINITY;
            a1 = (col + 1 <= rel) ? a1 : -INFINITY;
          }
          pv[col] = ex2(a0);
          pv[col + 1] = ex2(a1);
        }
      // dP_t written: the commit that also frees V slot t % VR (its (t / VR)-th phase); the
      // next phase needs dP_{t+VR}, which waits for this warpgroup's read of dP_{t+VR-1}
      if (!ew_wait(V_EMPTY(t % VR), (t / VR) & 1, abort_flag, p.status)) {
        ok = false;
        break;
      }
      tc_fence_after();
      uint32_t dpv[2][32];
      tmem_ld32(row_tmem + dp_col, dpv[0]);
      tmem_ld32(row_tmem + dp_col + 32, dpv[1]);
      tmem_wait_ld();
      tc_fence_before();
      mbar_arrive(bar_dpfree);  // dP_{t+1} may overwrite
      // dS = P o (dP scale + (-scale D)): two packed FMAs a pair
      uint32_t dd[32];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          const int col = h * 32 + e;
          float u0, u1, g0, g1;
          fma2(u0, u1, __uint_as_float(dpv[h][e]), __uint_as_float(dpv[h][e + 1]), scale, scale, nsd, nsd);
          fma2(g0, g1, pv[col], pv[col + 1], u0, u1, 0.0f, 0.0f);
          dd[col >> 1] = pack2<BF16>(g0, g1);
        }
      // this warpgroup's half of the dS buffer: free once dQ's product over it for tile t - 1
      // has finished
      if (t > 0 && !ew_wait(DS_FREE(wg), (t - 1) & 1, abort_flag, p.status)) {
        ok = false;
        break;
      }
      tc_fence_after();
      tmem_st32(row_tmem + ds_col, dd);  // keys c0 .. c0+63 as 16-bit pairs
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(DS_READY(wg));
    }
    if (ok && n > 0) ok = ew_wait(bar_drain, 0, abort_flag, p.status);
    if (n > 0) {
      // over dO, whose products are done; each warpgroup half of the columns
      if (ok) {
        tc_fence_after();
        stage_acc_row<BF16>(row_tmem + L::kColDQ, gbase + L::kDO, quarter * 32 + lane, wg * (D / 2),
                            (wg + 1) * (D / 2), gs.ds);
      }
      fence_proxy_async_smem();
      named_bar_sync(1, 2 * kEwThreads);
      if (threadIdx.x == 0 && *abort_flag == 0)
        store_staged<D>(&tm_dq, base + L::kDO, qt * kBT, bh);
    } else if (wg == 0 && row < p.N_q) {
      store_zero_row<D>(p.dq + (static_cast<size_t>(bh) * p.N_q + row) * D);
    }
  }
#undef K_FULL
#undef K_EMPTY
#undef V_FULL
#undef V_EMPTY
#undef DS_READY
#undef DS_FREE
  tc_fence_before();
  __syncthreads();
  if (warp == kBwdIssuerWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kBwdTmemCols);
  }
  // This grid may have started while the dK/dV kernel was still running; no block of it
  // finishes before that kernel has, so that whatever follows on the stream sees dK and dV
  // complete.
  if (threadIdx.x == 0) griddep_wait();
}

// ------------------------------------------------------------------------------------------
// kernel 3 (window variant): dK and dV of the key tiles with sinks from their blocks' partial sums,
// added in block order.  Four values a thread; grid (elements, key tile of a plane, dV or dK).
// ------------------------------------------------------------------------------------------
template <int D, bool BF16>
__global__ void __launch_bounds__(256) attn_bwd_sink_sum_kernel(const BwdParams p) {
  griddep_wait();
  const int e = (blockIdx.x * 256 + threadIdx.x) * 4;
  const int r = e / D, c = e % D;
  const int bkv = blockIdx.y / p.sink_tiles, kt = blockIdx.y % p.sink_tiles;
  const int which = blockIdx.z;
  const int key = kt * kBT + r;
  if (key >= p.N_kv) return;
  const float* src = p.part + (static_cast<size_t>(blockIdx.y) * p.sink_parts * 2 + which) * kBT * D + e;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i = 0; i < p.sink_parts; ++i) {
    const float4 v = *reinterpret_cast<const float4*>(src + static_cast<size_t>(i) * 2 * kBT * D);
    s.x += v.x;
    s.y += v.y;
    s.z += v.z;
    s.w += v.w;
  }
  uint16_t* dst = (which ? p.dk : p.dv) + (static_cast<size_t>(bkv) * p.N_kv + key) * D + c;
  *reinterpret_cast<uint2*>(dst) = make_uint2(pack2<BF16>(s.x, s.y), pack2<BF16>(s.z, s.w));
}

// ------------------------------------------------------------------------------------------
// launcher
// ------------------------------------------------------------------------------------------
size_t bwd_workspace_bytes(int B, int Hq, int N_q) {
  if (B <= 0 || Hq <= 0 || N_q <= 0) return 0;
  const size_t nqp = (static_cast<size_t>(N_q) + kBT - 1) / kBT * kBT;
  // L log2(e) and D, fp32; four words of ranges a plane (at most one a query head)
  return static_cast<size_t>(B) * Hq * (nqp * 8 + 16);
}

// 64-query steps of the dK/dV job for key tile kt (as the kernel counts them).
static int kv_job_steps(int kt, int n_qtiles, int G, int causal, int off, int window, int sinks) {
  int qt_lo = 0;
  if (window >= 0) {
    int qt_hi;
    window_q_tiles(kt, n_qtiles, off, window, sinks, qt_lo, qt_hi);
    return 2 * G * (qt_hi - qt_lo);
  }
  if (causal) {
    const int first_row = kt * kBT - off;
    qt_lo = first_row > 0 ? first_row / kBT : 0;
  }
  const int nq_per = n_qtiles - qt_lo;
  return nq_per > 0 ? 2 * G * nq_per : 0;
}

// How the key tiles with sinks are cut (window variant): into parts of at most half an SM's share
// of all steps, and 32 steps at least.
static void sink_split(int n_planes, int n_kvtiles, int n_qtiles, int G, int off, int window,
                       int sinks, int& tiles, int& parts) {
  constexpr int kSms = 152;
  tiles = static_cast<int>(std::min<long long>((static_cast<long long>(sinks) + kBT - 1) / kBT, n_kvtiles));
  parts = 1;
  if (tiles == 0) return;
  long long total = 0, longest = 0;
  for (int kt = 0; kt < n_kvtiles; ++kt) {
    const long long w = kv_job_steps(kt, n_qtiles, G, 1, off, window, sinks);
    total += w * n_planes;
    if (kt < tiles) longest = std::max(longest, w);
  }
  const long long target = std::max<long long>(total / (2 * kSms), 32);
  parts = static_cast<int>(std::min<long long>((longest + target - 1) / target, 32));
  if (parts < 1) parts = 1;
}

// Floats of the partial sums.
static size_t sink_part_floats(size_t n_planes, int tiles, int parts, int d) {
  return parts > 1 ? n_planes * tiles * parts * 2 * kBT * static_cast<size_t>(d) : 0;
}

size_t bwd_window_workspace_bytes(int B, int Hq, int Hkv, int N_q, int N_kv, int d, int window,
                                  int sinks) {
  const size_t base = bwd_workspace_bytes(B, Hq, N_q);
  if (base == 0 || N_kv <= 0) return base;
  int tiles, parts;
  sink_split(B * Hkv, (N_kv + kBT - 1) / kBT, (N_q + kBT - 1) / kBT, Hq / Hkv, N_kv - N_q, window,
             sinks, tiles, parts);
  return base + sink_part_floats(static_cast<size_t>(B) * Hkv, tiles, parts, d) * 4;
}

// The packed dispatch order for a grid of n_planes x n_kvtiles jobs on n_sm SMs: writes the job
// of every block to job[0 .. n) and returns n, or 0 when the default order stands (no causal
// mask: equal jobs; no more jobs than SMs; more than `cap` jobs).
int bwd_kv_order(int n_planes, int n_kvtiles, int n_qtiles, int G, int causal, int off, int window,
                 int sinks, int n_sm, uint16_t* job, int cap) {
  int sink_tiles = 0, sink_parts = 1;
  if (window >= 0)
    sink_split(n_planes, n_kvtiles, n_qtiles, G, off, window, sinks, sink_tiles, sink_parts);
  const int n_sink = n_planes * sink_tiles;  // jobs cut into sink_parts blocks, numbered first
  const long long n_jobs_ll = static_cast<long long>(n_planes) * n_kvtiles +
                              static_cast<long long>(n_sink) * (sink_parts - 1);
  if (!causal || n_sm <= 0 || n_jobs_ll <= n_sm || n_jobs_ll > cap || n_jobs_ll > 65536) return 0;
  const int n_jobs = static_cast<int>(n_jobs_ll);
  // job weights: its steps plus a block's fixed cost (about four steps: setup, K/V load,
  // pipeline fill, dK/dV store)
  std::vector<long long> w(n_jobs);
  long long total = 0;
  for (int j = 0; j < n_jobs; ++j) {
    const bool cut = j < n_sink * sink_parts;
    const int kt = (cut ? j % n_sink : j - n_sink * (sink_parts - 1)) / n_planes;
    w[j] = kv_job_steps(kt, n_qtiles, G, causal, off, window, sinks) / (cut ? sink_parts : 1) + 4;
    total += w[j];
  }
  std::vector<int> by_size(n_jobs);
  for (int j = 0; j < n_jobs; ++j) by_size[j] = j;
  std::stable_sort(by_size.begin(), by_size.end(), [&](int x, int y) { return w[x] > w[y]; });
  // best fit under a cap a little above the average load; of a few caps, the plan whose
  // fullest bin is lowest
  const long long avg = (total + n_sm - 1) / n_sm;
  std::vector<std::vector<int>> bins;
  long long best_max = -1;
  for (int step = 0; step <= 12; ++step) {
    const long long bin_cap = avg + avg * step / 400;  // up to 3% above the average
    std::vector<std::vector<int>> trial(n_sm);
    std::vector<long long> load(n_sm, 0);
    for (int j : by_size) {
      int best = -1, emptiest = 0;
      for (int b = 0; b < n_sm; ++b) {
        if (load[b] + w[j] <= bin_cap && (best < 0 || load[b] > load[best])) best = b;
        if (load[b] < load[emptiest]) emptiest = b;
      }
      const int b = best >= 0 ? best : emptiest;
      trial[b].push_back(j);  // largest first within a bin
      load[b] += w[j];
    }
    const long long mx = *std::max_element(load.begin(), load.end());
    if (best_max < 0 || mx < best_max) {
      best_max = mx;
      bins.swap(trial);
    }
  }
  // the order in which SMs that free up in turn take the bins' jobs
  int n = 0;
  using Slot = std::pair<long long, int>;  // (time the SM frees up, bin)
  std::priority_queue<Slot, std::vector<Slot>, std::greater<Slot>> free_at;
  std::vector<size_t> next(n_sm, 0);
  for (int b = 0; b < n_sm; ++b) free_at.push({0, b});
  while (!free_at.empty()) {
    const Slot sl = free_at.top();
    free_at.pop();
    const int b = sl.second;
    if (next[b] < bins[b].size()) {
      const int j = bins[b][next[b]++];
      job[n++] = static_cast<uint16_t>(j);
      free_at.push({sl.first + w[j], b});
    }
  }
  return n == n_jobs ? n : 0;
}

// The packed dispatch order (KvOrder) for one shape on the current device.  Packing takes a few
// milliseconds, so the orders of the last kKeptOrders shapes are kept (4 KB each; a shape in the default
// order needs none).
constexpr size_t kKeptOrders = 512;

static void kv_order(int n_planes, int n_kvtiles, int n_qtiles, int G, int causal, int off, int window,
                     int sinks, KvOrder& order) {
  order.n = 0;
  int dev = 0, n_sm = 0;
  if (!causal || cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&n_sm, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return;
  using Key = std::tuple<int, int, int, int, int, int, int, int>;
  struct Kept {
    KvOrder order;
    std::list<Key>::iterator at;
  };
  static std::map<Key, Kept> cache;
  static std::list<Key> used;  // last used first
  static std::mutex mu;
  const Key key{n_planes, n_kvtiles, n_qtiles, G, off, window, sinks, n_sm};
  try {
    {
      std::lock_guard<std::mutex> lock(mu);
      auto it = cache.find(key);
      if (it != cache.end()) {
        used.splice(used.begin(), used, it->second.at);
        order = it->second.order;
        return;
      }
    }
    order.n = bwd_kv_order(n_planes, n_kvtiles, n_qtiles, G, causal, off, window, sinks, n_sm, order.job,
                           kMaxKvOrder);
    if (order.n == 0) return;
    std::lock_guard<std::mutex> lock(mu);
    if (cache.count(key)) return;  // another thread has packed it meanwhile
    while (cache.size() >= kKeptOrders) {
      cache.erase(used.back());
      used.pop_back();
    }
    used.push_front(key);
    try {
      cache.emplace(key, Kept{order, used.begin()});
    } catch (...) {
      used.pop_front();
      throw;
    }
  } catch (...) {  // out of host memory: the default order, or this one unkept, serves
  }
}

template <int D, bool BF16, bool WINDOW>
static int launch_bwd_variant(const BwdArgs& a, cudaStream_t stream) {
  constexpr int QS = (D == 128) ? 4 : 6;  // 64-query stages of the dK/dV kernel
  constexpr int KR = (D == 128) ? 3 : 6;  // K slots of the dQ kernel
  constexpr int VR = (D == 128) ? 3 : 6;  // V slots of the dQ kernel (dO takes one tile too)
  using LK = KvLayout<D, QS>;
  using LQ = QLayout<D, KR, VR>;
  const uint64_t bhq = static_cast<uint64_t>(a.B) * a.Hq;
  const uint64_t bhk = static_cast<uint64_t>(a.B) * a.Hkv;
  const uint64_t rb = static_cast<uint64_t>(D) * 2;
  CUtensorMap tk, tv, tdo;
  CUtensorMap tq64, tdo64;  // 64-row boxes: the stages of the dK/dV kernel
  if (!make_tmap_3d(&tq64, a.q, BF16, D, a.N_q, bhq, rb, rb * a.N_q, 64, kStepQ, 1) ||
      !make_tmap_3d(&tdo64, a.dout, BF16, D, a.N_q, bhq, rb, rb * a.N_q, 64, kStepQ, 1))
    return -5;
  if (!make_tmap_3d(&tdo, a.dout, BF16, D, a.N_q, bhq, rb, rb * a.N_q, 64, kBT, 1) ||
      !make_tmap_3d(&tk, a.k, BF16, D, a.N_kv, bhk, rb, rb * a.N_kv, 64, kBT, 1) ||
      !make_tmap_3d(&tv, a.v, BF16, D, a.N_kv, bhk, rb, rb * a.N_kv, 64, kBT, 1))
    return -5;
  CUtensorMap tdq, tdk, tdv;
  if (!make_tmap_3d(&tdq, a.dq, BF16, D, a.N_q, bhq, rb, rb * a.N_q, 64, kBT, 1) ||
      !make_tmap_3d(&tdk, a.dk, BF16, D, a.N_kv, bhk, rb, rb * a.N_kv, 64, kBT, 1) ||
      !make_tmap_3d(&tdv, a.dv, BF16, D, a.N_kv, bhk, rb, rb * a.N_kv, 64, kBT, 1))
    return -5;
  BwdParams p;
  const int n_qtiles = (a.N_q + kBT - 1) / kBT;
  const int nqp = n_qtiles * kBT;
  p.lse2 = static_cast<const float*>(a.workspace);
  p.dvec = p.lse2 + bhq * nqp;
  p.q = static_cast<const uint16_t*>(a.q);
  p.k = static_cast<const uint16_t*>(a.k);
  p.v = static_cast<const uint16_t*>(a.v);
  p.dout = static_cast<const uint16_t*>(a.dout);
  p.dq = static_cast<uint16_t*>(a.dq);
  p.dk = static_cast<uint16_t*>(a.dk);
  p.dv = static_cast<uint16_t*>(a.dv);
  p.status = device_status_ptr();
  if (!p.status) return -5;
  p.Hq = a.Hq;
  p.Hkv = a.Hkv;
  p.G = a.Hq / a.Hkv;
  p.N_q = a.N_q;
  p.N_kv = a.N_kv;
  p.n_qtiles = n_qtiles;
  p.n_kvtiles = (a.N_kv + kBT - 1) / kBT;
  p.nqp = nqp;
  p.causal = a.causal;
  p.scale = a.scale;
  p.sl2 = a.scale * 1.4426950408889634f;
  p.window = a.window;
  p.sinks = a.sinks;
  p.sink_tiles = 0;
  p.sink_parts = 1;
  p.part = nullptr;
  if constexpr (WINDOW) {
    sink_split(static_cast<int>(bhk), p.n_kvtiles, n_qtiles, p.G, a.N_kv - a.N_q, a.window, a.sinks,
               p.sink_tiles, p.sink_parts);
    p.part = const_cast<float*>(p.lse2) + bhq * (2 * static_cast<uint64_t>(nqp) + 4);
  }
  uint32_t* range = reinterpret_cast<uint32_t*>(const_cast<float*>(p.lse2) + 2 * bhq * nqp);
  p.range = range;
  const long long rows = static_cast<long long>(bhq) * nqp;
  const unsigned pre_blocks = static_cast<unsigned>((rows / kPreRows * (D / 8) + 255) / 256);
  unsigned v_blocks = 0;
  if (!BF16) {
    constexpr int kRows = 256 / (D / 8) * kPreRows;
    v_blocks = static_cast<unsigned>(bhk * ((a.N_kv + kRows - 1) / kRows));
    if (cudaMemsetAsync(range, 0, bhk * 16, stream) != cudaSuccess) return -5;
  }
  attn_bwd_pre_kernel<D, BF16><<<pre_blocks + v_blocks, 256, 0, stream>>>(
      static_cast<const uint16_t*>(a.o), static_cast<const uint16_t*>(a.dout), p.v, a.lse,
      const_cast<float*>(p.lse2), const_cast<float*>(p.dvec), range, a.N_q, nqp, a.N_kv, a.Hq, a.Hkv, rows,
      pre_blocks, a.scale);
  if (cudaGetLastError() != cudaSuccess) return -5;
  // two blocks on an SM (attn_bwd_window.cu) for either kernel
  const bool kv_two = WINDOW && D == 64 && bwd_window_two_kv(a), q_two = WINDOW && D == 64 && bwd_window_two_q(a);
  auto kkv = attn_bwd_dkdv_kernel<D, BF16, QS, WINDOW>;
  auto kq = attn_bwd_dq_kernel<D, BF16, KR, VR, WINDOW>;
  if (cudaFuncSetAttribute(kkv, cudaFuncAttributeMaxDynamicSharedMemorySize, LK::kBytes) != cudaSuccess ||
      cudaFuncSetAttribute(kq, cudaFuncAttributeMaxDynamicSharedMemorySize, LQ::kBytes) != cudaSuccess)
    return -5;
  const uint64_t kv_blocks =
      bhk * (static_cast<uint64_t>(p.n_kvtiles) + static_cast<uint64_t>(p.sink_tiles) * (p.sink_parts - 1));
  const uint64_t q_blocks = bhq * n_qtiles;
  if (kv_blocks > 0x7fffffffull || q_blocks > 0x7fffffffull) return -2;
  // dK/dV as a programmatic dependent of kernel 0 (its setup and first loads under that kernel's end),
  // dQ as one of dK/dV.
  cudaLaunchConfig_t cfg = {};
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (kv_two) {
    const int st = launch_bwd_window_dkdv(a, p, static_cast<unsigned>(kv_blocks), stream);
    if (st != 0) return st;
  } else {
    KvOrder order;
    kv_order(static_cast<int>(bhk), p.n_kvtiles, n_qtiles, p.G, a.causal, a.N_kv - a.N_q, a.window, a.sinks,
             order);
    cfg.gridDim = dim3(static_cast<unsigned>(kv_blocks));
    cfg.blockDim = dim3(kKvThreads);
    cfg.dynamicSmemBytes = LK::kBytes;
    if (cudaLaunchKernelEx(&cfg, kkv, tq64, tk, tv, tdo64, tdk, tdv, p, order) != cudaSuccess) return -5;
  }
  // dQ's blocks fill the SMs of dK/dV's tail.
  cfg.gridDim = dim3(static_cast<unsigned>(q_blocks));
  cfg.blockDim = dim3(kQThreads);
  cfg.dynamicSmemBytes = LQ::kBytes;
  if (q_two) {
    const int st = launch_bwd_window_dq(a, p, static_cast<unsigned>(q_blocks), stream);
    if (st != 0) return st;
  } else if (cudaLaunchKernelEx(&cfg, kq, tk, tv, tdo, tdq, p) != cudaSuccess) {
    return -5;
  }
  if constexpr (WINDOW) {
    if (p.sink_parts > 1) {
      // a dependent of dQ, whose blocks end after the dK/dV kernel has (more than 65,535 tiles are
      // never cut: together they are over 100 times an SM's share)
      cfg.gridDim = dim3(kBT * D / 1024, static_cast<unsigned>(bhk * p.sink_tiles), 2);
      cfg.blockDim = dim3(256);
      cfg.dynamicSmemBytes = 0;
      if (cudaLaunchKernelEx(&cfg, attn_bwd_sink_sum_kernel<D, BF16>, p) != cudaSuccess) return -5;
    }
  }
  return cudaGetLastError() == cudaSuccess ? 0 : -5;
}

int launch_attn_bwd(const BwdArgs& a, cudaStream_t stream) {
  const bool w = a.window >= 0;
  if (a.d == 64) {
    if (a.bf16)
      return w ? launch_bwd_variant<64, true, true>(a, stream)
               : launch_bwd_variant<64, true, false>(a, stream);
    return w ? launch_bwd_variant<64, false, true>(a, stream)
             : launch_bwd_variant<64, false, false>(a, stream);
  }
  if (a.d == 128) {
    if (a.bf16)
      return w ? launch_bwd_variant<128, true, true>(a, stream)
               : launch_bwd_variant<128, true, false>(a, stream);
    return w ? launch_bwd_variant<128, false, true>(a, stream)
             : launch_bwd_variant<128, false, false>(a, stream);
  }
  return -2;
}

}  // namespace attn
