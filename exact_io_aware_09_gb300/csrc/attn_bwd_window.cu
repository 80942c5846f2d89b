// Backward under a sliding window (with or without sinks) whose tiles see few others, d = 64: the two
// gradient kernels of attn_bwd.cu with two blocks on an SM.
//
// A tile of a short window runs a handful of steps, so a block's start and end (tensor-memory
// allocation, first loads, first products, the gradients' way out) cost as much as its steps; with one
// block on an SM nothing covers them.  Here a block holds half of what an SM has: 256 tensor-memory
// columns, about 105 KB of shared memory, 224 threads of up to 128 registers, so that one block's
// start and end, and its waits, lie under the other's steps.  At d = 128 the two accumulators of dK and
// dV alone fill the 256 columns, and Q, dO and two steps of K and V the shared memory.
//
// Both kernels step through 64 rows of the other side, one elementwise warpgroup (thread = row of the
// block's own tile) and two issuing threads.  Roles (224 threads): warps 0-3 elementwise and epilogue,
// warp 4 TMA producer, warps 5 and 6 tcgen05 issuers (warp 5 owns the tensor memory).  Every wait on a barrier is
// bounded.
//
// Roundings as in attn_bwd.cu: P and dS to the operands' type (in fp16 times powers of two), everything
// else fp32.
//
// Bound by a step's chain of products and elementwise work at two blocks an SM (tensor pipe 25% busy,
// 1.4 instructions a cycle).  B=8 H=12 N=1024 bf16, W=256, 4 sinks: dK/dV 37 us, dQ 26.5 (one block an
// SM: 48 and 43).  Steps that count there: the gradients through shared memory and TMA 43 -> 40 and 30 ->
// 28; dQ's scores in a buffer of their own, and a thread each for the two pairs of products 39 -> 37 and
// 27.5 -> 26.5.  Tried for dK/dV and slower: P^T and dS^T in shared memory, which frees the scores early
// but leaves two stages for Q and dO (46 us against 40); S^T in two halves of 32 queries (46 against 39).
#include "attn_bwd.cuh"

namespace attn {

namespace {

constexpr int kBwThreads = 224;
constexpr int kBwD = 64;
constexpr uint32_t kBwTmemCols = 256;
constexpr uint32_t kBwTile = kBT * kBwD * 2;     // 128 rows
constexpr uint32_t kBwStep = kStepQ * kBwD * 2;  // 64 rows

// dK/dV: K, V and a ring of 64-query stages (Q, dO, their L log2(e) and D).  Tensor memory: S^T 0-63,
// dP^T 64-127, dV 128-191, dK 192-255; P^T and dS^T as 16-bit pairs over the first half of the columns
// they came from.
struct KvShort {
  static constexpr int kQS = 4;
  static constexpr uint32_t kStage = (2 * kBwStep + 512 + 1023) / 1024 * 1024;
  static constexpr uint32_t kK = 0, kV = kBwTile, kStages = 2 * kBwTile;
  static constexpr uint32_t kBar = kStages + kQS * kStage;
  // kv_full, st_full[QS], st_empty[QS], s_full, dp_full, p_ready, ds_ready, p_free, ds_free,
  // drains of the two issuers
  static constexpr uint32_t kNumBars = 1 + 2 * kQS + 8;
  static constexpr uint32_t kMisc = kBar + kNumBars * 8;
  static constexpr uint32_t kBytes = kMisc + 16 + 1024;  // + alignment
  static constexpr uint32_t kColS = 0, kColDP = 64, kColDV = 128, kColDK = 192;
  static_assert(2 * (kBytes + 1024) <= 233472, "two blocks on an SM");
};

// dQ: Q, dO and rings of 64-key K and V steps.  Tensor memory: S 0-63, dS[2] 64-127 (16-bit pairs), dP
// 128-191, dQ 192-255.
struct QShort {
  static constexpr int kKS = 5, kVS = 4;
  static constexpr uint32_t kQ = 0, kDO = kBwTile, kK = 2 * kBwTile, kV = kK + kKS * kBwStep;
  static constexpr uint32_t kBar = kV + kVS * kBwStep;
  // q and dO, k_full[KS], k_empty[KS], v_full[VS], v_empty[VS], s_full, s_free, ds_ready[2],
  // dq_done[2], dp_full, dp_free, drains of the two issuers
  static constexpr uint32_t kNumBars = 1 + 2 * kKS + 2 * kVS + 10;
  static constexpr uint32_t kMisc = kBar + kNumBars * 8;
  static constexpr uint32_t kBytes = kMisc + 16 + 1024;
  static constexpr uint32_t kColS = 0, kColDS = 64, kColDP = 128, kColDQ = 192;
  static_assert(2 * (kBytes + 1024) <= 233472, "two blocks on an SM");
};

// A [128 x 64] times B^T, B [64 x 64], both K-major: [128 x 64].
__device__ __forceinline__ void mma_scores(uint32_t d_tmem, uint32_t a_smem, uint32_t b_smem,
                                           uint32_t idesc) {
  mma_rows_rows_d<kBwD, kBwTile, kBwStep>(d_tmem, make_sdesc_sw128(a_smem, 16, 1024),
                                          make_sdesc_sw128(b_smem, 16, 1024), idesc);
}

// A [128 x 64] in tensor memory as 16-bit pairs times B [64 rows x 64]: [128 x 64] (+)=.
__device__ __forceinline__ void mma_grad(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_smem,
                                         uint32_t idesc, bool accumulate) {
  mma_tmem_rows_d<kStepQ>(d_tmem, a_tmem, make_sdesc_sw128(b_smem, kBwStep, 1024), idesc, accumulate);
}

}  // namespace

template <bool BF16>
__global__ void __launch_bounds__(kBwThreads, 2)
    attn_bwd_short_dkdv_kernel(const __grid_constant__ CUtensorMap tm_q,
                               const __grid_constant__ CUtensorMap tm_k,
                               const __grid_constant__ CUtensorMap tm_v,
                               const __grid_constant__ CUtensorMap tm_do,
                               const __grid_constant__ CUtensorMap tm_dk,
                               const __grid_constant__ CUtensorMap tm_dv, const BwdParams p) {
  using L = KvShort;
  constexpr int QS = L::kQS;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  const uint32_t bar_kv = base + L::kBar;
#define ST_FULL(s) (bar_kv + 8u * (1 + (s)))
#define ST_EMPTY(s) (bar_kv + 8u * (1 + QS + (s)))
  const uint32_t bar_b = bar_kv + 8u * (1 + 2 * QS);
  const uint32_t bar_s = bar_b;             // S^T written (MMA commit)
  const uint32_t bar_dp = bar_b + 8u;       // dP^T written
  const uint32_t bar_p = bar_b + 16u;       // P^T stored (128 arrivals)
  const uint32_t bar_ds = bar_b + 24u;      // dS^T stored (128)
  const uint32_t bar_pfree = bar_b + 32u;   // dV product done: S^T columns free
  const uint32_t bar_dsfree = bar_b + 40u;  // dK product done: dP^T columns free
  const uint32_t bar_drain = bar_b + 48u, bar_drain2 = bar_b + 56u;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + L::kMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(gbase + L::kMisc + 4);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    griddep_wait();  // (dQ reads kernel 0's vectors too)
    griddep_launch_dependents();  // dQ needs nothing of this kernel
  }

  // job: key tile kt of (batch, key/value head) bkv, key tile major; the tiles with sinks come first,
  // cut into sink_parts blocks each (part major)
  const int n_planes =
      static_cast<int>(gridDim.x) / (p.n_kvtiles + p.sink_tiles * (p.sink_parts - 1));
  const int n_sink = n_planes * p.sink_tiles;
  int job = static_cast<int>(blockIdx.x), part = 0;
  if (job < n_sink * p.sink_parts) {
    part = job / n_sink;
    job -= part * n_sink;
  } else {
    job -= n_sink * (p.sink_parts - 1);
  }
  const int kt = job / n_planes;
  const int bkv = job % n_planes;
  const int bhq0 = (bkv / p.Hkv) * p.Hq + (bkv % p.Hkv) * p.G;  // first of the group's query heads
  const int off = p.N_kv - p.N_q;
  int st_lo, st_hi;  // 64-query steps of a query head that see the tile
  {
    const long long first = static_cast<long long>(kt) * kBT - off;
    const long long last = first + (kBT - 1) + p.window;
    const int n_all = (p.N_q + kStepQ - 1) / kStepQ;
    st_lo = first > 0 ? static_cast<int>(first / kStepQ < n_all ? first / kStepQ : n_all) : 0;
    long long hi = last >= 0 ? last / kStepQ + 1 : 0;
    if (kt * kBT < p.sinks || hi > n_all) hi = n_all;
    st_hi = hi > st_lo ? static_cast<int>(hi) : st_lo;
  }
  const int per_head = st_hi - st_lo;
  int n = p.G * per_head, step0 = 0;
  const bool partial = kt < p.sink_tiles && p.sink_parts > 1;
  if (partial) {
    step0 = static_cast<int>(static_cast<long long>(n) * part / p.sink_parts);
    n = static_cast<int>(static_cast<long long>(n) * (part + 1) / p.sink_parts) - step0;
  }
  auto load_stage = [&](int i) {
    const int s = i % QS;
    const int g = (step0 + i) / per_head;
    const int q0 = (st_lo + (step0 + i) - g * per_head) * kStepQ;
    const uint32_t st = base + L::kStages + s * L::kStage;
    mbar_arrive_expect_tx(ST_FULL(s), 2 * kBwStep + 512);
    tma_load_3d(st, &tm_q, ST_FULL(s), 0, q0, bhq0 + g);
    tma_load_3d(st + kBwStep, &tm_do, ST_FULL(s), 0, q0, bhq0 + g);
    if (i == 0) griddep_wait();  // kernel 0's vectors
    const size_t vec = static_cast<size_t>(bhq0 + g) * p.nqp + static_cast<size_t>(q0);
    bulk_load(st + 2 * kBwStep, p.lse2 + vec, kStepQ * 4, ST_FULL(s));
    bulk_load(st + 2 * kBwStep + 256, p.dvec + vec, kStepQ * 4, ST_FULL(s));
  };

  if (warp == 4 && lane == 0) {
    prefetch_tmap(&tm_q);
    prefetch_tmap(&tm_k);
    prefetch_tmap(&tm_v);
    prefetch_tmap(&tm_do);
    mbar_init(bar_kv, 1);
    for (int s = 0; s < QS; ++s) {
      mbar_init(ST_FULL(s), 1);
      mbar_init(ST_EMPTY(s), 2);
    }
    mbar_init(bar_s, 1);
    mbar_init(bar_dp, 1);
    mbar_init(bar_p, kBT);
    mbar_init(bar_ds, kBT);
    mbar_init(bar_pfree, 1);
    mbar_init(bar_dsfree, 1);
    mbar_init(bar_drain, 1);
    mbar_init(bar_drain2, 1);
    *abort_flag = 0;
    fence_barrier_init();
    // the first loads go out before the block's setup is done
    if (n > 0) {
      mbar_arrive_expect_tx(bar_kv, 2 * kBwTile);
      tma_load_3d(base + L::kK, &tm_k, bar_kv, 0, kt * kBT, bkv);
      tma_load_3d(base + L::kV, &tm_v, bar_kv, 0, kt * kBT, bkv);
      load_stage(0);
    }
  }
  if (warp == 5) {
    tmem_alloc(smem_u32(tmem_slot), kBwTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 4) {
    // ----------------------------------------------------------------- TMA producer
    if (lane == 0 && n > 0) {
      int issued = 1;
      for (int i = 1; i < n; ++i) {
        if (i >= QS && !wait_bounded(ST_EMPTY(i % QS), ((i / QS) - 1) & 1, abort_flag, p.status)) break;
        load_stage(i);
        issued = i + 1;
      }
      // Every asynchronous write into this block's shared memory lands before it may exit.
      wait_bounded(bar_kv, 0, nullptr, p.status, kBwdDrainNs);
      for (int i = (issued > QS ? issued - QS : 0); i < issued; ++i)
        wait_bounded(ST_FULL(i % QS), (i / QS) & 1, nullptr, p.status, kBwdDrainNs);
    }
    __syncwarp();
  } else if (warp == 5) {
    // ------------------------------------------ tcgen05 issuer of S^T = K Q^T and dV += P^T dO
    if (lane == 0 && n > 0) {
      constexpr uint32_t idesc_s = make_idesc_f16(BF16, kBT, kStepQ, false);
      constexpr uint32_t idesc_g = make_idesc_f16(BF16, kBT, kBwD, true);
      auto stage = [&](int i) { return base + L::kStages + (i % QS) * L::kStage; };
      if (wait_bounded(bar_kv, 0, abort_flag, p.status)) {
        for (int i = 0; i < n; ++i) {
          if (!wait_bounded(ST_FULL(i % QS), (i / QS) & 1, abort_flag, p.status)) break;
          // S^T_i goes over P^T_{i-1}, once the product that reads it is done
          if (i > 0 && !wait_bounded(bar_pfree, (i - 1) & 1, abort_flag, p.status)) break;
          tc_fence_after();
          mma_scores(tmem + L::kColS, base + L::kK, stage(i), idesc_s);
          mma_commit(bar_s);
          if (!wait_bounded(bar_p, i & 1, abort_flag, p.status)) break;
          tc_fence_after();
          mma_grad(tmem + L::kColDV, tmem + L::kColS, stage(i) + kBwStep, idesc_g, i > 0);
          mma_commit(bar_pfree);
          mma_commit(ST_EMPTY(i % QS));
        }
      }
      // every MMA this thread issued completes before the block frees its tensor memory
      mma_commit(bar_drain);
      wait_bounded(bar_drain, 0, nullptr, p.status, kBwdDrainNs);
    }
    __syncwarp();
  } else if (warp == 6) {
    // ------------------------------------------ tcgen05 issuer of dP^T = V dO^T and dK += dS^T Q
    if (lane == 0 && n > 0) {
      constexpr uint32_t idesc_s = make_idesc_f16(BF16, kBT, kStepQ, false);
      constexpr uint32_t idesc_g = make_idesc_f16(BF16, kBT, kBwD, true);
      auto stage = [&](int i) { return base + L::kStages + (i % QS) * L::kStage; };
      if (wait_bounded(bar_kv, 0, abort_flag, p.status)) {
        for (int i = 0; i < n; ++i) {
          if (!wait_bounded(ST_FULL(i % QS), (i / QS) & 1, abort_flag, p.status)) break;
          if (i > 0 && !wait_bounded(bar_dsfree, (i - 1) & 1, abort_flag, p.status)) break;
          tc_fence_after();
          mma_scores(tmem + L::kColDP, base + L::kV, stage(i) + kBwStep, idesc_s);
          mma_commit(bar_dp);
          if (!wait_bounded(bar_ds, i & 1, abort_flag, p.status)) break;
          tc_fence_after();
          mma_grad(tmem + L::kColDK, tmem + L::kColDP, stage(i), idesc_g, i > 0);
          mma_commit(bar_dsfree);
          mma_commit(ST_EMPTY(i % QS));
        }
      }
      mma_commit(bar_drain2);
      wait_bounded(bar_drain2, 0, nullptr, p.status, kBwdDrainNs);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ elementwise (thread = key)
    const int r = warp * 32 + lane;
    const int kr = kt * kBT + r;
    const uint32_t row_tmem = tmem + (static_cast<uint32_t>(warp * 32) << 16);
    if constexpr (!BF16) griddep_wait();  // kernel 0's ranges
    const GradScale gs = grad_scale<BF16>(p, bkv);
    const float sl2 = p.sl2, scale = p.scale * gs.u;
    // the query rows [q_first, q_last] see this key
    const int q_first = kr - off;
    int q_last = 0x7fffffff;
    {
      const long long last = static_cast<long long>(kr) - off + p.window;
      if (kr >= p.sinks && last < q_last) q_last = static_cast<int>(last);
    }
    int st = per_head > 0 ? st_lo + step0 % per_head : 0;  // 64-query step of the head
    bool ok = true;
    for (int i = 0; i < n; ++i) {
      const int q0 = st * kStepQ;
      if (++st == st_hi) st = st_lo;
      const float* lv = reinterpret_cast<const float*>(gbase + L::kStages + (i % QS) * L::kStage +
                                                       2 * kBwStep);
      if (!ew_wait(bar_s, i & 1, abort_flag, p.status)) {
        ok = false;
        break;
      }
      tc_fence_after();
      // p = 2^(s scale log2(e) - L log2(e)), kept in registers for dS
      uint32_t sv[2][32];
      tmem_ld32(row_tmem + L::kColS, sv[0]);
      tmem_ld32(row_tmem + L::kColS + 32, sv[1]);
      tmem_wait_ld();
      if (!__all_sync(0xffffffffu, q0 >= q_first && q0 + (kStepQ - 1) <= q_last)) {
        const int lo = max(q_first, 0) - q0, hi = q_last - q0;
        mask32(sv[0], 0, lo, hi, -1);
        mask32(sv[1], 32, lo, hi, -1);
      }
      uint32_t w[32];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
          const float4 l4 = *reinterpret_cast<const float4*>(lv + h * 32 + e);
          float a0, a1, a2, a3;
          fma2(a0, a1, __uint_as_float(sv[h][e]), __uint_as_float(sv[h][e + 1]), sl2, sl2, l4.x, l4.y);
          fma2(a2, a3, __uint_as_float(sv[h][e + 2]), __uint_as_float(sv[h][e + 3]), sl2, sl2, l4.z,
               l4.w);
          a0 = ex2(a0);
          a1 = ex2(a1);
          a2 = ex2(a2);
          a3 = ex2(a3);
          w[(h * 32 + e) >> 1] = pack2<BF16>(a0, a1);
          w[((h * 32 + e) >> 1) + 1] = pack2<BF16>(a2, a3);
          sv[h][e] = __float_as_uint(a0);
          sv[h][e + 1] = __float_as_uint(a1);
          sv[h][e + 2] = __float_as_uint(a2);
          sv[h][e + 3] = __float_as_uint(a3);
        }
      tmem_st32(row_tmem + L::kColS, w);
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(bar_p);  // dV += P^T dO may start while dS^T is formed
      if (!ew_wait(bar_dp, i & 1, abort_flag, p.status)) {
        ok = false;
        break;
      }
      tc_fence_after();
      // dS^T = P^T o (dP^T scale + (-scale D))
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t dpv[32];
        tmem_ld32(row_tmem + L::kColDP + h * 32, dpv);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
          float4 d4 = *reinterpret_cast<const float4*>(lv + kStepQ + h * 32 + e);
          if constexpr (!BF16) {
            fma2(d4.x, d4.y, d4.x, d4.y, gs.u, gs.u, 0.0f, 0.0f);
            fma2(d4.z, d4.w, d4.z, d4.w, gs.u, gs.u, 0.0f, 0.0f);
          }
          float u0, u1, u2, u3, g0, g1, g2, g3;
          fma2(u0, u1, __uint_as_float(dpv[e]), __uint_as_float(dpv[e + 1]), scale, scale, d4.x, d4.y);
          fma2(u2, u3, __uint_as_float(dpv[e + 2]), __uint_as_float(dpv[e + 3]), scale, scale, d4.z, d4.w);
          fma2(g0, g1, __uint_as_float(sv[h][e]), __uint_as_float(sv[h][e + 1]), u0, u1, 0.0f, 0.0f);
          fma2(g2, g3, __uint_as_float(sv[h][e + 2]), __uint_as_float(sv[h][e + 3]), u2, u3, 0.0f, 0.0f);
          w[(h * 32 + e) >> 1] = pack2<BF16>(g0, g1);
          w[((h * 32 + e) >> 1) + 1] = pack2<BF16>(g2, g3);
        }
      }
      tmem_st32(row_tmem + L::kColDP, w);
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(bar_ds);
    }
    if (ok && n > 0)
      ok = ew_wait(bar_drain, 0, abort_flag, p.status) && ew_wait(bar_drain2, 0, abort_flag, p.status);
    if (ok) tc_fence_after();
    if (partial) {
      const size_t at = ((static_cast<size_t>(bkv) * p.sink_tiles + kt) * p.sink_parts + part) * 2;
      if (ok) {
        store_part_row<kBwD, BF16>(row_tmem + L::kColDV, p.part + (at * kBT + r) * kBwD, n > 0, gs.p);
        store_part_row<kBwD, BF16>(row_tmem + L::kColDK, p.part + ((at + 1) * kBT + r) * kBwD, n > 0, gs.ds);
      }
    } else if (n > 0) {
      // over K and V, whose products are done
      if (ok) {
        stage_acc_row<BF16>(row_tmem + L::kColDV, gbase + L::kK, r, 0, kBwD, gs.p);
        stage_acc_row<BF16>(row_tmem + L::kColDK, gbase + L::kV, r, 0, kBwD, gs.ds);
      }
      fence_proxy_async_smem();
      named_bar_sync(1, kBT);
      if (threadIdx.x == 0 && *abort_flag == 0) {
        store_staged<kBwD>(&tm_dv, base + L::kK, kt * kBT, bkv);
        store_staged<kBwD>(&tm_dk, base + L::kV, kt * kBT, bkv);
      }
    } else if (kr < p.N_kv) {
      const size_t row = (static_cast<size_t>(bkv) * p.N_kv + kr) * kBwD;
      store_zero_row<kBwD>(p.dv + row);
      store_zero_row<kBwD>(p.dk + row);
    }
  }
#undef ST_FULL
#undef ST_EMPTY
  tc_fence_before();
  __syncthreads();
  if (warp == 5) {
    tc_fence_after();
    tmem_dealloc(tmem, kBwTmemCols);
  }
}

template <bool BF16>
__global__ void __launch_bounds__(kBwThreads, 2)
    attn_bwd_short_dq_kernel(const __grid_constant__ CUtensorMap tm_q,
                             const __grid_constant__ CUtensorMap tm_k,
                             const __grid_constant__ CUtensorMap tm_v,
                             const __grid_constant__ CUtensorMap tm_do,
                             const __grid_constant__ CUtensorMap tm_dq, const BwdParams p) {
  using L = QShort;
  constexpr int KS = L::kKS, VS = L::kVS;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  const uint32_t bar_q = base + L::kBar;  // Q and dO
#define K_FULL(s) (bar_q + 8u * (1 + (s)))
#define K_EMPTY(s) (bar_q + 8u * (1 + KS + (s)))
#define V_FULL(s) (bar_q + 8u * (1 + 2 * KS + (s)))
#define V_EMPTY(s) (bar_q + 8u * (1 + 2 * KS + VS + (s)))
  const uint32_t bar_b = bar_q + 8u * (1 + 2 * KS + 2 * VS);
  const uint32_t bar_s = bar_b;           // S_t written (MMA commit)
  const uint32_t bar_sfree = bar_b + 8u;  // S_t read (128 arrivals)
#define DS_READY(b) (bar_b + 8u * (2 + (b)))  // dS_t stored (128 arrivals)
#define DQ_DONE(b) (bar_b + 8u * (4 + (b)))   // dQ += dS_t K_t done: dS buffer free
  const uint32_t bar_dp = bar_b + 48u;      // dP_t written
  const uint32_t bar_dpfree = bar_b + 56u;  // dP_t read (128 arrivals)
  const uint32_t bar_drain = bar_b + 64u, bar_drain2 = bar_b + 72u;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + L::kMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(gbase + L::kMisc + 4);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  // item: query tile qt of (batch, query head) bh; 64-key steps: those with sinks, then the window's
  const int n_bh = static_cast<int>(gridDim.x) / p.n_qtiles;
  const int qt = p.n_qtiles - 1 - static_cast<int>(blockIdx.x) / n_bh;
  const int bh = static_cast<int>(blockIdx.x) % n_bh;
  const int kv_plane = (bh / p.Hq) * p.Hkv + (bh % p.Hq) / p.G;
  int j_begin, j_end, lo_masked, hi_masked;
  kv_tile_span(qt, kBT, kStepQ, p.N_q, p.N_kv, 1, p.window, j_begin, j_end, lo_masked, hi_masked);
  const int sink_steps = min((p.sinks + kStepQ - 1) / kStepQ, j_begin);
  const int n = sink_steps + j_end - j_begin;
  auto key_step = [&](int t) { return t < sink_steps ? t : j_begin + t - sink_steps; };
  auto load_k = [&](int t) {
    mbar_arrive_expect_tx(K_FULL(t % KS), kBwStep);
    tma_load_3d(base + L::kK + (t % KS) * kBwStep, &tm_k, K_FULL(t % KS), 0, key_step(t) * kStepQ, kv_plane);
  };
  auto load_v = [&](int t) {
    mbar_arrive_expect_tx(V_FULL(t % VS), kBwStep);
    tma_load_3d(base + L::kV + (t % VS) * kBwStep, &tm_v, V_FULL(t % VS), 0, key_step(t) * kStepQ, kv_plane);
  };

  if (warp == 4 && lane == 0) {
    prefetch_tmap(&tm_q);
    prefetch_tmap(&tm_k);
    prefetch_tmap(&tm_v);
    prefetch_tmap(&tm_do);
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
      mbar_init(DS_READY(b), kBT);
      mbar_init(DQ_DONE(b), 1);
    }
    mbar_init(bar_s, 1);
    mbar_init(bar_sfree, kBT);
    mbar_init(bar_dp, 1);
    mbar_init(bar_dpfree, kBT);
    mbar_init(bar_drain, 1);
    mbar_init(bar_drain2, 1);
    *abort_flag = 0;
    fence_barrier_init();
    // the first loads go out before the block's setup is done
    if (n > 0) {
      mbar_arrive_expect_tx(bar_q, 2 * kBwTile);
      tma_load_3d(base + L::kQ, &tm_q, bar_q, 0, qt * kBT, bh);
      load_k(0);
      tma_load_3d(base + L::kDO, &tm_do, bar_q, 0, qt * kBT, bh);
      load_v(0);
    }
  }
  if (warp == 5) {
    tmem_alloc(smem_u32(tmem_slot), kBwTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 4) {
    // ----------------------------------------------------------------- TMA producer
    if (lane == 0 && n > 0) {
      int issued_k = 1, issued_v = 1;
      for (int t = 1; t < n; ++t) {
        if (t >= KS && !wait_bounded(K_EMPTY(t % KS), ((t / KS) - 1) & 1, abort_flag, p.status)) break;
        load_k(t);
        issued_k = t + 1;
        if (t >= VS && !wait_bounded(V_EMPTY(t % VS), ((t / VS) - 1) & 1, abort_flag, p.status)) break;
        load_v(t);
        issued_v = t + 1;
      }
      // Every asynchronous write into this block's shared memory lands before it may exit.
      wait_bounded(bar_q, 0, nullptr, p.status, kBwdDrainNs);
      for (int t = (issued_k > KS ? issued_k - KS : 0); t < issued_k; ++t)
        wait_bounded(K_FULL(t % KS), (t / KS) & 1, nullptr, p.status, kBwdDrainNs);
      for (int t = (issued_v > VS ? issued_v - VS : 0); t < issued_v; ++t)
        wait_bounded(V_FULL(t % VS), (t / VS) & 1, nullptr, p.status, kBwdDrainNs);
    }
    __syncwarp();
  } else if (warp == 5) {
    // ------------------------------------------ tcgen05 issuer of S = Q K^T and dQ += dS K
    if (lane == 0 && n > 0) {
      constexpr uint32_t idesc_s = make_idesc_f16(BF16, kBT, kStepQ, false);
      constexpr uint32_t idesc_g = make_idesc_f16(BF16, kBT, kBwD, true);
      auto issue_s = [&](int t) -> bool {
        if (!wait_bounded(K_FULL(t % KS), (t / KS) & 1, abort_flag, p.status)) return false;
        tc_fence_after();
        mma_scores(tmem + L::kColS, base + L::kQ, base + L::kK + (t % KS) * kBwStep, idesc_s);
        mma_commit(bar_s);
        return true;
      };
      bool ok = wait_bounded(bar_q, 0, abort_flag, p.status) && issue_s(0);
      for (int t = 0; ok && t < n; ++t) {
        const int b = t & 1;
        if (t + 1 < n) {  // the next step's scores as soon as this step's have been read
          if (!wait_bounded(bar_sfree, t & 1, abort_flag, p.status)) break;
          if (!issue_s(t + 1)) break;
        }
        if (!wait_bounded(DS_READY(b), (t >> 1) & 1, abort_flag, p.status)) break;
        tc_fence_after();
        mma_grad(tmem + L::kColDQ, tmem + L::kColDS + b * (kStepQ / 2), base + L::kK + (t % KS) * kBwStep,
                 idesc_g, t > 0);
        mma_commit(K_EMPTY(t % KS));
        mma_commit(DQ_DONE(b));
      }
      // every MMA this thread issued completes before the block frees its tensor memory
      mma_commit(bar_drain);
      wait_bounded(bar_drain, 0, nullptr, p.status, kBwdDrainNs);
    }
    __syncwarp();
  } else if (warp == 6) {
    // ------------------------------------------ tcgen05 issuer of dP = dO V^T
    if (lane == 0 && n > 0) {
      constexpr uint32_t idesc_s = make_idesc_f16(BF16, kBT, kStepQ, false);
      if (wait_bounded(bar_q, 0, abort_flag, p.status)) {
        for (int t = 0; t < n; ++t) {
          if (!wait_bounded(V_FULL(t % VS), (t / VS) & 1, abort_flag, p.status)) break;
          if (t > 0 && !wait_bounded(bar_dpfree, (t - 1) & 1, abort_flag, p.status)) break;
          tc_fence_after();
          mma_scores(tmem + L::kColDP, base + L::kDO, base + L::kV + (t % VS) * kBwStep, idesc_s);
          mma_commit(bar_dp);
          mma_commit(V_EMPTY(t % VS));
        }
      }
      mma_commit(bar_drain2);
      wait_bounded(bar_drain2, 0, nullptr, p.status, kBwdDrainNs);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ elementwise (thread = query)
    const int r = warp * 32 + lane;
    const int row = qt * kBT + r;
    const uint32_t row_tmem = tmem + (static_cast<uint32_t>(warp * 32) << 16);
    const GradScale gs = grad_scale<BF16>(p, kv_plane);
    const float sl2 = p.sl2, scale = p.scale * gs.u;
    const size_t vec = static_cast<size_t>(bh) * p.nqp + row;
    const float nl2 = p.lse2[vec], nd = p.dvec[vec] * gs.u;
    const int pos = row + (p.N_kv - p.N_q);
    const int lim = min(pos, p.N_kv - 1);          // last visible key
    const int first_key = max(pos - p.window, 0);  // first key of the window
    bool ok = true;
    for (int t = 0; t < n; ++t) {
      const int j = key_step(t);
      const int b = t & 1;
      if (!ew_wait(bar_s, t & 1, abort_flag, p.status)) {
        ok = false;
        break;
      }
      tc_fence_after();
      uint32_t sv[2][32];
      tmem_ld32(row_tmem + L::kColS, sv[0]);
      tmem_ld32(row_tmem + L::kColS + 32, sv[1]);
      tmem_wait_ld();
      tc_fence_before();
      mbar_arrive(bar_sfree);
      if (j >= hi_masked || j < lo_masked) {
        const int hi = lim - j * kStepQ;
        const int lo = max(first_key - j * kStepQ, 0);
        const int sk = min(p.sinks - 1 - j * kStepQ, hi);
        mask32(sv[0], 0, lo, hi, sk);
        mask32(sv[1], 32, lo, hi, sk);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          float a0, a1;
          fma2(a0, a1, __uint_as_float(sv[h][e]), __uint_as_float(sv[h][e + 1]), sl2, sl2, nl2, nl2);
          sv[h][e] = __float_as_uint(ex2(a0));
          sv[h][e + 1] = __float_as_uint(ex2(a1));
        }
      if (!ew_wait(bar_dp, t & 1, abort_flag, p.status)) {
        ok = false;
        break;
      }
      tc_fence_after();
      uint32_t w[32];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t dpv[32];
        tmem_ld32(row_tmem + L::kColDP + h * 32, dpv);
        tmem_wait_ld();
        if (h == 1) {
          tc_fence_before();
          mbar_arrive(bar_dpfree);  // dP_{t+1} may overwrite
        }
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          float u0, u1, g0, g1;
          fma2(u0, u1, __uint_as_float(dpv[e]), __uint_as_float(dpv[e + 1]), scale, scale, nd, nd);
          fma2(g0, g1, __uint_as_float(sv[h][e]), __uint_as_float(sv[h][e + 1]), u0, u1, 0.0f, 0.0f);
          w[(h * 32 + e) >> 1] = pack2<BF16>(g0, g1);
        }
      }
      if (t > 1) {  // dQ's product of step t - 2 read this buffer
        if (!ew_wait(DQ_DONE(b), ((t - 2) >> 1) & 1, abort_flag, p.status)) {
          ok = false;
          break;
        }
        tc_fence_after();
      }
      tmem_st32(row_tmem + L::kColDS + b * (kStepQ / 2), w);
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(DS_READY(b));
    }
    if (n > 0) {
      if (ok) ok = ew_wait(DQ_DONE((n - 1) & 1), ((n - 1) >> 1) & 1, abort_flag, p.status);
      if (ok) {
        tc_fence_after();
        // over Q, whose products are done
        stage_acc_row<BF16>(row_tmem + L::kColDQ, gbase + L::kQ, r, 0, kBwD, gs.ds);
      }
      fence_proxy_async_smem();
      named_bar_sync(1, kBT);
      if (threadIdx.x == 0 && *abort_flag == 0) store_staged<kBwD>(&tm_dq, base + L::kQ, qt * kBT, bh);
    } else if (row < p.N_q) {
      store_zero_row<kBwD>(p.dq + (static_cast<size_t>(bh) * p.N_q + row) * kBwD);
    }
  }
#undef K_FULL
#undef K_EMPTY
#undef V_FULL
#undef V_EMPTY
#undef DS_READY
#undef DQ_DONE
  tc_fence_before();
  __syncthreads();
  if (warp == 5) {
    tc_fence_after();
    tmem_dealloc(tmem, kBwTmemCols);
  }
  // no block ends before the dK/dV kernel has, so that what follows on the stream sees dK and dV
  if (threadIdx.x == 0) griddep_wait();
}

// Tensor maps of Q and dO with boxes of q_rows rows, of K and V with boxes of k_rows.
static bool short_maps(const BwdArgs& a, uint32_t q_rows, uint32_t k_rows, CUtensorMap (&m)[4]) {
  const uint64_t bhq = static_cast<uint64_t>(a.B) * a.Hq, bhk = static_cast<uint64_t>(a.B) * a.Hkv;
  const uint64_t rb = kBwD * 2;
  return make_tmap_3d(&m[0], a.q, a.bf16, kBwD, a.N_q, bhq, rb, rb * a.N_q, 64, q_rows, 1) &&
         make_tmap_3d(&m[1], a.k, a.bf16, kBwD, a.N_kv, bhk, rb, rb * a.N_kv, 64, k_rows, 1) &&
         make_tmap_3d(&m[2], a.v, a.bf16, kBwD, a.N_kv, bhk, rb, rb * a.N_kv, 64, k_rows, 1) &&
         make_tmap_3d(&m[3], a.dout, a.bf16, kBwD, a.N_q, bhq, rb, rb * a.N_q, 64, q_rows, 1);
}

// dK/dV with one / two blocks an SM, us of all three gradient kernels (bf16, 4 sinks; dQ with two):
//   many key tiles, few steps   B=8 H=12 N=1024 (768 tiles): W=64 60 / 52, 256 69 / 61, 1023 81 / 73;
//                               B=8 H=8 N=2048 (1,024) W=256 95 / 83, 2047 155 / 147; B=1 H=32 N=8192
//                               (2,048) W=2048 483 / 472
//   more steps                  B=1 H=32 N=8192 W=4095 (67 a tile) 715 / 720; B=1 Hq=32 Hkv=8 N=16384
//                               W=1024 (76) 598 / 623; B=1 Hq=16 Hkv=4 N=8192 W=4096 (268) 359 / 431
//   fewer tiles                 B=4 H=12 N=1024 (384) W=256 36 / 38; B=4 H=8 N=2048 (512) W=256 49 / 61;
//                               B=1 H=12 N=1024 (96) 18 / 26
// A step here takes longer than there: it pays where starts and ends are many and both blocks of every
// SM stay busy, from about five tiles an SM on and up to 64 steps a tile.
bool bwd_window_two_kv(const BwdArgs& a) {
  long long rows = static_cast<long long>(a.window) + kBT + kStepQ;  // of a head that see a key tile
  if (rows > a.N_q) rows = a.N_q;
  return a.d == kBwD && a.window >= 0 && rows * (a.Hq / a.Hkv) <= 64 * kStepQ &&
         static_cast<long long>(a.B) * a.Hkv * ((a.N_kv + kBT - 1) / kBT) >= 5 * 152;
}

// dQ with one / two blocks an SM likewise (dK/dV with one):
//   more query tiles than SMs   B=8 H=12 N=1024 (768): W=64 76 / 60, 1023 93 / 81; B=1 Hq=16 Hkv=4 N=8192
//                               (1,024): W=256 108 / 91, 2048 266 / 245, 8191 450 / 428; B=2 H=8 N=2048
//                               (256) W=256 35 / 28; B=3 (384) W=2047 66 / 63
//   fewer                       B=1 H=8 N=2048 (128) W=256 28 / 28; B=1 H=2 N=4096 (64) W=4095 43 / 45
bool bwd_window_two_q(const BwdArgs& a) {
  return a.d == kBwD && a.window >= 0 &&
         static_cast<long long>(a.B) * a.Hq * ((a.N_q + kBT - 1) / kBT) > 152;
}

int launch_bwd_window_dkdv(const BwdArgs& a, const BwdParams& p, unsigned blocks, cudaStream_t stream) {
  CUtensorMap m[4], dk, dv;
  const uint64_t bhk = static_cast<uint64_t>(a.B) * a.Hkv, rb = kBwD * 2;
  if (!short_maps(a, kStepQ, kBT, m) ||
      !make_tmap_3d(&dk, a.dk, a.bf16, kBwD, a.N_kv, bhk, rb, rb * a.N_kv, 64, kBT, 1) ||
      !make_tmap_3d(&dv, a.dv, a.bf16, kBwD, a.N_kv, bhk, rb, rb * a.N_kv, 64, kBT, 1))
    return -5;
  auto kern = a.bf16 ? attn_bwd_short_dkdv_kernel<true> : attn_bwd_short_dkdv_kernel<false>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, KvShort::kBytes) != cudaSuccess)
    return -5;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(kBwThreads);
  cfg.dynamicSmemBytes = KvShort::kBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, m[0], m[1], m[2], m[3], dk, dv, p) == cudaSuccess ? 0 : -5;
}

// A programmatic dependent of dK/dV: its blocks fill the SMs of that kernel's tail.
int launch_bwd_window_dq(const BwdArgs& a, const BwdParams& p, unsigned blocks, cudaStream_t stream) {
  CUtensorMap m[4], dq;
  const uint64_t bhq = static_cast<uint64_t>(a.B) * a.Hq, rb = kBwD * 2;
  if (!short_maps(a, kBT, kStepQ, m) ||
      !make_tmap_3d(&dq, a.dq, a.bf16, kBwD, a.N_q, bhq, rb, rb * a.N_q, 64, kBT, 1))
    return -5;
  auto kern = a.bf16 ? attn_bwd_short_dq_kernel<true> : attn_bwd_short_dq_kernel<false>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, QShort::kBytes) != cudaSuccess)
    return -5;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(kBwThreads);
  cfg.dynamicSmemBytes = QShort::kBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, m[0], m[1], m[2], m[3], dq, p) == cudaSuccess ? 0 : -5;
}

}  // namespace attn
