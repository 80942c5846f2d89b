// Split-KV decode over a quantised paged cache (attn_cache_fp8.cu writes it): one new query token
// per sequence attends to keys and values held as E4M3 codes with a power-of-two scale per
// (token, key/value head) row.
//
// With codes kc_j, vc_j and scales 2^a_j, 2^b_j:  x_j = scale log2(e) 2^a_j (q . kc_j),
// p_j = 2^(x_j - m), o = sum_j p_j 2^b_j vc_j / sum_j p_j.  m and the row sum are those of the scores
// alone.  The weights of the second product take the values' scales into their exponent, y_j = x_j + b_j,
// and have a reference of their own: w_j = 2^(y_j - r + 7), r at most 8 below the largest y_j so far, so
// that w_j <= 2^15 fits a 16-bit number and o is off by at most half a step of each w_j (2^-12 of it) and,
// where w_j is below fp16's normal numbers, by 2^-32 of the largest p_j 2^b_j for each code.  A value row
// of zeros adds nothing to o whatever its scale (the writer's is 1, often far above the other rows'), so
// it takes no part in r: sixteen tokens that would raise r look at their codes first.  m, too, only
// follows a score that exceeds it by 8: most steps find neither, and need no maximum over the warp.
//
// The split kernel is the 16-bit one's (attn_decode.cu) with half the bytes: blocks of (split,
// key/value head, sequence), a producer warp bringing 64-token stages page by page with TMA, four
// compute warps of 16 tokens each.  Both products run on the warp-level f16 tiles: an E4M3 code is
// exactly an f16 number, so the codes are converted and not rounded.  A bf16 query is scaled by a
// power of two to at most 2 in magnitude before its own conversion to f16, which then loses only
// what is 2^-25 of the row's largest element.
//
// Channel order.  The sum over channels may run in any order, so thread (g, c) takes the contiguous
// channels D/4 c .. D/4 c + D/4 - 1 of its keys (16-byte loads, free of bank conflicts in the
// swizzled stage), four of them per 16-wide step, and the query fragments are loaded in that order.
// Likewise its output channels are the contiguous g D/8 .., so that the values' operand is made
// from contiguous bytes of four tokens by byte permutes.
//
// Merging.  A call whose sequences have at most eight splits runs each (sequence, head)'s splits as
// one cluster, whose blocks read one another's states through distributed shared memory: one
// launch, no workspace.  More splits go through the workspace and the 16-bit decode's merge kernel.
//
// Bound by HBM: 2 (d + 4) bytes per cached token and head.  64 sequences of 1k-32k tokens (Hq=64 Hkv=8
// d=128, 64-token pages, 2.45 GB): 394 us, 6.2 TB/s, against 723 for the 16-bit cache.  Without its
// arithmetic it takes as long; what counts is how the bytes are asked for: codes and scales both with the
// policy that evicts their lines first (codes with the default one 411 us, scales as short asynchronous
// copies with it 408).  One sequence of 1,001 tokens (Hq=16 Hkv=4 d=64): 12 us on the device, one launch.
#include "attn_decode.cuh"
#include "attn_rows.cuh"

namespace attn {

namespace {

struct DecFp8Params : DecParams {
  const float* k_scales;  // [num_pages, Hkv, page_size]
  const float* v_scales;
  int cluster;            // a sequence's splits are the blocks of one cluster
  uint16_t* out;          // [B, Hq, D], [B, Hq]: written here when they are
  float* lse;
};

// m and the weights' reference r rise when a key exceeds them by more than 2^kRise; a key at r weighs 2^kTop.
constexpr float kRise = 8.0f, kTop = 7.0f;

template <int D>
struct Fp8Layout {
  static constexpr uint32_t kTensor = kDecTok * D;  // codes of K or V of one stage
  static constexpr uint32_t kStage = 2 * kTensor;
  static constexpr uint32_t kRing = kDecStages * kStage;
  static constexpr uint32_t kRed = kDecWarps * kMaxGroup * (D + 2) * 4;  // reuses the ring
  // the block's merged state for its cluster: [row][D] and (m, l) per row
  static constexpr uint32_t kFin = kRed;
  static_assert(kFin + kMaxGroup * (D + 2) * 4 <= kRing, "merge scratch must fit in the ring");
  static constexpr uint32_t kBar = kRing;
  static constexpr uint32_t kMisc = kBar + 2 * kDecStages * 8;
  static constexpr uint32_t kPages = kMisc + 16;  // the split's pages, or -1
  static constexpr int kMaxSplitPages = 8192 / 16;
  static constexpr uint32_t kBytes = kPages + kMaxSplitPages * 4 + 1024;
};

// Two codes in the low half of a word -> an f16 pair (exact).
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t}"
      : "=r"(r)
      : "r"(w));
  return r;
}
__device__ __forceinline__ uint32_t e4m3x2_f16x2_hi(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, b;\n\t}"
      : "=r"(r)
      : "r"(w));
  return r;
}

// Byte offset of 16-byte chunk `chunk` of a stage's row: D-byte rows in the swizzle of that width
// (address bits 4-6 exclusive-ored with bits 7-9, at d = 64 bits 4-5 with bits 7-8).
template <int D>
__device__ __forceinline__ uint32_t code_off(int row, int chunk) {
  const uint32_t a = static_cast<uint32_t>(row) * D + static_cast<uint32_t>(chunk) * 16;
  return a ^ ((a >> 3) & (D == 128 ? 0x70u : 0x30u));
}

// The query row (16-bit) as f16 pairs times 2^-e, and 2^e: e = 0 for f16, for bf16 such that the
// largest magnitude lies in [1, 2) (0 where the row is zero or not finite).
template <bool BF16>
__device__ __forceinline__ uint32_t q_pair(uint32_t w, float inv) {
  if constexpr (!BF16) return w;
  return pack2<false>(__uint_as_float(w << 16) * inv, __uint_as_float(w & 0xffff0000u) * inv);
}

__device__ __forceinline__ float pair_amax(uint32_t w) {  // of a bf16 pair
  return fmaxf(fabsf(__uint_as_float(w << 16)), fabsf(__uint_as_float(w & 0xffff0000u)));
}

// Biased exponent of a bf16 query row's scale: that of its largest magnitude, kept where 2^-e is a
// normal number too.
__device__ __forceinline__ int q_biased_exp(float amax) {
  const int e = static_cast<int>(__float_as_uint(amax) >> 23);
  return e == 255 || amax == 0.0f ? 127 : e < 1 ? 1 : e > 253 ? 253 : e;
}

// The D / 8 codes of channels g D/8 .. of a stage row.
template <int D>
__device__ __forceinline__ void load_v_words(const uint8_t* vbuf, int row, int g,
                                             uint32_t (&v)[D / 32]) {
  if constexpr (D == 128)
    *reinterpret_cast<uint4*>(v) = *reinterpret_cast<const uint4*>(vbuf + code_off<D>(row, g));
  else
    *reinterpret_cast<uint2*>(v) =
        *reinterpret_cast<const uint2*>(vbuf + code_off<D>(row, g >> 1) + (g & 1) * 8);
}

}  // namespace

// A warp's query rows and state (attn_rows.cuh) and its work on sixteen tokens.  The state's m and l are
// those of the scores, its o counts in units of 2^(ref - kTop).
template <int D, bool BF16, int NT>
struct Fp8Warp : RowState<D, NT, false> {
  uint32_t qf[NT][D / 16][2];
  float f[NT][2];    // factors of the rows' products
  float ref[NT][2];  // the weights' reference; -inf before the first value row that is not zero

  // q: the group's query rows, G of them
  __device__ __forceinline__ void init(const uint16_t* q, int G, float sl2, int lane) {
    RowState<D, NT, false>::init();
    const int g = lane >> 2, c = lane & 3;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      ref[n][0] = ref[n][1] = -INFINITY;
      const int row = n * 8 + g;
      float mx = 0.0f;
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        // channels D/4 c + 4 ks .. + 3: the first pair at the step's k = 2c, 2c + 1, the second at
        // k = 2c + 8, 2c + 9
        const uint2 a = row < G ? *reinterpret_cast<const uint2*>(q + row * D + c * (D / 4) + ks * 4)
                                : make_uint2(0, 0);
        qf[n][ks][0] = a.x;
        qf[n][ks][1] = a.y;
        if constexpr (BF16) mx = fmaxf(mx, fmaxf(pair_amax(a.x), pair_amax(a.y)));
      }
      float mine = sl2;
      if constexpr (BF16) {
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const int e = q_biased_exp(mx);
        const float inv = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
        mine *= __uint_as_float(static_cast<uint32_t>(e) << 23);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          qf[n][ks][0] = q_pair<BF16>(qf[n][ks][0], inv);
          qf[n][ks][1] = q_pair<BF16>(qf[n][ks][1], inv);
        }
      }
      f[n][0] = __shfl_sync(0xffffffffu, mine, 8 * c);
      f[n][1] = __shfl_sync(0xffffffffu, mine, 8 * c + 4);
    }
  }

  // Stage rows w0 .. w0 + 15, of which the first `valid` count.  scale: lane i holds the key scale of
  // row i, lane 16 + i its value scale.
  __device__ __forceinline__ void tokens(const uint8_t* kbuf, const uint8_t* vbuf, float scale, int w0,
                                         int valid, int lane) {
    const int g = lane >> 2, c = lane & 3;
    float sc[NT][4] = {};
#pragma unroll
    for (int h = 0; h < D / 64; ++h) {
      const uint4 u = *reinterpret_cast<const uint4*>(kbuf + code_off<D>(w0 + g, c * (D / 64) + h));
      const uint4 v = *reinterpret_cast<const uint4*>(kbuf + code_off<D>(w0 + g + 8, c * (D / 64) + h));
      const uint32_t wa[4] = {u.x, u.y, u.z, u.w}, wb[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t a[4] = {e4m3x2_f16x2(wa[i]), e4m3x2_f16x2(wb[i]), e4m3x2_f16x2_hi(wa[i]),
                               e4m3x2_f16x2_hi(wb[i])};
#pragma unroll
        for (int n = 0; n < NT; ++n)
          mma_m16n8k16<false>(sc[n], a, qf[n][h * 4 + i][0], qf[n][h * 4 + i][1]);
      }
    }
    float x[NT][2][2], y[NT][2][2];  // scores, and with the values' exponents
    bool rise = false;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float vj = __shfl_sync(0xffffffffu, scale, 16 + g + 8 * k);
      const float kj = __shfl_sync(0xffffffffu, scale, g + 8 * k);
      const float bj = static_cast<float>((static_cast<int>(__float_as_uint(vj) >> 23) & 0xff) - 127);
      const bool in = g + 8 * k < valid;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          x[n][k][r] = in ? sc[n][2 * k + r] * (f[n][r] * kj) : -INFINITY;
          y[n][k][r] = x[n][k][r] + bj;
          rise = rise || x[n][k][r] > this->m[n][r] + kRise || y[n][k][r] > ref[n][r] + kRise;
        }
    }
    if (__any_sync(0xffffffffu, rise)) raise(x, y, vbuf, w0, lane);
    uint32_t pb[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float w[2][2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float mu = (this->m[n][r] == -INFINITY) ? 0.f : this->m[n][r];
        const float shift = (ref[n][r] == -INFINITY) ? 0.f : kTop - ref[n][r];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          this->l[n][r] += ex2(x[n][k][r] - mu);
          w[k][r] = ex2(y[n][k][r] + shift);
        }
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) pb[n][k] = transpose_8x8(pack2<false>(w[k][0], w[k][1]));
    }
    // this thread's channels of tile t are g D/8 + 2t and + 1: D/8 contiguous bytes of a token
    constexpr int kW = D / 32;
    uint32_t v[4][kW];
#pragma unroll
    for (int r = 0; r < 4; ++r) load_v_words<D>(vbuf, w0 + (r >> 1) * 8 + 2 * c + (r & 1), g, v[r]);
#pragma unroll
    for (int i = 0; i < kW; ++i)
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        const uint32_t sel = hh ? 0x7362u : 0x5140u;  // bytes 2hh, 2hh + 1 of two tokens, paired
        const uint32_t lo = __byte_perm(v[0][i], v[1][i], sel);
        const uint32_t hi = __byte_perm(v[2][i], v[3][i], sel);
        const uint32_t av[4] = {e4m3x2_f16x2(lo), e4m3x2_f16x2_hi(lo), e4m3x2_f16x2(hi),
                                e4m3x2_f16x2_hi(hi)};
#pragma unroll
        for (int n = 0; n < NT; ++n)
          mma_m16n8k16<false>(this->o[n][i * 2 + hh], av, pb[n][0], pb[n][1]);
      }
  }

  // Takes value rows of zeros out of y, and raises m to the largest x, the references to the largest y left,
  // where those exceed them by more than 2^kRise.  Lane i looks at half a row's codes.
  __device__ __forceinline__ void raise(const float (&x)[NT][2][2], float (&y)[NT][2][2], const uint8_t* vbuf,
                                        int w0, int lane) {
    uint32_t any = 0;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      const uint4 u = *reinterpret_cast<const uint4*>(
          vbuf + code_off<D>(w0 + (lane >> 1), (lane & 1) * (D / 32) + i));
      any |= u.x | u.y | u.z | u.w;
    }
    const uint32_t some = __ballot_sync(0xffffffffu, (any & 0x7f7f7f7fu) != 0);  // two bits a row
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float a[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
#pragma unroll
        for (int k = 0; k < 2; ++k)
          if (!((some >> (2 * ((lane >> 2) + 8 * k))) & 3u)) y[n][k][r] = -INFINITY;
        float mx = fmaxf(x[n][0][r], x[n][1][r]), my = fmaxf(y[n][0][r], y[n][1][r]);
#pragma unroll
        for (int sh = 4; sh < 32; sh <<= 1) {
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, sh));
          my = fmaxf(my, __shfl_xor_sync(0xffffffffu, my, sh));
        }
        float& m = this->m[n][r];
        if (mx > m + kRise) {
          this->l[n][r] *= (m == -INFINITY) ? 0.f : ex2(m - mx);
          m = mx;
        }
        a[r] = 1.0f;
        if (my > ref[n][r] + kRise) {
          a[r] = (ref[n][r] == -INFINITY) ? 0.f : ex2(ref[n][r] - my);
          ref[n][r] = my;
        }
      }
#pragma unroll
      for (int t = 0; t < D / 16; ++t) {
        this->o[n][t][0] *= a[0];
        this->o[n][t][1] *= a[1];
        this->o[n][t][2] *= a[0];
        this->o[n][t][3] *= a[1];
      }
    }
  }

  // The state to the merge scratch, its rows divided by their sums: o 2^(ref - kTop - m) / l, the power
  // of two in two halves, so that it leaves fp32's range only where the result does.
  __device__ __forceinline__ void store(float* rw, int rows, int lane) const {
    float h[NT][2], hl[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const bool none = ref[n][r] == -INFINITY;  // no key, or no value row that is not zero
        h[n][r] = none ? 1.0f : ex2(0.5f * (ref[n][r] - kTop - this->m[n][r]));
        hl[n][r] = this->l[n][r] == 0.f ? 0.f : h[n][r] / this->l[n][r];
      }
    RowState<D, NT, false>::store(
        rw, rows, lane, [&](int t, int i) { return (lane >> 2) * (D / 8) + 2 * t + i; },
        [&](int n, int r, float x) { return x * h[n][r] * hl[n][r]; });
  }
};

// One column tile: four blocks of 160 threads an SM at up to 102 registers (two column tiles need
// more), which hides the latency of a stage's conversions and products behind other blocks.
template <int D, bool BF16, int NT>
__global__ void __launch_bounds__(kDecThreads, NT == 1 ? 4 : 2)
    attn_decode_fp8_split_kernel(const __grid_constant__ CUtensorMap tm_k,
                                 const __grid_constant__ CUtensorMap tm_v, const DecFp8Params p) {
  using L = Fp8Layout<D>;
  const int split = blockIdx.x;
  const int hk = blockIdx.y;
  const int b = blockIdx.z;
  if (threadIdx.x == 0) griddep_launch_dependents();  // the merge may be scheduled (it waits)
  int t_start, t_stop;
  if (!seq_bounds(p, b, t_start, t_stop)) {
    if (split == 0 && hk == 0 && threadIdx.x == 0) latch_status(p.status, kStatusBadLengths);
    return;
  }
  const int n_splits = (t_stop + p.split - 1) / p.split;
  if (split >= n_splits && !p.cluster) return;
  const int t0 = split * p.split;
  const int n_tok = max(min(p.split, t_stop - t0), 0);
  const int n_stages = (n_tok + kDecTok - 1) / kDecTok;

  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  const uint32_t bars = base + L::kBar;
#define FULL(s) (bars + 8u * (s))
#define EMPTY(s) (bars + 8u * (kDecStages + (s)))
  volatile int* abort_flag = reinterpret_cast<volatile int*>(gbase + L::kMisc);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kDecStages; ++s) {
      mbar_init(FULL(s), 1);
      mbar_init(EMPTY(s), kDecWarps);
    }
    *abort_flag = 0;
    fence_barrier_init();
  }
  int* page_row = reinterpret_cast<int*>(gbase + L::kPages);
  const int first = t0 >> p.page_log2;
  {
    const int32_t* tbl = p.block_table + static_cast<size_t>(b) * p.max_pages;
    const int n_pg_all = n_tok > 0 ? ((t0 + n_tok - 1) >> p.page_log2) - first + 1 : 0;
    for (int i = threadIdx.x; i < n_pg_all; i += kDecThreads) {
      const int pg = tbl[first + i];
      const bool good = pg >= 0 && pg < p.num_pages;
      if (!good) latch_status(p.status, kStatusBadLengths);
      page_row[i] = good ? pg : -1;
    }
  }
  __syncthreads();

  if (warp == kDecWarps) {
    // ------------------------------------------------------------------ TMA producer
    // Lane i brings the i-th page of a stage: its codes of K and V as one box each.
    const uint64_t stream_policy = l2_policy_evict_first();
    const int rows = min(p.page_size, kDecTok);
    const int n_pg = kDecTok / rows;
    const uint32_t page_bytes = 2u * rows * D;
    int issued = 0;
    for (int st = 0; st < n_stages; ++st) {
      const int s = st % kDecStages;
      bool ok = true;
      if (lane == 0 && st >= kDecStages)
        ok = wait_bounded(EMPTY(s), ((st / kDecStages) - 1) & 1, abort_flag, p.status);
      if (!__shfl_sync(0xffffffffu, ok, 0)) break;
      const uint32_t kbuf = base + s * L::kStage;
      const uint32_t vbuf = kbuf + L::kTensor;
      int page = -1, off = 0;
      if (lane < n_pg) {
        const int t = t0 + st * kDecTok + lane * rows;
        if (t < t_stop) {
          page = page_row[(t >> p.page_log2) - first];
          off = t & (p.page_size - 1);
        }
      }
      const uint32_t n_loads = __popc(__ballot_sync(0xffffffffu, page >= 0));
      if (lane == 0) mbar_arrive_expect_tx(FULL(s), n_loads * page_bytes);
      __syncwarp();
      if (page >= 0) {
        const uint32_t box_off = static_cast<uint32_t>(lane) * rows * D;
        const int row = (page << p.page_log2) + off;
        tma_load_3d_hint(kbuf + box_off, &tm_k, FULL(s), 0, hk, row, stream_policy);
        tma_load_3d_hint(vbuf + box_off, &tm_v, FULL(s), 0, hk, row, stream_policy);
      }
      issued = st + 1;
    }
    if (lane == 0)
      for (int st = (issued > kDecStages ? issued - kDecStages : 0); st < issued; ++st)
        wait_bounded(FULL(st % kDecStages), (st / kDecStages) & 1, nullptr, p.status, 100000000ull);
    return;  // the producer takes no part in the reduction below
  }

  // -------------------------------------------------------------------- compute warps
  const int hq0 = hk * p.G;
  Fp8Warp<D, BF16, NT> st_w;
  st_w.init(p.q + (static_cast<size_t>(b) * p.Hq + hq0) * D, p.G, p.sl2, lane);

  // The scales go straight to registers, two stages ahead: a warp's sixteen tokens lie in one page, and
  // lane i < 16 loads the key scale of token i, lane 16 + i its value scale.  (As copies into the stage,
  // two of 256 bytes each, they cost 408 us against 392 back to back at the 64 sequences above.)
  auto scale_at = [&](int st) -> float {
    const int t = t0 + st * kDecTok + warp * 16;
    if (t >= t_stop || st >= n_stages) return 0.0f;
    const int page = page_row[(t >> p.page_log2) - first];
    if (page < 0) return 0.0f;
    return __ldcs((lane < 16 ? p.k_scales : p.v_scales) +
                  ((static_cast<size_t>(page) * p.Hkv + hk) << p.page_log2) + (t & (p.page_size - 1)) +
                  (lane & 15));
  };
  float sc0 = scale_at(0), sc1 = scale_at(1);
  bool ok = true;
  for (int st = 0; st < n_stages; ++st) {
    const int s = st % kDecStages;
    const float scale = sc0;
    sc0 = sc1;
    sc1 = scale_at(st + 2);
    if (!dec_warp_wait(FULL(s), (st / kDecStages) & 1, abort_flag, p.status)) {
      ok = false;
      break;
    }
    uint8_t* kbuf = gbase + s * L::kStage;
    uint8_t* vbuf = kbuf + L::kTensor;
    const int w0 = warp * 16;                     // first stage row of this warp
    const int valid = n_tok - st * kDecTok - w0;  // rows of this warp that belong to the chunk
    if (valid > 0) {
      if (valid < 16) {
        // Rows past the chunk: their weight is 0, and 0 times a NaN code has to stay 0.
        for (int i = lane; i < (16 - valid) * (D / 16); i += 32)
          *reinterpret_cast<uint4*>(vbuf + code_off<D>(w0 + valid + i / (D / 16), i % (D / 16))) =
              make_uint4(0, 0, 0, 0);
        __syncwarp();
      }
      st_w.tokens(kbuf, vbuf, scale, w0, valid, lane);
      if (valid < 16) fence_proxy_async_smem();  // generic zeros before the next TMA write
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(EMPTY(s));
  }

  // ---------------------------------------------------- merge the four warps' states
  st_w.finish();
  named_bar_sync(1, kDecWarps * 32);  // every warp is done with the ring
  ok = ok && (*abort_flag == 0);
  float* red = reinterpret_cast<float*>(gbase);  // [warp][row][D + 2]
  if (ok) st_w.store(red + warp * kMaxGroup * (D + 2), p.G, lane);
  named_bar_sync(1, kDecWarps * 32);
  const RowsOut w{p.ws_o, p.ws_ml, p.out, p.lse, p.max_splits, split, p.cluster != 0};
  merge_rows<D, BF16, kDecWarps, kMaxGroup, true>(
      red, reinterpret_cast<float*>(gbase + L::kFin), p.G, ok, n_tok > 0, w,
      [&](int row) { return static_cast<size_t>(b) * p.Hq + hq0 + row; });
#undef FULL
#undef EMPTY
}

template <int D, bool BF16>
static int launch_decode_fp8_variant(const DecodeArgs& a, const CacheFp8& c, cudaStream_t stream) {
  using L = Fp8Layout<D>;
  const int max_splits = (a.max_seqlen + a.split - 1) / a.split;
  const bool any_keys = c.num_pages > 0 && max_splits > 0;
  const uint64_t tokens = static_cast<uint64_t>(c.num_pages) * c.page_size;
  const uint32_t box_rows = static_cast<uint32_t>(c.page_size < kDecTok ? c.page_size : kDecTok);
  CUtensorMap tk, tv;
  if (any_keys &&
      (!make_tmap_3d_u8(&tk, c.k_pages, D, a.Hkv, tokens, D, static_cast<uint64_t>(D) * a.Hkv, D, 1,
                        box_rows) ||
       !make_tmap_3d_u8(&tv, c.v_pages, D, a.Hkv, tokens, D, static_cast<uint64_t>(D) * a.Hkv, D, 1,
                        box_rows)))
    return -5;
  DecFp8Params p = {};
  p.q = static_cast<const uint16_t*>(a.q);
  p.block_table = c.block_table;
  p.seqlens = a.seqlens;
  p.page_size = c.page_size;
  while ((1 << p.page_log2) < c.page_size) ++p.page_log2;
  p.max_pages = c.max_pages;
  p.num_pages = c.num_pages;
  p.max_splits = max_splits > 0 ? max_splits : 1;
  const size_t parts = static_cast<size_t>(a.B) * a.Hq * p.max_splits;
  p.ws_o = static_cast<float*>(a.workspace);
  p.ws_ml = reinterpret_cast<float*>(static_cast<char*>(a.workspace) +
                                     ((parts * D * 4 + 255) & ~static_cast<size_t>(255)));
  p.status = device_status_ptr();
  if (!p.status) return -5;
  p.Hq = a.Hq;
  p.Hkv = a.Hkv;
  p.G = a.Hq / a.Hkv;
  p.max_seqlen = a.max_seqlen;
  p.split = a.split;
  p.sl2 = a.scale * 1.4426950408889634f;
  p.k_scales = c.k_scales;
  p.v_scales = c.v_scales;
  p.cluster = any_keys && max_splits <= kMaxCluster;
  p.out = static_cast<uint16_t*>(a.o);
  p.lse = a.lse;
  // up to eight heads a group fill one column tile; more need two
  auto kern = p.G <= 8 ? attn_decode_fp8_split_kernel<D, BF16, 1>
                       : attn_decode_fp8_split_kernel<D, BF16, 2>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kBytes) !=
      cudaSuccess)
    return -5;
  if (any_keys && p.cluster) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(max_splits, a.Hkv, a.B);
    cfg.blockDim = dim3(kDecThreads);
    cfg.dynamicSmemBytes = L::kBytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = max_splits;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kern, tk, tv, p) != cudaSuccess) return -5;
    return cudaGetLastError() == cudaSuccess ? 0 : -5;
  }
  if (any_keys) {
    kern<<<dim3(max_splits, a.Hkv, a.B), kDecThreads, L::kBytes, stream>>>(tk, tv, p);
    if (cudaGetLastError() != cudaSuccess) return -5;
  }
  return launch_decode_merge(p, D, BF16, a.B, a.o, a.lse, stream);
}

size_t decode_fp8_workspace_bytes(int B, int Hq, int max_seqlen, int split, int d) {
  if (split <= 0 || max_seqlen < 0) return 0;
  // one cluster merges up to eight splits; an empty cache's rows need no state either
  if (max_seqlen > 0 && (max_seqlen - 1) / split < kMaxCluster) return 0;
  return max_seqlen > 0 ? decode_workspace_bytes(B, Hq, max_seqlen, split, d) : 0;
}

// Tokens of a split, with four blocks an SM.
int decode_fp8_split(int B, int Hkv, int max_seqlen) {
  return row_split_tokens(static_cast<long long>(B) * Hkv, max_seqlen, 152 * 4);
}

int launch_attn_decode_fp8(const DecodeArgs& a, const CacheFp8& c, cudaStream_t stream) {
  if (a.d == 64)
    return a.bf16 ? launch_decode_fp8_variant<64, true>(a, c, stream)
                  : launch_decode_fp8_variant<64, false>(a, c, stream);
  if (a.d == 128)
    return a.bf16 ? launch_decode_fp8_variant<128, true>(a, c, stream)
                  : launch_decode_fp8_variant<128, false>(a, c, stream);
  return -2;
}

}  // namespace attn
