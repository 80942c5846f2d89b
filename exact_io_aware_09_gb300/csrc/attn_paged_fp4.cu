// New tokens of each sequence over a paged cache held in 4 bits (fp4.cuh; attn_cache_fp4.cu writes it): at
// most 16 (token, query head) rows per key/value head, so a decode step, or a few tokens of a small group.
//
// Keys and values are code * scale, exact in fp16, so both products run on the warp-level f16 tiles with
// nothing rounded but the weights: x_j = scale log2(e) (q . k_j), w_j = 2^(x_j - m + 7) rounded to fp16,
// o = sum_j w_j v_j / sum_j w_j.  m is at most 8 below the largest x_j so far (it follows a score that
// exceeds it by 8: most steps find none, and need no maximum over the warp), so that w_j <= 2^15 fits fp16
// and half a step of a weight below fp16's normal numbers is 2^-32 of the largest.  A bf16 query is scaled
// by a power of two to at most 2 in magnitude before its conversion to f16.
//
// The split kernel is that of a few rows over the 16-bit cache (attn_paged_few.cu) with the codes' channel
// orders: thread (g, c) = (lane / 4, lane % 4) takes channels D/4 c .. of its keys for the scores, so that a
// 16-byte load holds its operands of several steps, and channels D/8 g .. of its values, so that their
// scale is one byte a token.  Values meet the second product as pairs of tokens: the low four bits of two
// tokens' bytes side by side in one, and the high ones, which convert as pairs.  The pool's order (a
// head's rows of a page side by side) makes a page's codes one contiguous copy, and its scale bytes another.
// A token that no row sees gets a value scale of zero, which makes its values zeros whatever they hold.
//
// A stage is 128 tokens, 32 of each warp: its barriers, mask and maximum check cost as much as a third of the
// work on sixteen tokens.  Three stages and 96 registers let four blocks share an SM.
//
// Bound by latency: half an instruction a cycle and scheduler with 4.5 warps to choose from and no pipe above 45%;
// what a warp waits for most are its own results, through conversion, scale and product (fixed latency), then
// the pipes.  128 of the 350 instructions it takes for sixteen tokens at d = 128 convert a pair of codes and scale
// it.  64 sequences of 16k tokens (Hq=64 Hkv=8 d=128,
// 1.21 GB): 250 us (4.8 TB/s) in 64-token pages, 299 in 16-token ones (four copies a page and stage);
// of 1k-32k tokens 283 with the merge, the 8-bit cache 394; d = 64: 167 us.  Measured at the first shape: 64-token
// stages 307, one of 128 tokens more with three blocks an SM 281; scale bytes straight to registers, as the 8-bit
// decode has them, 329; a ring for every warp without a producer, five blocks an SM, 278; two chains of products
// for the scores 262; splits of 1,024 tokens 297.
#include "attn_decode.cuh"
#include "attn_rows.cuh"
#include "fp4.cuh"

namespace attn {

namespace {

constexpr int kFew4Rows = 16;
constexpr int kFew4Tok = 128;                    // tokens of a stage, 32 of each compute warp
constexpr int kFew4Groups = kFew4Tok / 16 / kDecWarps;
constexpr int kFew4Stages = 3;                   // of the ring
constexpr int kFew4MaxStages = 2048 / kFew4Tok;  // of a split (row_split_tokens)
constexpr float kRise = 8.0f, kTop = 7.0f, kNone = 3.402823466e38f;

struct Few4Params {
  const uint16_t* q;  // [total_q, Hq, D]
  const int32_t* block_table;
  const int32_t* cu_q;  // null: sequence b's one token is row b
  const int32_t* seqlens;
  const uint8_t* k_scales;
  const uint8_t* v_scales;
  int* status;
  int page_log2, max_pages, num_pages, total_q, max_q, max_k;
  int Hq, Hkv, G, window, sinks, split_stages;
  float sl2;
  float* ws_o;  // partial states, or null with a cluster
  float* ws_ml;
  uint16_t* out;
  float* lse;
  int n_splits, cluster;
};

template <int D, int NT>
struct Few4Layout {
  static constexpr int kMaxR = NT * 8;
  static constexpr uint32_t kTensor = kFew4Tok * D / 2;   // codes of K or V of one stage
  static constexpr uint32_t kScales = kFew4Tok * D / 16;  // and scale bytes
  static constexpr uint32_t kStage = 2 * (kTensor + kScales);
  static constexpr uint32_t kRing = kFew4Stages * kStage;
  static constexpr uint32_t kRed = kDecWarps * kMaxR * (D + 2) * 4;  // reuses the ring
  static constexpr uint32_t kFin = kRed;
  static_assert(kFin + kMaxR * (D + 2) * 4 <= kRing, "merge scratch must fit in the ring");
  static constexpr uint32_t kBar = (kRing + 7) / 8 * 8;
  static constexpr uint32_t kMisc = kBar + 2 * kFew4Stages * 8;
  static constexpr uint32_t kPages = kMisc + 16;  // the split's pages, box by box, or -1
  static constexpr uint32_t kBytes = kPages + kFew4MaxStages * (kFew4Tok / 16) * 4 + 1024;
};

// Blocks that share an SM, by registers.
constexpr int few4_blocks_per_sm(int d, int nt) { return nt == 1 ? 4 : d == 64 ? 3 : 2; }

template <typename T>
__device__ __forceinline__ T lds(uint32_t addr);
template <>
__device__ __forceinline__ uint32_t lds<uint32_t>(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}
template <>
__device__ __forceinline__ uint2 lds<uint2>(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
  return v;
}
template <>
__device__ __forceinline__ uint4 lds<uint4>(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr));
  return v;
}
// One byte and two, zero extended.
__device__ __forceinline__ uint32_t lds8(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}

// Byte offset of 16-byte chunk `chunk` of a stage's row: D/2-byte rows in the swizzle of that width
// (address bits 4-5 exclusive-ored with bits 7-8, at d = 64 bit 4 with bit 7).
template <int D>
__device__ __forceinline__ uint32_t code4_off(int row, int chunk) {
  const uint32_t a = static_cast<uint32_t>(row) * (D / 2) + static_cast<uint32_t>(chunk) * 16;
  return a ^ ((a >> 3) & (D == 128 ? 0x30u : 0x10u));
}

}  // namespace

// A warp's query rows and state and its work on sixteen tokens; o and l count in units of 2^(m - kTop), and
// a score's weight is 2^(x + shift), shift = kTop - m (kNone before the first key: any score is above it, and
// one of -inf has no weight).
template <int D, bool BF16, int NT>
struct Few4Warp : RowState<D, NT, false> {
  static constexpr int kB = D / kFp4Block;  // scale bytes of a row
  uint32_t qf[NT][D / 16][2];
  float f[NT][2];  // factors of the rows' products
  float shift[NT][2];

  // row(r): query row r < rows
  template <typename F>
  __device__ __forceinline__ void init(F row, int rows, float sl2, int lane) {
    RowState<D, NT, false>::init();
    const int g = lane >> 2, c = lane & 3;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const uint16_t* q = row(n * 8 + g < rows ? n * 8 + g : 0) + c * (D / 4);
      float mx = 0.0f;
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        // channels D/4 c + 4 ks .. + 3: the first pair at the step's k = 2c, 2c + 1, the second at
        // k = 2c + 8, 2c + 9
        const uint2 a = n * 8 + g < rows ? *reinterpret_cast<const uint2*>(q + ks * 4) : make_uint2(0, 0);
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
      shift[n][0] = shift[n][1] = kNone;
    }
  }

  // Places of this thread's operands in a stage, from the warp's first token: key g and, eight rows on, key
  // g + 8; value tokens 2c and 2c + 1 in the thread's order and those eight rows on (the swizzles do not
  // change over eight rows); their scale bytes.
  uint32_t k_at, v_at[2], ks_at, vs_at[2];

  __device__ __forceinline__ void places(int warp, int lane) {
    using L = Few4Layout<D, NT>;
    const int g = lane >> 2, c = lane & 3, w0 = warp * 16 * kFew4Groups;
    k_at = D == 128 ? code4_off<D>(w0 + g, c) : code4_off<D>(w0 + g, c >> 1) + (c & 1) * 8;
    ks_at = 2 * L::kTensor + (w0 + g) * kB + c * (kB / 4);
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int row = w0 + 2 * c + (r ^ swap(c));
      v_at[r] = L::kTensor + code4_off<D>(row, D == 128 ? g >> 1 : g >> 2) + (D == 128 ? (g & 1) * 8 : (g & 3) * 4);
      vs_at[r] = 2 * L::kTensor + L::kScales + row * kB + (D == 128 ? g : g >> 1);
    }
  }
  // Token pairs are taken in the order that keeps the values' loads free of bank conflicts: a thread whose
  // `swap` is set has its pairs the other way round, of the weights too.
  static __device__ __forceinline__ int swap(int c) { return D == 128 ? c & 1 : c >> 1; }

  // The warp's tokens of the stage at shared address `stage`, in groups of sixteen.  Where `edge`:
  // see(i, n, k, r), whether row 2c + r of tile n sees key g + 8k of group i, and some(t), whether any row
  // sees the warp's token t.
  template <typename F, typename S>
  __device__ __forceinline__ void tokens(uint32_t stage, bool edge, F see, S some, int lane) {
    constexpr uint32_t kRow8 = 8 * D / 2, kS8 = 8 * kB;  // eight rows of codes, of scale bytes
    const int c = lane & 3;
    float x[kFew4Groups][NT][2][2];
#pragma unroll
    for (int gr = 0; gr < kFew4Groups; ++gr) {
      float acc[NT][4] = {};
      constexpr int kW = D / 32;  // words of a thread's keys' channels: eight codes each
      uint32_t wa[kW], wb[kW], sa[kB / 4], sb[kB / 4];
      const uint32_t at = stage + k_at + 2 * gr * kRow8, s_at = stage + ks_at + 2 * gr * kS8;
      if constexpr (D == 128) {
        *reinterpret_cast<uint4*>(wa) = lds<uint4>(at);
        *reinterpret_cast<uint4*>(wb) = lds<uint4>(at + kRow8);
        const uint32_t a = lds16(s_at), b = lds16(s_at + kS8);
        sa[0] = fp4_scale_pair(a & 0xffu);
        sa[1] = fp4_scale_pair(a >> 8);
        sb[0] = fp4_scale_pair(b & 0xffu);
        sb[1] = fp4_scale_pair(b >> 8);
      } else {
        *reinterpret_cast<uint2*>(wa) = lds<uint2>(at);
        *reinterpret_cast<uint2*>(wb) = lds<uint2>(at + kRow8);
        sa[0] = fp4_scale_pair(lds8(s_at));
        sb[0] = fp4_scale_pair(lds8(s_at + kS8));
      }
#pragma unroll
      for (int i = 0; i < kW; ++i) {
        uint32_t a[4], b[4];
        fp4_values8(wa[i], sa[i / 2], a);
        fp4_values8(wb[i], sb[i / 2], b);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t ab[4] = {a[2 * h], b[2 * h], a[2 * h + 1], b[2 * h + 1]};
#pragma unroll
          for (int n = 0; n < NT; ++n)
            mma_m16n8k16<false>(acc[n], ab, qf[n][2 * i + h][0], qf[n][2 * i + h][1]);
        }
      }
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int r = 0; r < 2; ++r) x[gr][n][k][r] = acc[n][2 * k + r] * f[n][r];
    }
    if (edge) {
#pragma unroll
      for (int gr = 0; gr < kFew4Groups; ++gr)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int r = 0; r < 2; ++r)
              if (!see(gr, n, k, r)) x[gr][n][k][r] = -INFINITY;
    }
    bool rise = false;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float top = fmaxf(x[0][n][0][r], x[0][n][1][r]);
#pragma unroll
        for (int gr = 1; gr < kFew4Groups; ++gr) top = max3f(top, x[gr][n][0][r], x[gr][n][1][r]);
        rise = rise || top + shift[n][r] > kRise + kTop;
      }
    if (__any_sync(0xffffffffu, rise)) raise(x);
#pragma unroll
    for (int gr = 0; gr < kFew4Groups; ++gr) {
      uint32_t pb[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float w[2][2];
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            w[k][r] = ex2(x[gr][n][k][r] + shift[n][r]);
            this->l[n][r] += w[k][r];
          }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const uint32_t t = transpose_8x8(pack2<false>(w[k][0], w[k][1]));
          pb[n][k] = __byte_perm(t, t, swap(c) ? 0x1032 : 0x3210);
        }
      }
      constexpr int kV = D / 64;  // words of a thread's channels of one token
      uint32_t v[4][kV], by[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const uint32_t at = stage + v_at[r & 1] + (2 * gr + (r >> 1)) * kRow8;
        if constexpr (D == 128)
          *reinterpret_cast<uint2*>(v[r]) = lds<uint2>(at);
        else
          v[r][0] = lds<uint32_t>(at);
        by[r] = lds8(stage + vs_at[r & 1] + (2 * gr + (r >> 1)) * kS8);
      }
      if (edge) {
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (!some(gr * 16 + (r >> 1) * 8 + 2 * c + ((r & 1) ^ swap(c)))) by[r] = 0;
      }
      const uint32_t sv[2] = {fp4_scale_pair(by[0], by[1]), fp4_scale_pair(by[2], by[3])};
#pragma unroll
      for (int i = 0; i < kV; ++i) {
        // byte t: the codes of channel 2t of two tokens (even), of channel 2t + 1 (odd)
        constexpr uint32_t kLow = 0x0f0f0f0fu;
        uint32_t ev[2][4], od[2][4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t u0 = v[2 * h][i], u1 = v[2 * h + 1][i];
          fp4_values8((u0 & kLow) | ((u1 << 4) & ~kLow), sv[h], ev[h]);
          fp4_values8(((u0 >> 4) & kLow) | (u1 & ~kLow), sv[h], od[h]);
        }
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const uint32_t av[4] = {ev[0][t], od[0][t], ev[1][t], od[1][t]};
#pragma unroll
          for (int n = 0; n < NT; ++n) mma_m16n8k16<false>(this->o[n][i * 4 + t], av, pb[n][0], pb[n][1]);
        }
      }
    }
  }

  // Raises m to the largest x where that exceeds it by more than kRise: where its weight would pass
  // 2^(kRise + kTop), by the sum that makes the weight (of an m past 2^24 shift is rounded, and x - m > kRise
  // may say otherwise).  After it no weight passes 2^(kTop + 1).
  __device__ __forceinline__ void raise(const float (&x)[kFew4Groups][NT][2][2]) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float a[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float mx = fmaxf(x[0][n][0][r], x[0][n][1][r]);
#pragma unroll
        for (int gr = 1; gr < kFew4Groups; ++gr) mx = max3f(mx, x[gr][n][0][r], x[gr][n][1][r]);
#pragma unroll
        for (int sh = 4; sh < 32; sh <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, sh));
        float& m = this->m[n][r];
        a[r] = 1.0f;
        if (mx + shift[n][r] > kRise + kTop) {
          a[r] = ex2((kTop - mx) - shift[n][r]);  // (0 at the first key)
          m = mx;
          shift[n][r] = kTop - mx;
        }
        this->l[n][r] *= a[r];
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

  // The state to the merge scratch, m such that l counts in units of 2^m.
  __device__ __forceinline__ void store(float* rw, int rows, int lane) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int r = 0; r < 2; ++r) this->m[n][r] -= kTop;
    RowState<D, NT, false>::store(
        rw, rows, lane, [&](int t, int i) { return (lane >> 2) * (D / 8) + 2 * t + i; },
        [](int, int, float x) { return x; });
  }
};

template <int D, bool BF16, int NT>
__global__ void __launch_bounds__(kDecThreads, few4_blocks_per_sm(D, NT))
    attn_paged_fp4_few_kernel(const __grid_constant__ CUtensorMap tm_k,
                              const __grid_constant__ CUtensorMap tm_v, const Few4Params p) {
  using L = Few4Layout<D, NT>;
  using Warp = Few4Warp<D, BF16, NT>;
  const int split = blockIdx.x;
  const int hk = blockIdx.y;
  const int b = blockIdx.z;
  if (threadIdx.x == 0) griddep_launch_dependents();  // the merge may be scheduled (it waits)
  const int c0 = p.cu_q ? p.cu_q[b] : b, n = p.cu_q ? p.cu_q[b + 1] - c0 : 1;
  const int len = p.seqlens[b];
  if (c0 < 0 || n < 0 || n > p.max_q || n > p.total_q - c0 || len < (p.cu_q ? n : 0) || len > p.max_k ||
      ((len - 1) >> p.page_log2) >= p.max_pages) {
    if (split == 0 && hk == 0 && threadIdx.x == 0) latch_status(p.status, kStatusBadLengths);
    return;
  }
  if (n == 0) return;
  const int rows = n * p.G;
  const int pos0 = len - n;  // (-1: an empty cache, whose row sees no key)
  // stages of the visible keys: `sink_st` of them from key 0, then from stage w_begin on
  const int w_begin = p.window < 0 ? 0 : max(pos0 - p.window, 0) / kFew4Tok;
  const int sink_st = p.window < 0 ? 0 : min((min(p.sinks, len) + kFew4Tok - 1) / kFew4Tok, w_begin);
  const int all = sink_st + (len + kFew4Tok - 1) / kFew4Tok - w_begin;
  const int i0 = split * p.split_stages;
  const int n_stages = min(max(all - i0, 0), p.split_stages);
  auto stage_token = [&](int st) {
    const int i = i0 + st;
    return (i < sink_st ? i : w_begin + i - sink_st) * kFew4Tok;
  };
  auto out_row = [&](int row) {
    const int t = row / p.G;
    return static_cast<size_t>(c0 + t) * p.Hq + hk * p.G + (row - t * p.G);
  };
  if (n_stages == 0 && !p.cluster) {
    // no key of its own: the merge gives it no weight
    if (static_cast<int>(threadIdx.x) < rows)
      reinterpret_cast<float2*>(p.ws_ml)[out_row(threadIdx.x) * p.n_splits + split] =
          make_float2(-INFINITY, 0.0f);
    return;
  }

  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  const uint32_t bars = base + L::kBar;
#define FULL(s) (bars + 8u * (s))
#define EMPTY(s) (bars + 8u * (kFew4Stages + (s)))
  volatile int* abort_flag = reinterpret_cast<volatile int*>(gbase + L::kMisc);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kFew4Stages; ++s) {
      mbar_init(FULL(s), 1);
      mbar_init(EMPTY(s), kDecWarps);
    }
    *abort_flag = 0;
    fence_barrier_init();
  }
  // pages of the split, as boxes of a page's rows (a stage's where it has more)
  constexpr int kTokLog2 = 7;
  static_assert(1 << kTokLog2 == kFew4Tok, "tokens of a stage");
  const int box_log2 = min(p.page_log2, kTokLog2), box = 1 << box_log2, pg_log2 = kTokLog2 - box_log2;
  int* pages = reinterpret_cast<int*>(gbase + L::kPages);  // [stage][box of it]
  for (int i = threadIdx.x; i < n_stages << pg_log2; i += kDecThreads) {
    const int t = stage_token(i >> pg_log2) + (i & ((1 << pg_log2) - 1)) * box;
    int page = -1;
    if (t < len) {
      page = p.block_table[static_cast<size_t>(b) * p.max_pages + (t >> p.page_log2)];
      if (page < 0 || page >= p.num_pages) {
        latch_status(p.status, kStatusBadLengths);
        page = -1;
      }
    }
    pages[i] = page;
  }
  __syncthreads();

  const int page_mask = (1 << p.page_log2) - 1;
  if (warp == kDecWarps) {
    // ------------------------------------------------------------------ TMA producer
    const uint64_t stream_policy = l2_policy_evict_first();
    const uint32_t box_bytes = static_cast<uint32_t>(box) * (D / 2), box_scales = box * Warp::kB;
    int issued = 0;
    for (int st = 0; st < n_stages; ++st) {
      const int s = st % kFew4Stages;
      bool ok = true;
      if (lane == 0 && st >= kFew4Stages)
        ok = wait_bounded(EMPTY(s), ((st / kFew4Stages) - 1) & 1, abort_flag, p.status);
      if (!__shfl_sync(0xffffffffu, ok, 0)) break;
      const uint32_t kbuf = base + s * L::kStage + lane * box_bytes;
      const uint32_t ks = base + s * L::kStage + 2 * L::kTensor + lane * box_scales;
      const int page = lane < (1 << pg_log2) ? pages[(st << pg_log2) + lane] : -1;
      const uint32_t n_loads = __popc(__ballot_sync(0xffffffffu, page >= 0));
      if (lane == 0) mbar_arrive_expect_tx(FULL(s), n_loads * 2 * (box_bytes + box_scales));
      __syncwarp();
      if (page >= 0) {
        const int at = (stage_token(st) + lane * box) & page_mask;
        tma_load_4d_hint(kbuf, &tm_k, FULL(s), 0, at, hk, page, stream_policy);
        tma_load_4d_hint(kbuf + L::kTensor, &tm_v, FULL(s), 0, at, hk, page, stream_policy);
        const size_t row = ((static_cast<size_t>(page) * p.Hkv + hk) << p.page_log2) + at;
        bulk_load_hint(ks, p.k_scales + row * Warp::kB, box_scales, FULL(s), stream_policy);
        bulk_load_hint(ks + L::kScales, p.v_scales + row * Warp::kB, box_scales, FULL(s), stream_policy);
      }
      issued = st + 1;
    }
    if (lane == 0)
      for (int st = (issued > kFew4Stages ? issued - kFew4Stages : 0); st < issued; ++st)
        wait_bounded(FULL(st % kFew4Stages), (st / kFew4Stages) & 1, nullptr, p.status, 100000000ull);
    return;  // the producer takes no part in the reduction below
  }

  // -------------------------------------------------------------------- compute warps
  const int g = lane >> 2, c = lane & 3;
  Warp ws;
  ws.init([&](int row) { return p.q + out_row(row) * D; }, rows, p.sl2, lane);
  ws.places(warp, lane);
  const int last = pos0 + n - 1;                     // position of the last new token
  const int first = p.window < 0 ? 0 : pos0 - p.window;  // first key of the first one's window
  bool ok = true;
  int s = 0, parity = 0;
  for (int st = 0; st < n_stages; ++st) {
    if (!dec_warp_wait(FULL(s), parity, abort_flag, p.status)) {
      ok = false;
      break;
    }
    const int key0 = stage_token(st) + warp * 16 * kFew4Groups;  // first key of this warp
    if (key0 <= last) {
      const bool edge = key0 + 16 * kFew4Groups - 1 > pos0 || (p.window >= 0 && key0 < last - p.window);
      ws.tokens(
          base + s * L::kStage, edge,
          [&](int i, int u, int k, int r) {
            const int key = key0 + 16 * i + g + 8 * k;
            const int pos = pos0 + min((u * 8 + 2 * c + r) / p.G, n - 1);
            return key <= pos && (p.window < 0 || pos - key <= p.window || key < p.sinks);
          },
          [&](int t) { return key0 + t <= last && (key0 + t >= first || key0 + t < p.sinks); }, lane);
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(EMPTY(s));
    if (++s == kFew4Stages) {
      s = 0;
      parity ^= 1;
    }
  }

  // ---------------------------------------------------- merge the four warps' states
  ws.finish();
  named_bar_sync(1, kDecWarps * 32);  // every warp is done with the ring
  ok = ok && (*abort_flag == 0);
  float* red = reinterpret_cast<float*>(gbase);  // [warp][row][D + 2]
  if (ok) ws.store(red + warp * L::kMaxR * (D + 2), rows, lane);
  named_bar_sync(1, kDecWarps * 32);
  const RowsOut w{p.ws_o, p.ws_ml, p.out, p.lse, p.n_splits, split, p.cluster != 0};
  merge_rows<D, BF16, kDecWarps, L::kMaxR, false>(red, reinterpret_cast<float*>(gbase + L::kFin), rows, ok,
                                                  n_stages > 0, w, out_row);
#undef FULL
#undef EMPTY
}

static bool few_rows(int max_q, int G) { return static_cast<long long>(max_q) * G <= kFew4Rows; }

// Splits of a call with few rows, and 128-token stages of each.
static void few_split(int B, int Hkv, int G, int max_q, int max_k, int window, int sinks, int d,
                      int& n_splits, int& stages) {
  long long tokens = max_k;
  if (window >= 0) {
    // the window's keys with those of the stages its ends lie in, and the sinks' stages
    const long long near = static_cast<long long>(window) + max_q + 2 * kFew4Tok +
                           (static_cast<long long>(sinks) + kFew4Tok - 1) / kFew4Tok * kFew4Tok;
    if (near < tokens) tokens = near;
  }
  const int slots = 152 * few4_blocks_per_sm(d, max_q * G <= 8 ? 1 : 2);
  const int per = row_split_tokens(static_cast<long long>(B) * Hkv, tokens, slots);
  stages = (per + kFew4Tok - 1) / kFew4Tok;
  const long long all = (tokens + kFew4Tok - 1) / kFew4Tok;
  n_splits = all > 0 ? static_cast<int>((all + stages - 1) / stages) : 1;
}

template <int D, bool BF16, int NT>
static int launch_few4(const PagedArgs& a, const CacheFp4& c, cudaStream_t stream) {
  using L = Few4Layout<D, NT>;
  // {bytes of a row, token of a page, head, page}
  const uint64_t row = D / 2, head = row * c.page_size;
  const uint64_t dims[4] = {row, static_cast<uint64_t>(c.page_size), static_cast<uint64_t>(a.Hkv),
                            static_cast<uint64_t>(c.num_pages)};
  const uint64_t strides[3] = {row, head, head * a.Hkv};
  const uint32_t box[4] = {D / 2, static_cast<uint32_t>(c.page_size < kFew4Tok ? c.page_size : kFew4Tok), 1, 1};
  CUtensorMap tk = {}, tv = {};
  if (c.num_pages > 0 &&
      (!make_tmap_4d_u8(&tk, c.k_codes, dims, strides, box) || !make_tmap_4d_u8(&tv, c.v_codes, dims, strides, box)))
    return -5;
  Few4Params p = {};
  p.q = static_cast<const uint16_t*>(a.q);
  p.block_table = c.block_table;
  p.cu_q = a.cu_q;
  p.seqlens = a.seqlens;
  p.k_scales = c.k_scales;
  p.v_scales = c.v_scales;
  p.status = device_status_ptr();
  if (!p.status) return -5;
  while ((1 << p.page_log2) < c.page_size) ++p.page_log2;
  p.max_pages = c.max_pages;
  p.num_pages = c.num_pages;
  p.total_q = a.total_q;
  p.max_q = a.max_q;
  p.max_k = a.max_k;
  p.Hq = a.Hq;
  p.Hkv = a.Hkv;
  p.G = a.Hq / a.Hkv;
  p.window = a.window;
  p.sinks = a.sinks;
  p.sl2 = a.scale * 1.4426950408889634f;
  p.out = static_cast<uint16_t*>(a.o);
  p.lse = a.lse;
  few_split(a.B, a.Hkv, p.G, a.max_q, a.max_k, a.window, a.sinks, D, p.n_splits,
            p.split_stages);
  p.cluster = p.n_splits <= kMaxCluster;
  if (!p.cluster) paged_parts(a, D, p.n_splits, p.ws_o, p.ws_ml);
  auto kern = attn_paged_fp4_few_kernel<D, BF16, NT>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kBytes) != cudaSuccess)
    return -5;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.n_splits, a.Hkv, a.B);
  cfg.blockDim = dim3(kDecThreads);
  cfg.dynamicSmemBytes = L::kBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = p.n_splits;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.cluster ? 1 : 0;
  if (cudaLaunchKernelEx(&cfg, kern, tk, tv, p) != cudaSuccess) return -5;
  return p.cluster ? 0 : launch_paged_merge(a, p.n_splits, stream);
}

template <int D, bool BF16>
static int launch_variant(const PagedArgs& a, const CacheFp4& c, cudaStream_t stream) {
  const int G = a.Hq / a.Hkv;
  if (few_rows(a.max_q, G))
    return a.max_q * G <= 8 ? launch_few4<D, BF16, 1>(a, c, stream) : launch_few4<D, BF16, 2>(a, c, stream);
  return launch_attn_fp4_chunk(a, c, stream);
}

int launch_attn_paged_fp4(const PagedArgs& a, const CacheFp4& c, cudaStream_t stream) {
  if (a.d == 64)
    return a.bf16 ? launch_variant<64, true>(a, c, stream) : launch_variant<64, false>(a, c, stream);
  return a.bf16 ? launch_variant<128, true>(a, c, stream) : launch_variant<128, false>(a, c, stream);
}

size_t paged_fp4_workspace_bytes(int total_q, int B, int Hq, int Hkv, int max_q, int max_k, int window,
                                 int sinks, int d) {
  if (total_q <= 0 || B <= 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv || max_q <= 0 || max_k <= 0 || d <= 0) return 0;
  const int G = Hq / Hkv;
  if (!few_rows(max_q, G))
    return G <= 128 ? fp4_chunk_workspace_bytes(total_q, B, Hq, Hkv, max_q, max_k, window, sinks, d) : 0;
  int n_splits, stages;
  few_split(B, Hkv, G, max_q, max_k, window, sinks, d, n_splits, stages);
  return n_splits <= kMaxCluster ? 0 : paged_parts_bytes(total_q, Hq, n_splits, d);
}

}  // namespace attn
