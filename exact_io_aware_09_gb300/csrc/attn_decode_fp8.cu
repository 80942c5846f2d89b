// Split-KV decode over a quantised paged cache (attn_cache_fp8.cu writes it): one new query token
// per sequence attends to keys and values held as E4M3 codes with a power-of-two scale per
// (token, key/value head) row.
//
// With codes kc_j, vc_j and scales 2^a_j, 2^b_j:  x_j = scale log2(e) 2^a_j (q . kc_j),
// p_j = 2^(x_j - m), o = sum_j p_j 2^b_j vc_j / sum_j p_j.  The values' scale joins the exponent:
// the running maximum is taken of x_j + b_j, the weight of vc_j is w_j = 2^(x_j + b_j - m) <= 1,
// and the row sum adds w_j 2^-b_j.  So w_j goes into the second product as a 16-bit number
// whatever the scales are, at the cost of one multiply.
//
// The split kernel is the 16-bit one's (attn_decode.cu) with half the bytes: blocks of (split,
// key/value head, sequence), a producer warp bringing 64-token stages page by page with TMA, four
// compute warps of 16 tokens each.  Both products run on the warp-level f16 tiles: an E4M3 code is
// exactly an f16 number, so the codes are converted and not rounded.  A bf16 query is scaled by a
// power of two to at most 2 in magnitude before its own conversion to f16, which then loses only
// what is 2^-25 of the row's largest element.
//
// Channel order.  The sum over channels may run in any order, so thread c of a row group takes
// the contiguous channels D/4 c .. D/4 c + D/4 - 1 of its key (16-byte loads, free of bank
// conflicts in the swizzled stage), four of them per 16-wide step, and the query fragments are
// loaded in that order.  Likewise output column (tile t, n) stands for channel n (D/8) + t, so
// that the values' operand is made from contiguous bytes of four tokens by byte permutes.
//
// Bound by HBM: 2 (d + 4) bytes per cached token and head.
#include "attn_decode.cuh"

namespace attn {

namespace {

struct DecFp8Params : DecParams {
  const float* k_scales;  // [num_pages, Hkv, page_size]
  const float* v_scales;
};

// l adds w_j 2^(-b_j - kSumShift): the sum stays in range for scales from 2^-126 to 2^94.
constexpr int kSumShift = 32;

template <int D>
struct Fp8Layout {
  static constexpr uint32_t kTensor = kDecTok * D;  // codes of K or V of one stage
  static constexpr uint32_t kStage = 2 * kTensor;
  static constexpr uint32_t kRing = kDecStages * kStage;
  static constexpr uint32_t kRed = kDecWarps * kMaxGroup * (D + 2) * 4;  // reuses the ring
  static_assert(kRed <= kRing, "merge scratch must fit in the ring");
  static constexpr uint32_t kScales = kRing;  // [stage][K, V][64] floats
  static constexpr uint32_t kBar = kScales + kDecStages * 2 * kDecTok * 4;
  static constexpr uint32_t kMisc = kBar + 2 * kDecStages * 8;
  static constexpr uint32_t kPages = kMisc + 16;  // first pool row of the split's pages, or -1
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

}  // namespace

template <int D, bool BF16>
__global__ void __launch_bounds__(kDecThreads)
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
  if (split >= n_splits) return;
  const int t0 = split * p.split;
  const int n_tok = min(p.split, t_stop - t0);
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
  __syncthreads();

  if (warp == kDecWarps) {
    // ------------------------------------------------------------------ TMA producer
    // Lane i brings the i-th page of a stage: its codes of K and V as one box each, its scales as
    // two short copies.
    int* page_row = reinterpret_cast<int*>(gbase + L::kPages);
    const int32_t* tbl = p.block_table + static_cast<size_t>(b) * p.max_pages;
    const int first = t0 >> p.page_log2;
    const int n_pg_all = ((t0 + n_tok - 1) >> p.page_log2) - first + 1;
    for (int i = lane; i < n_pg_all; i += 32) {
      const int pg = tbl[first + i];
      const bool good = pg >= 0 && pg < p.num_pages;
      if (!good) latch_status(p.status, kStatusBadLengths);
      page_row[i] = good ? pg : -1;
    }
    __syncwarp();
    const uint64_t stream_policy = l2_policy_evict_first();
    const int rows = min(p.page_size, kDecTok);
    const int n_pg = kDecTok / rows;
    const uint32_t page_bytes = 2u * rows * D + 2u * rows * 4u;
    int issued = 0;
    for (int st = 0; st < n_stages; ++st) {
      const int s = st % kDecStages;
      bool ok = true;
      if (lane == 0 && st >= kDecStages)
        ok = wait_bounded(EMPTY(s), ((st / kDecStages) - 1) & 1, abort_flag, p.status);
      if (!__shfl_sync(0xffffffffu, ok, 0)) break;
      const uint32_t kbuf = base + s * L::kStage;
      const uint32_t vbuf = kbuf + L::kTensor;
      const uint32_t sbuf = base + L::kScales + s * (2 * kDecTok * 4);
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
        const size_t sc = ((static_cast<size_t>(page) * p.Hkv + hk) << p.page_log2) + off;
        bulk_load(sbuf + lane * rows * 4, p.k_scales + sc, rows * 4, FULL(s));
        bulk_load(sbuf + kDecTok * 4 + lane * rows * 4, p.v_scales + sc, rows * 4, FULL(s));
      }
      issued = st + 1;
    }
    if (lane == 0)
      for (int st = (issued > kDecStages ? issued - kDecStages : 0); st < issued; ++st)
        wait_bounded(FULL(st % kDecStages), (st / kDecStages) & 1, nullptr, p.status, 100000000ull);
    return;  // the producer takes no part in the reduction below
  }

  // -------------------------------------------------------------------- compute warps
  const int g = lane >> 2;  // accumulator row (query head inside the group) and +8
  const int c = lane & 3;
  const int hq0 = hk * p.G;
  const bool row0 = g < p.G, row1 = g + 8 < p.G;
  const uint16_t* qb = p.q + (static_cast<size_t>(b) * p.Hq + hq0) * D;
  uint32_t qa[D / 16][4];
  float f0 = p.sl2, f1 = p.sl2;  // factors of the two rows' products
  {
    float mx0 = 0.0f, mx1 = 0.0f;
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
      // channels D/4 c + 4 ks .. + 3: the first pair at the step's k = 2c, 2c + 1, the second at
      // k = 2c + 8, 2c + 9
      const int col = c * (D / 4) + ks * 4;
      const uint2 a = row0 ? *reinterpret_cast<const uint2*>(qb + g * D + col) : make_uint2(0, 0);
      const uint2 d = row1 ? *reinterpret_cast<const uint2*>(qb + (g + 8) * D + col) : make_uint2(0, 0);
      qa[ks][0] = a.x;
      qa[ks][2] = a.y;
      qa[ks][1] = d.x;
      qa[ks][3] = d.y;
      if constexpr (BF16) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint32_t u = e ? a.y : a.x, v = e ? d.y : d.x;
          mx0 = fmaxf(mx0, fmaxf(fabsf(__uint_as_float(u << 16)), fabsf(__uint_as_float(u & 0xffff0000u))));
          mx1 = fmaxf(mx1, fmaxf(fabsf(__uint_as_float(v << 16)), fabsf(__uint_as_float(v & 0xffff0000u))));
        }
      }
    }
    if constexpr (BF16) {
#pragma unroll
      for (int sh = 1; sh < 4; sh <<= 1) {
        mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, sh));
        mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, sh));
      }
      // biased exponent of the largest magnitude, kept where 2^-e is a normal number too
      auto biased = [](float m) {
        const int E = static_cast<int>(__float_as_uint(m) >> 23);
        return E == 255 || m == 0.0f ? 127 : E < 1 ? 1 : E > 253 ? 253 : E;
      };
      const int e0 = biased(mx0), e1 = biased(mx1);
      const float i0 = __uint_as_float(static_cast<uint32_t>(254 - e0) << 23);
      const float i1 = __uint_as_float(static_cast<uint32_t>(254 - e1) << 23);
      f0 *= __uint_as_float(static_cast<uint32_t>(e0) << 23);
      f1 *= __uint_as_float(static_cast<uint32_t>(e1) << 23);
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        qa[ks][0] = q_pair<BF16>(qa[ks][0], i0);
        qa[ks][2] = q_pair<BF16>(qa[ks][2], i0);
        qa[ks][1] = q_pair<BF16>(qa[ks][1], i1);
        qa[ks][3] = q_pair<BF16>(qa[ks][3], i1);
      }
    }
  }
  float m[2] = {-INFINITY, -INFINITY};
  float l[2] = {0.f, 0.f};  // partial over this thread's columns
  float o[D / 8][4];
#pragma unroll
  for (int nd = 0; nd < D / 8; ++nd) o[nd][0] = o[nd][1] = o[nd][2] = o[nd][3] = 0.f;

  bool ok = true;
  for (int st = 0; st < n_stages; ++st) {
    const int s = st % kDecStages;
    if (!dec_warp_wait(FULL(s), (st / kDecStages) & 1, abort_flag, p.status)) {
      ok = false;
      break;
    }
    uint8_t* kbuf = gbase + s * L::kStage;
    uint8_t* vbuf = kbuf + L::kTensor;
    const float* k_sc = reinterpret_cast<const float*>(gbase + L::kScales) + s * 2 * kDecTok;
    const float* v_sc = k_sc + kDecTok;
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
      // S = Q K^T: key n of tile nt is stage row w0 + 8 nt + n
      float sc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        const int row = w0 + nt * 8 + g;
#pragma unroll
        for (int h = 0; h < D / 64; ++h) {
          const uint4 w = *reinterpret_cast<const uint4*>(kbuf + code_off<D>(row, c * (D / 64) + h));
          const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int i = 0; i < 4; ++i)
            mma_m16n8k16<false>(sc[nt], qa[h * 4 + i], e4m3x2_f16x2(ww[i]), e4m3x2_f16x2_hi(ww[i]));
        }
      }
      // online softmax over the 16 tokens, rows g and g + 8 (see the file's head)
      float x[2][4], inv_b[2][2];
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        const float2 ks = *reinterpret_cast<const float2*>(k_sc + w0 + nt * 8 + 2 * c);
        const float2 vs = *reinterpret_cast<const float2*>(v_sc + w0 + nt * 8 + 2 * c);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int vb = static_cast<int>(__float_as_uint(e ? vs.y : vs.x) >> 23) & 0xff;
          const float bj = static_cast<float>(vb - 127);
          const float kj = e ? ks.y : ks.x;
          inv_b[nt][e] = __uint_as_float(static_cast<uint32_t>(max(254 - kSumShift - vb, 0)) << 23);
          const bool in = nt * 8 + 2 * c + e < valid;
          x[nt][e] = in ? fmaf(sc[nt][e], f0 * kj, bj) : -INFINITY;
          x[nt][2 + e] = in ? fmaf(sc[nt][2 + e], f1 * kj, bj) : -INFINITY;
        }
      }
      float mx0 = fmaxf(fmaxf(x[0][0], x[0][1]), fmaxf(x[1][0], x[1][1]));
      float mx1 = fmaxf(fmaxf(x[0][2], x[0][3]), fmaxf(x[1][2], x[1][3]));
      mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, 1));
      mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, 2));
      mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, 1));
      mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, 2));
      const float mn0 = fmaxf(m[0], mx0), mn1 = fmaxf(m[1], mx1);
      const float a0 = (m[0] == -INFINITY) ? 0.f : ex2(m[0] - mn0);
      const float a1 = (m[1] == -INFINITY) ? 0.f : ex2(m[1] - mn1);
      const float mu0 = (mn0 == -INFINITY) ? 0.f : mn0;
      const float mu1 = (mn1 == -INFINITY) ? 0.f : mn1;
      m[0] = mn0;
      m[1] = mn1;
      float pr[2][4];
      l[0] *= a0;
      l[1] *= a1;
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          pr[nt][e] = ex2(x[nt][e] - mu0);
          pr[nt][2 + e] = ex2(x[nt][2 + e] - mu1);
          l[0] = fmaf(pr[nt][e], inv_b[nt][e], l[0]);
          l[1] = fmaf(pr[nt][2 + e], inv_b[nt][e], l[1]);
        }
#pragma unroll
      for (int nd = 0; nd < D / 8; ++nd) {
        o[nd][0] *= a0;
        o[nd][1] *= a0;
        o[nd][2] *= a1;
        o[nd][3] *= a1;
      }
      uint32_t pa[4];
      pa[0] = pack2<false>(pr[0][0], pr[0][1]);
      pa[1] = pack2<false>(pr[0][2], pr[0][3]);
      pa[2] = pack2<false>(pr[1][0], pr[1][1]);
      pa[3] = pack2<false>(pr[1][2], pr[1][3]);
      // O += P V: tokens 2c, 2c + 1 (tile 0) and 2c + 8, 2c + 9 (tile 1); this thread's output
      // column of tile t is channel g (D/8) + t: D/8 contiguous bytes of each token
      constexpr int kW = D / 32;  // words of a token
      uint32_t v[4][kW];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = w0 + (r >> 1) * 8 + 2 * c + (r & 1);
        if constexpr (D == 128)
          *reinterpret_cast<uint4*>(v[r]) = *reinterpret_cast<const uint4*>(vbuf + code_off<D>(row, g));
        else
          *reinterpret_cast<uint2*>(v[r]) =
              *reinterpret_cast<const uint2*>(vbuf + code_off<D>(row, g >> 1) + (g & 1) * 8);
      }
#pragma unroll
      for (int i = 0; i < kW; ++i) {
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          const uint32_t sel = hh ? 0x7362u : 0x5140u;  // (a_2h, b_2h, a_2h+1, b_2h+1)
          const uint32_t lo = __byte_perm(v[0][i], v[1][i], sel);
          const uint32_t hi = __byte_perm(v[2][i], v[3][i], sel);
          mma_m16n8k16<false>(o[i * 4 + hh * 2], pa, e4m3x2_f16x2(lo), e4m3x2_f16x2(hi));
          mma_m16n8k16<false>(o[i * 4 + hh * 2 + 1], pa, e4m3x2_f16x2_hi(lo), e4m3x2_f16x2_hi(hi));
        }
      }
      if (valid < 16) fence_proxy_async_smem();  // generic zeros before the next TMA write
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(EMPTY(s));
  }

  // ---------------------------------------------------- merge the four warps' states
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
    l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
  }
  named_bar_sync(1, kDecWarps * 32);  // every warp is done with the ring
  ok = ok && (*abort_flag == 0);
  float* red = reinterpret_cast<float*>(gbase);  // [warp][row][D + 2]
  constexpr int kRow = D + 2;
  constexpr int kT = D / 8;
  if (ok) {
    float* rw = red + warp * kMaxGroup * kRow;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (!(e < 2 ? row0 : row1)) continue;
      float* dst = rw + (e < 2 ? g : g + 8) * kRow + (2 * c + (e & 1)) * kT;
#pragma unroll
      for (int nd = 0; nd < kT; ++nd) dst[nd] = o[nd][e];
    }
    if (c == 0) {
      if (row0) {
        rw[g * kRow + D] = m[0];
        rw[g * kRow + D + 1] = l[0];
      }
      if (row1) {
        rw[(g + 8) * kRow + D] = m[1];
        rw[(g + 8) * kRow + D + 1] = l[1];
      }
    }
  }
  named_bar_sync(1, kDecWarps * 32);
  if (ok) {
    const size_t part0 = (static_cast<size_t>(b) * p.Hq + hq0) * p.max_splits + split;
    constexpr float kUnshift = 1.0f / 4294967296.0f;  // 2^-kSumShift
    for (int i = threadIdx.x; i < p.G * D; i += kDecWarps * 32) {
      const int row = i / D, col = i % D;
      float mm = -INFINITY;
#pragma unroll
      for (int w = 0; w < kDecWarps; ++w) mm = fmaxf(mm, red[(w * kMaxGroup + row) * kRow + D]);
      float ll = 0.f, acc = 0.f;
#pragma unroll
      for (int w = 0; w < kDecWarps; ++w) {
        const float mw = red[(w * kMaxGroup + row) * kRow + D];
        const float wgt = (mw == -INFINITY) ? 0.f : ex2(mw - mm);
        ll += wgt * red[(w * kMaxGroup + row) * kRow + D + 1];
        acc += wgt * red[(w * kMaxGroup + row) * kRow + col];
      }
      const size_t part = part0 + static_cast<size_t>(row) * p.max_splits;
      p.ws_o[part * D + col] = acc / ll * kUnshift;
      if (col == 0) {
        p.ws_ml[part * 2] = mm + static_cast<float>(kSumShift);
        p.ws_ml[part * 2 + 1] = ll;
      }
    }
  }
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
  auto kern = attn_decode_fp8_split_kernel<D, BF16>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kBytes) !=
      cudaSuccess)
    return -5;
  if (any_keys) {
    kern<<<dim3(max_splits, a.Hkv, a.B), kDecThreads, L::kBytes, stream>>>(tk, tv, p);
    if (cudaGetLastError() != cudaSuccess) return -5;
  }
  return launch_decode_merge(p, D, BF16, a.B, a.o, a.lse, stream);
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
