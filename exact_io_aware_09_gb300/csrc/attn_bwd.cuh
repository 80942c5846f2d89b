// Declarations shared by the backward kernels (attn_bwd.cu, attn_bwd_window.cu).
#pragma once
#include "internal.h"
#include "ptx.cuh"

namespace attn {

constexpr int kBT = 128;            // rows of a query tile and keys of a key tile
constexpr int kStepQ = 64;          // queries per step of the dK/dV kernels
constexpr uint32_t kSub = 128 * 128;  // bytes of one 64-column, 128-row swizzled sub-tile
constexpr uint64_t kBwdDrainNs = 100000000ull;

struct BwdParams {
  const float* lse2;  // [B*Hq, nqp]  -L * log2(e), fp16: + kPShift; -inf on padding rows
  const float* dvec;  // [B*Hq, nqp]  -scale * D; 0 on padding rows
  const uint16_t* q;     // [B, Hq, N_q, d]
  const uint16_t* k;     // [B, Hkv, N_kv, d]
  const uint16_t* v;
  const uint16_t* dout;  // [B, Hq, N_q, d]
  uint16_t* dq;       // [B, Hq, N_q, d]
  uint16_t* dk;       // [B, Hkv, N_kv, d]
  uint16_t* dv;
  int* status;
  int Hq, Hkv, G, N_q, N_kv, n_qtiles, n_kvtiles, nqp, causal;
  float sl2;    // scale * log2(e)
  float scale;
  int window, sinks;  // window variant: keys behind the diagonal, first keys always visible
  int sink_tiles, sink_parts;  // ... its key tiles with sinks, each cut into that many blocks
  float* part;        // [B*Hkv, sink_tiles, sink_parts][dV, dK][128, d] their partial sums
  // fp16: [B*Hkv][4] the largest |dO_i|, scale |D_i| and |V_j| (row norms) of a plane, as bits
  const uint32_t* range;
};

// fp16 holds numbers from 2^-14 to 2^16 with all their bits.  P and dS enter their products there times
// powers of two that the gradients are divided by at the end: P times 2^kPShift (P <= 1; lse2 carries the
// shift), dS of a (batch, key/value head) plane times 2^t, the largest for which
//   |dS_ij| <= scale (|dP_ij| + |D_i|) <= scale max |dO_i| max |V_j| + max scale |D_i|
// stays below 2^15.  Error of dQ and dK, N=2048 W=1024 d=128, of their norm, without / with: dO ~ 1 2.9e-4
// / 2.9e-4, 2^-6 4.6e-4 / 2.9e-4, 2^-10 5.9e-3 / 3.4e-4 (rounding the result alone: 2.6e-4); of all three,
// 131,072 keys a row: 1.3e-3 / 3.4e-4.  bf16 has fp32's range.
constexpr int kPShift = 6;  // a weight is normal down to 2^-20; some room above 1
struct GradScale {
  float u;   // of dP and D, beside the 2^kPShift that P brings
  float p;   // of dV's sum
  float ds;  // of dQ's and dK's sums
};
template <bool BF16>
__device__ __forceinline__ GradScale grad_scale(const BwdParams& p, int plane) {
  if constexpr (BF16) return {1.0f, 1.0f, 1.0f};
  const uint4 w = __ldcg(reinterpret_cast<const uint4*>(p.range) + plane);
  const float bound = p.scale * __uint_as_float(w.x) * __uint_as_float(w.z) + __uint_as_float(w.y);
  int t = 0;  // a plane of zeros, or one that is not finite
  if (bound > 0.0f && bound < INFINITY) t = 14 - (static_cast<int>(__float_as_uint(bound) >> 23) - 127);
  t = max(-80, min(t, 80));
  return {__uint_as_float(static_cast<uint32_t>(127 + t - kPShift) << 23),
          __uint_as_float(static_cast<uint32_t>(127 - kPShift) << 23),
          __uint_as_float(static_cast<uint32_t>(127 - t) << 23)};
}

// Window variant: the query tiles [qt_lo, qt_hi) that see key tile kt.  A tile with a sink is seen
// from its diagonal to the last row, any other until the window has passed its last key.
__host__ __device__ inline void window_q_tiles(int kt, int n_qtiles, int off, int window, int sinks,
                                               int& qt_lo, int& qt_hi) {
  const long long first = static_cast<long long>(kt) * 128 - off;
  const long long last = first + 127 + window;
  qt_lo = first > 0 ? static_cast<int>(first / 128) : 0;
  if (qt_lo > n_qtiles) qt_lo = n_qtiles;
  long long hi = last >= 0 ? last / 128 + 1 : 0;
  if (static_cast<long long>(kt) * 128 < sinks || hi > n_qtiles) hi = n_qtiles;
  qt_hi = hi > qt_lo ? static_cast<int>(hi) : qt_lo;
}

__device__ __forceinline__ bool ew_wait(uint32_t bar, uint32_t parity, volatile int* abort,
                                        int* status) {
  const bool ok = wait_bounded(bar, parity, abort, status);
  return __all_sync(0xffffffffu, ok);
}

// Columns [c0, c1) (multiples of 32) of row r of a 128 x D accumulator, times mul where the operands are
// fp16 (a power of two; 1 for bf16), as 16-bit values in a tile of
// shared memory (64-column sub-tiles kSub apart, 128-byte swizzle), from where TMA stores take the rows
// that exist: written to memory by the threads that hold them, a warp's stores would touch 32 lines each
// (a block's end took a microsecond longer).
template <bool BF16>
__device__ __forceinline__ void stage_acc_row(uint32_t row_tmem_col, uint8_t* tile, int r, int c0, int c1,
                                              [[maybe_unused]] float mul) {
#pragma unroll 1
  for (int c = c0 / 32; c < c1 / 32; ++c) {
    uint32_t a[32];
    tmem_ld32(row_tmem_col + c * 32, a);
    tmem_wait_ld();
    if constexpr (!BF16) {
#pragma unroll
      for (int e = 0; e < 32; ++e) a[e] = __float_as_uint(__uint_as_float(a[e]) * mul);
    }
    uint8_t* sub = tile + (c >> 1) * kSub;
#pragma unroll
    for (int q4 = 0; q4 < 4; ++q4)
      *reinterpret_cast<uint4*>(sub + sw128(r, (c & 1) * 4 + q4)) =
          make_uint4(pack2<BF16>(__uint_as_float(a[8 * q4 + 0]), __uint_as_float(a[8 * q4 + 1])),
                     pack2<BF16>(__uint_as_float(a[8 * q4 + 2]), __uint_as_float(a[8 * q4 + 3])),
                     pack2<BF16>(__uint_as_float(a[8 * q4 + 4]), __uint_as_float(a[8 * q4 + 5])),
                     pack2<BF16>(__uint_as_float(a[8 * q4 + 6]), __uint_as_float(a[8 * q4 + 7])));
  }
}

// A staged tile out to rows row0 .. of plane z (one thread; the stages' writes fenced before).
template <int D>
__device__ __forceinline__ void store_staged(const CUtensorMap* m, uint32_t tile, int row0, int z) {
#pragma unroll
  for (int sub = 0; sub < D / 64; ++sub) tma_store_3d(m, tile + sub * kSub, sub * 64, row0, z);
  tma_store_commit();
  tma_store_wait_read0();  // the block's shared memory may go
}

// Row of a 128 x D accumulator as fp32 values (zeros for an accumulator nothing was added to); mul as
// above.
template <int D, bool BF16>
__device__ __forceinline__ void store_part_row(uint32_t row_tmem_col, float* dst, bool any,
                                               [[maybe_unused]] float mul) {
#pragma unroll 1
  for (int c = 0; c < D / 32; ++c) {
    uint32_t a[32];
    if (any) {
      tmem_ld32(row_tmem_col + c * 32, a);
      tmem_wait_ld();
      if constexpr (!BF16) {
#pragma unroll
        for (int e = 0; e < 32; ++e) a[e] = __float_as_uint(__uint_as_float(a[e]) * mul);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 32; ++e) a[e] = 0;
    }
    uint4* out = reinterpret_cast<uint4*>(dst + c * 32);
#pragma unroll
    for (int e = 0; e < 8; ++e) out[e] = make_uint4(a[4 * e], a[4 * e + 1], a[4 * e + 2], a[4 * e + 3]);
  }
}

// 32 scores of a row: kept where their column (less col0) lies in [lo, hi] or is at most sk, -inf
// elsewhere.  By bits, so that a NaN or infinite score of a masked pair leaves no trace; called from a
// branch of its own, where a test per column in the exponential loop would cost every tile.
__device__ __forceinline__ void mask32(uint32_t (&s)[32], int col0, int lo, int hi, int sk) {
  const int a = max(lo - col0, 0), b = min(hi - col0, 31), c = min(sk - col0, 31);
  uint32_t vis = (a > b) ? 0u : ((0xffffffffu >> (31 - b)) & (0xffffffffu << a));
  vis |= (c < 0) ? 0u : (0xffffffffu >> (31 - c));
#pragma unroll
  for (int e = 0; e < 32; ++e) s[e] = (vis & (1u << e)) ? s[e] : 0xff800000u;
}

template <int D>
__device__ __forceinline__ void store_zero_row(uint16_t* dst) {
  uint4* out = reinterpret_cast<uint4*>(dst);
#pragma unroll
  for (int c = 0; c < D / 8; ++c) out[c] = make_uint4(0, 0, 0, 0);
}

// K-major A (128 rows x D, 64-column sub-tiles A_SUB bytes apart) x K-major B^T (N rows x D,
// sub-tiles B_SUB apart): D[128 x N] = A B^T, from the descriptors of the operands' first K
// step: a descriptor's start address field counts 16-byte units, so a later K step's
// descriptor is the first one plus a constant (the issuing thread builds two descriptors per
// product instead of two per MMA).
template <int D, uint32_t A_SUB, uint32_t B_SUB>
__device__ __forceinline__ void mma_rows_rows_d(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                                uint32_t idesc) {
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk)
    mma_ss(d_tmem, a_desc + (((kk >> 2) * A_SUB + (kk & 3) * 32) >> 4),
           b_desc + (((kk >> 2) * B_SUB + (kk & 3) * 32) >> 4), idesc, kk > 0 ? 1u : 0u);
}

// A [128 x K] in tensor memory as 16-bit pairs (K / 2 columns from a_tmem) times B [K rows x D]
// in shared memory read MN-major, from the descriptor of its first 16 rows: D[128 x D] (+)= A B.
template <int K>
__device__ __forceinline__ void mma_tmem_rows_d(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                                uint32_t idesc, bool accumulate) {
#pragma unroll
  for (int kk = 0; kk < K / 16; ++kk)
    mma_ts(d_tmem, a_tmem + kk * 8, b_desc + ((kk * 16 * 128) >> 4), idesc,
           (accumulate || kk > 0) ? 1u : 0u);
}

// d = 64 under a window: the gradient kernels with two blocks on an SM (attn_bwd_window.cu), and
// whether a call's dK/dV and dQ take them.
bool bwd_window_two_kv(const BwdArgs& a);
bool bwd_window_two_q(const BwdArgs& a);
int launch_bwd_window_dkdv(const BwdArgs& a, const BwdParams& p, unsigned blocks, cudaStream_t stream);
int launch_bwd_window_dq(const BwdArgs& a, const BwdParams& p, unsigned blocks, cudaStream_t stream);

}  // namespace attn
