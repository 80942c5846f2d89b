// Attention of a few query rows (up to 16 per key/value head) on warp-level matrix tiles: the state
// of one warp and the merges of warps and of a cluster's blocks.  Used by the split kernels over the
// 8-bit cache and over the paged cache for a few new tokens.
//
// A warp takes sixteen keys at a time and NT column tiles of eight query rows each:
//   S^T = K Q^T   keys by rows, so that up to eight rows fill a tile's columns (rows by keys would
//                 leave half of a sixteen-row tile empty); thread (g, c) = (lane / 4, lane % 4)
//                 holds keys g and g + 8 of rows 2c and 2c + 1 of each column tile;
//   O^T += V^T P^T   channels by rows, P^T being the transpose of what the thread holds (movmatrix);
//                 tile t holds two channels of thread (g, c) for the same two rows.
//
// P is rounded to the 16 bits of the second product's other operand (half a step of each weight); the row
// sums take the unrounded weights, and scores, statistics and O are fp32.
#pragma once
#include "ptx.cuh"

namespace attn {

constexpr int kMaxCluster = 8;  // blocks of a portable cluster

// Transpose of an 8 x 8 matrix of 16-bit values held as the matrix instructions hold them.
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

template <int D, int NT, bool BF16_MMA>
struct RowState {
  float m[NT][2], l[NT][2];  // running maximum (log2 units); partial sum over this thread's keys
  float o[NT][D / 16][4];

  __device__ __forceinline__ void init() {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      m[n][0] = m[n][1] = -INFINITY;
      l[n][0] = l[n][1] = 0.0f;
#pragma unroll
      for (int t = 0; t < D / 16; ++t) o[n][t][0] = o[n][t][1] = o[n][t][2] = o[n][t][3] = 0.0f;
    }
  }

  // Online softmax over sixteen keys: x[n][k][r] the score of key g + 8k and row 2c + r (log2 units,
  // -inf where masked).  Rescales the state and gives the weights as the second operand of the next
  // product.
  __device__ __forceinline__ void step(const float (&x)[NT][2][2], uint32_t (&pb)[NT][2]) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float p[2][2], a[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float mx = fmaxf(x[n][0][r], x[n][1][r]);
#pragma unroll
        for (int sh = 4; sh < 32; sh <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, sh));
        const float mn = fmaxf(m[n][r], mx);
        a[r] = (m[n][r] == -INFINITY) ? 0.f : ex2(m[n][r] - mn);
        const float mu = (mn == -INFINITY) ? 0.f : mn;
        m[n][r] = mn;
        l[n][r] *= a[r];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          p[k][r] = ex2(x[n][k][r] - mu);
          l[n][r] += p[k][r];
        }
      }
      if (__any_sync(0xffffffffu, a[0] != 1.0f || a[1] != 1.0f)) {
#pragma unroll
        for (int t = 0; t < D / 16; ++t) {
          o[n][t][0] *= a[0];
          o[n][t][1] *= a[1];
          o[n][t][2] *= a[0];
          o[n][t][3] *= a[1];
        }
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) pb[n][k] = transpose_8x8(pack2<BF16_MMA>(p[k][0], p[k][1]));
    }
  }

  __device__ __forceinline__ void finish() {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int sh = 4; sh < 32; sh <<= 1) l[n][r] += __shfl_xor_sync(0xffffffffu, l[n][r], sh);
  }

  // The state to the warp's part of the merge scratch, [row][D + 2]; channel(t, i) is the channel
  // of the thread's i-th row of tile t, value(n, r, x) what is stored for x of row 2c + r of tile n.
  template <typename F, typename V>
  __device__ __forceinline__ void store(float* rw, int rows, int lane, F channel, V value) const {
    const int g = lane >> 2, c = lane & 3;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int row = n * 8 + 2 * c + r;
        if (row >= rows) continue;
        float* dst = rw + row * (D + 2);
#pragma unroll
        for (int t = 0; t < D / 16; ++t) {
          dst[channel(t, 0)] = value(n, r, o[n][t][r]);
          dst[channel(t, 1)] = value(n, r, o[n][t][2 + r]);
        }
        if (g == 0) {
          dst[D] = m[n][r];
          dst[D + 1] = l[n][r];
        }
      }
  }
};

// Where the block's rows go: partial states of split `split` of n_splits in the workspace, or, with
// the splits of a row as one cluster's blocks, the rows themselves.
struct RowsOut {
  float* ws_o;   // [row, n_splits, D] normalised
  float* ws_ml;  // [row, n_splits, 2]
  uint16_t* out;  // [row, D]
  float* lse;     // [row]
  int n_splits, split;
  bool cluster;
};

// Merges the states of WARPS warps (red: [warp][MAXR][D + 2]) for `rows` rows and writes them out;
// every one of the WARPS * 32 threads calls it, after the last of them has stored its state and a
// barrier.  fin: shared scratch of MAXR (D + 2) floats at the same address in every block.  ok: the
// block's state is sound; any: it has keys.  NORM: the stored rows are divided by their sums already.
// grow(row): the output row.
template <int D, bool BF16, int WARPS, int MAXR, bool NORM, typename F>
__device__ __forceinline__ void merge_rows(const float* red, float* fin, int rows, bool ok, bool any,
                                           const RowsOut& w, F grow) {
  constexpr int kRow = D + 2;
  if (ok || w.cluster) {
    for (int i = threadIdx.x; i < rows * D; i += WARPS * 32) {
      const int row = i / D, col = i % D;
      float mm = -INFINITY;
#pragma unroll
      for (int u = 0; u < WARPS; ++u) mm = fmaxf(mm, red[(u * MAXR + row) * kRow + D]);
      float ll = 0.f, acc = 0.f;
#pragma unroll
      for (int u = 0; u < WARPS; ++u) {
        const float mw = red[(u * MAXR + row) * kRow + D];
        const float lw = red[(u * MAXR + row) * kRow + D + 1];
        // (no key: weight 0; a NaN sum stays one)
        const float wgt = (mw == -INFINITY) ? (lw == 0.f ? 0.f : lw) : ex2(mw - mm);
        ll += wgt * lw;
        acc += (NORM ? wgt * lw : wgt) * red[(u * MAXR + row) * kRow + col];
      }
      const float o = ll == 0.f ? 0.f : acc / ll;
      if (w.cluster) {
        const bool use = ok && any;
        fin[row * D + col] = use ? o : 0.0f;
        if (col == 0) {
          fin[MAXR * D + row * 2] = use ? mm : -INFINITY;
          fin[MAXR * D + row * 2 + 1] = use ? ll : 0.0f;
        }
      } else {
        const size_t part = grow(row) * w.n_splits + w.split;
        w.ws_o[part * D + col] = o;
        if (col == 0) {
          w.ws_ml[part * 2] = mm;
          w.ws_ml[part * 2 + 1] = ll;
        }
      }
    }
  }
  if (!w.cluster) return;
  // block `split` of n_splits writes every n_splits-th stretch of the rows
  __syncwarp();
  cluster_sync();
  const int n = w.n_splits;
  const uint32_t fin_u = smem_u32(fin);
  for (int i = w.split * (WARPS * 32) + threadIdx.x; i < rows * D; i += n * WARPS * 32) {
    const int row = i / D, col = i % D;
    float ms[kMaxCluster], mm = -INFINITY;
#pragma unroll
    for (int s = 0; s < kMaxCluster; ++s) {
      ms[s] = s < n ? ld_cluster_f32(fin_u + (MAXR * D + row * 2) * 4, s) : -INFINITY;
      mm = fmaxf(mm, ms[s]);
    }
    float ll = 0.f, acc = 0.f;
#pragma unroll
    for (int s = 0; s < kMaxCluster; ++s) {
      if (s >= n) break;
      const float ls = ld_cluster_f32(fin_u + (MAXR * D + row * 2 + 1) * 4, s);
      const float wgt = ms[s] == -INFINITY ? ls : ex2(ms[s] - mm) * ls;
      ll += wgt;
      acc += wgt * ld_cluster_f32(fin_u + i * 4, s);
    }
    const size_t orow = grow(row);
    w.out[orow * D + col] =
        static_cast<uint16_t>(pack2<BF16>(ll == 0.0f ? 0.0f : acc / ll, 0.0f) & 0xffffu);
    if (col == 0) w.lse[orow] = ll == 0.0f ? -INFINITY : (mm + lg2(ll)) * 0.69314718055994531f;
  }
  __syncwarp();
  cluster_sync();  // no block leaves while another reads its shared memory
}

// Keys of a split, in multiples of 64, for `pairs` (sequence, head) pairs of at most `tokens` keys
// when `slots` blocks run at a time: as many splits as fill one round of blocks, at least 128 keys
// each; where that leaves over 2,048 keys, equal splits of at most 2,048 in several rounds.  A block
// costs 4-5 us besides its keys (it reads its lengths, then its pages, then the first stage), which
// speaks for long splits, the last round's idle blocks for short ones.  Measured with at most
// 1,024 / 2,048 / 4,096 keys, us: the 8-bit decode of 64 sequences of 1k-32k tokens (Hq=64 Hkv=8
// d=128) 406 / 398 / 475, one 16-bit token of the same 623 / 594 / 703, of 32 sequences of 2k-4k 76 /
// 64 / 62, one token under a 4,095-key window (16 sequences, Hkv=8, d=64) 35 / 26 / 27.
inline int row_split_tokens(long long pairs, long long tokens, int slots) {
  long long n = pairs > 0 && slots / pairs > 1 ? slots / pairs : 1;
  if ((tokens + n - 1) / n > 2048) n = (tokens + 2047) / 2048;
  long long per = (tokens + n - 1) / n;
  per = (per + 63) / 64 * 64;
  return static_cast<int>(per < 128 ? 128 : per);
}

}  // namespace attn
