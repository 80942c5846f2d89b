// What the kernels that write and read the 8-bit and the 4-bit cache share.
#pragma once
#include "internal.h"
#include "ptx.cuh"

namespace attn {

constexpr int kCacheThreads = 256;
constexpr int kMaxRun = 64;  // tokens of a block

// Magnitudes of a 16-bit pair, and the larger of two pairs (a NaN stays one).
template <bool BF16>
__device__ __forceinline__ uint32_t max_abs2(uint32_t a, uint32_t b) {
  uint32_t r;
  if constexpr (BF16)
    asm("{\n\t.reg .b32 t;\n\tabs.bf16x2 t, %2;\n\tmax.NaN.bf16x2 %0, %1, t;\n\t}" : "=r"(r) : "r"(a), "r"(b));
  else
    asm("{\n\t.reg .b32 t;\n\tabs.f16x2 t, %2;\n\tmax.NaN.f16x2 %0, %1, t;\n\t}" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

template <bool BF16>
__device__ __forceinline__ void unpack8(const uint4 w, float* v) {
  const uint32_t h[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (BF16) {
      v[2 * i] = __uint_as_float(h[i] << 16);
      v[2 * i + 1] = __uint_as_float(h[i] & 0xffff0000u);
    } else {
      asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\t"
          "cvt.f32.f16 %1, b;\n\t}"
          : "=f"(v[2 * i]), "=f"(v[2 * i + 1])
          : "r"(h[i]));
    }
  }
}

// The sequence that owns packed row i (cu[b] <= i < cu[b + 1]); i lies in [cu[0], cu[B]).
__device__ __forceinline__ int find_sequence(const int32_t* cu, int B, int i) {
  int lo = 0, hi = B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (cu[mid] <= i)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

// Tokens of a block: short runs while there are few tokens, so that they spread over the SMs.
inline int cache_run(int total) {
  const int want = total / (152 * 8);
  return want < 1 ? 1 : want > kMaxRun ? kMaxRun : want;
}

}  // namespace attn
