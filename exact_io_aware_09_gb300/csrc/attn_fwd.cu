// Launchers of the prefill forward kernel (attn_fwd_kernel.cuh): the dense, sliding-window,
// block-sparse and FP8 variants.
#include <atomic>

#include "attn_fwd_kernel.cuh"

namespace attn {

// O = 0 and L = -inf for every row (used when there is no key at all).
template <bool BF16>
__global__ void attn_empty_rows_kernel(uint16_t* o, float* lse, size_t rows, int d) {
  const size_t i = blockIdx.x * static_cast<size_t>(blockDim.x) + threadIdx.x;
  if (i < rows * d) o[i] = 0;
  if (i < rows) lse[i] = -INFINITY;
}

template <int D, bool BF16, int KS, int VS, bool FP8 = false, bool SINKS = false>
static int launch_fwd_variant(const FwdArgs& a, cudaStream_t stream) {
  using L = FwdLayout<D, KS, VS, FP8>;
  CUtensorMap tq, tk, tv, to;
  const uint64_t bhq = static_cast<uint64_t>(a.B) * a.Hq;
  const uint64_t bhk = static_cast<uint64_t>(a.B) * a.Hkv;
  const uint64_t rq = static_cast<uint64_t>(D) * 2, rk = rq;
  if constexpr (FP8) {
    // E4M3 codes: Q and K rows of d bytes (one 128-byte swizzle chunk at d = 128); V^T rows of
    // nkvp keys, loaded as d x 128-key tiles
    if (!make_tmap_3d_u8(&tq, a.q8, D, a.N_q, bhq, D, static_cast<uint64_t>(D) * a.N_q, D, kBlockM, 1) ||
        !make_tmap_3d_u8(&tk, a.k8, D, a.N_kv, bhk, D, static_cast<uint64_t>(D) * a.N_kv, D, kBlockN, 1) ||
        !make_tmap_3d_u8(&tv, a.vt8, a.nkvp, D, bhk, a.nkvp, static_cast<uint64_t>(a.nkvp) * D,
                         kBlockN, D, 1))
      return -5;
  } else {
    if (!make_tmap_3d(&tq, a.q, BF16, D, a.N_q, bhq, rq, rq * a.N_q, 64, kBlockM, 1) ||
        !make_tmap_3d(&tk, a.k, BF16, D, a.N_kv, bhk, rk, rk * a.N_kv, 64, kBlockN, 1) ||
        !make_tmap_3d(&tv, a.v, BF16, D, a.N_kv, bhk, rk, rk * a.N_kv, 64, kBlockN, 1))
      return -5;
  }
  if (!make_tmap_3d(&to, a.o, BF16, D, a.N_q, bhq, rq, rq * a.N_q, 64, kBlockM, 1)) return -5;
  typename FwdParamsOf<SINKS, false>::T p;
  p.o = a.o;
  p.lse = a.lse;
  p.status = device_status_ptr();
  p.Hq = a.Hq;
  p.Hkv = a.Hkv;
  p.N_q = a.N_q;
  p.N_kv = a.N_kv;
  p.n_qtiles = (a.N_q + kBlockM - 1) / kBlockM;
  p.group = a.Hq / a.Hkv;
  p.causal = (a.causal || a.window >= 0) ? 1 : 0;
  p.window = a.window;
  if constexpr (SINKS) p.sinks = a.sinks;
  p.n_kvtiles = (a.N_kv + kBlockN - 1) / kBlockN;
  p.block_mask = a.block_mask;
  p.q_scale = a.q_scale;
  p.k_scale = a.k_scale;
  p.v_scale = a.v_scale;
  p.BH = static_cast<int>(bhq);
  {
    // Query heads whose K/V planes fill about half of L2, a multiple of the heads sharing one
    // key/value plane.
    static int l2_bytes = -1;
    if (l2_bytes < 0) {
      int dev = 0, v = 0;
      if (cudaGetDevice(&dev) != cudaSuccess ||
          cudaDeviceGetAttribute(&v, cudaDevAttrL2CacheSize, dev) != cudaSuccess || v <= 0)
        v = 64 << 20;
      l2_bytes = v;
    }
    const uint64_t plane_bytes = 2ull * a.N_kv * D * L::kElem;
    uint64_t planes = (static_cast<uint64_t>(l2_bytes) / 2) / plane_bytes;
    if (planes < 1) planes = 1;
    uint64_t heads = planes * static_cast<uint64_t>(a.Hq / a.Hkv);
    if (heads > bhq) heads = bhq;
    p.head_group = static_cast<int>(heads);
  }
  p.sl2 = a.scale * 1.4426950408889634f;
  if (!p.status) return -5;
  auto kern = attn_fwd_kernel<D, BF16, KS, VS, FP8, SINKS>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kBytes) !=
      cudaSuccess)
    return -5;
  // One block per work item; the running blocks take over the items of the others.
  const uint64_t blocks = static_cast<uint64_t>(p.n_qtiles) * bhq;
  if (blocks > 0x7fffffffull) return -2;
  kern<<<static_cast<unsigned>(blocks), kFwdThreads, L::kBytes, stream>>>(tq, tk, tv, to, p);
  return cudaGetLastError() == cudaSuccess ? 0 : -5;
}

#ifdef ATTN_FWD_TRACE
}  // namespace attn
extern "C" int attn_fwd_trace_copy(void* dst) {
  return static_cast<int>(cudaMemcpyFromSymbol(dst, attn::g_fwd_trace, sizeof(attn::g_fwd_trace)));
}
namespace attn {
#endif

static std::atomic<int> g_d64_mode{0};

int set_d64_kernel(int mode) {
  if (mode < 0 || mode > 2) return -1;
  return g_d64_mode.exchange(mode);
}

int launch_attn_fwd_fp8_kernel(const FwdArgs& a, cudaStream_t stream) {
  if (a.d != 128) return -2;
  return a.bf16 ? launch_fwd_variant<128, true, 4, 4, true>(a, stream)
                : launch_fwd_variant<128, false, 4, 4, true>(a, stream);
}

int launch_attn_fwd(const FwdArgs& a, cudaStream_t stream) {
  if (a.B == 0 || a.N_q == 0) return 0;
  if (a.N_kv == 0) {
    const size_t rows = static_cast<size_t>(a.B) * a.Hq * a.N_q;
    const size_t n = rows * a.d;
    const unsigned blocks = static_cast<unsigned>((n + 255) / 256);
    if (a.bf16)
      attn_empty_rows_kernel<true><<<blocks, 256, 0, stream>>>(static_cast<uint16_t*>(a.o), a.lse, rows, a.d);
    else
      attn_empty_rows_kernel<false><<<blocks, 256, 0, stream>>>(static_cast<uint16_t*>(a.o), a.lse, rows, a.d);
    return cudaGetLastError() == cudaSuccess ? 0 : -5;
  }
  if (a.sinks >= 0) {
    // the window with first keys that stay visible
    if (window_sinks_short(a)) return launch_attn_fwd_window_sinks(a, stream);
    if (a.d == 64)
      return a.bf16 ? launch_fwd_variant<64, true, 4, 4, false, true>(a, stream)
                    : launch_fwd_variant<64, false, 4, 4, false, true>(a, stream);
    if (a.d == 128)
      return a.bf16 ? launch_fwd_variant<128, true, 3, 2, false, true>(a, stream)
                    : launch_fwd_variant<128, false, 3, 2, false, true>(a, stream);
    return -2;
  }
  if (a.d == 64) {
    // Two query tiles per item when there are more query tiles than SMs (so that the pairs
    // still cover every SM), else one.
    const int mode = g_d64_mode.load();
    bool pair = (mode == 1);
    if (mode == 0) {
      const uint64_t tiles = static_cast<uint64_t>(a.B) * a.Hq * ((a.N_q + kBlockM - 1) / kBlockM);
      int dev = 0, n_sm = 0;
      if (cudaGetDevice(&dev) != cudaSuccess ||
          cudaDeviceGetAttribute(&n_sm, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return -5;
      pair = tiles > static_cast<uint64_t>(n_sm);
    }
    if (pair) return launch_attn_fwd_pair(a, stream);
    return a.bf16 ? launch_fwd_variant<64, true, 4, 4>(a, stream)
                  : launch_fwd_variant<64, false, 4, 4>(a, stream);
  }
  if (a.d == 128)
    return a.bf16 ? launch_fwd_variant<128, true, 3, 2>(a, stream)
                  : launch_fwd_variant<128, false, 3, 2>(a, stream);
  return -2;
}

}  // namespace attn
