// Prefill under a sliding window whose first keys (sinks) stay visible: the launcher of the kernel with
// two blocks on an SM (attn_fwd_two.cuh).
#include "attn_fwd_two.cuh"

namespace attn {

template <int D, bool BF16>
static int launch_window_variant(const FwdArgs& a, cudaStream_t stream) {
  using L = WinLayout<D>;
  const uint64_t bhq = static_cast<uint64_t>(a.B) * a.Hq;
  const uint64_t bhk = static_cast<uint64_t>(a.B) * a.Hkv;
  const uint64_t rb = static_cast<uint64_t>(D) * 2;
  CUtensorMap tq, tk, tv, to;
  if (!make_tmap_3d(&tq, a.q, BF16, D, a.N_q, bhq, rb, rb * a.N_q, 64, kWM, 1) ||
      !make_tmap_3d(&tk, a.k, BF16, D, a.N_kv, bhk, rb, rb * a.N_kv, 64, kWN, 1) ||
      !make_tmap_3d(&tv, a.v, BF16, D, a.N_kv, bhk, rb, rb * a.N_kv, 64, kWN, 1) ||
      !make_tmap_3d(&to, a.o, BF16, D, a.N_q, bhq, rb, rb * a.N_q, 64, kWM, 1))
    return -5;
  WinParams p;
  p.o = a.o;
  p.lse = a.lse;
  p.status = device_status_ptr();
  if (!p.status) return -5;
  p.Hq = a.Hq;
  p.Hkv = a.Hkv;
  p.G = a.Hq / a.Hkv;
  p.N_q = a.N_q;
  p.N_kv = a.N_kv;
  p.n_qtiles = (a.N_q + kWM - 1) / kWM;
  const uint64_t blocks = static_cast<uint64_t>(p.n_qtiles) * bhq;
  if (blocks > 0x7fffffffull) return -2;
  p.BH = static_cast<int>(bhq);
  uint64_t planes = (64ull << 20) / (2ull * a.N_kv * D * 2);  // about half of L2
  if (planes < 1) planes = 1;
  const uint64_t heads = planes * p.G;
  p.head_group = static_cast<int>(heads < bhq ? heads : bhq);
  p.window = a.window;
  p.sinks = a.sinks;
  p.sl2 = a.scale * 1.4426950408889634f;
  auto kern = attn_fwd_two_kernel<D, BF16, false>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kBytes) !=
      cudaSuccess)
    return -5;
  kern<<<static_cast<unsigned>(blocks), two_threads(false), L::kBytes, stream>>>(tq, tk, tv, to, p);
  return cudaGetLastError() == cudaSuccess ? 0 : -5;
}

// This kernel against the prefill kernel's sinks variant, us (bf16, 4 sinks):
//   more query tiles than SMs   B=1 Hq=64 Hkv=8 N=8192 d=128: W=0 99 / 146, 1024 248 / 334, 4096 594 /
//                               667, 8192 762 / 828; B=1 Hq=16 Hkv=4 N=8192 d=64: W=256 35 / 58, 8192
//                               156 / 192; B=4 H=16 N=1024 d=128: W=256 19 / 31
//   fewer (one block an SM)     B=1 Hq=Hkv=4 N=4096 d=128: W=256 9.5 / 11.9, 512 11.9 / 13.5, 1024 16.8 /
//                               16.4, 4096 43 / 32; d=64: W=512 10.8 / 12.4, 1024 14.9 / 15.0, 2048 23 / 21
bool window_sinks_short(const FwdArgs& a) {
  const long long items = static_cast<long long>(a.B) * a.Hq * ((a.N_q + kWM - 1) / kWM);
  long long keys = static_cast<long long>(a.window) + kWM + a.sinks;  // a query tile sees
  if (keys > a.N_kv) keys = a.N_kv;
  return items > 152 || keys <= 1024;
}

int launch_attn_fwd_window_sinks(const FwdArgs& a, cudaStream_t stream) {
  if (a.d == 64)
    return a.bf16 ? launch_window_variant<64, true>(a, stream)
                  : launch_window_variant<64, false>(a, stream);
  return a.bf16 ? launch_window_variant<128, true>(a, stream)
                : launch_window_variant<128, false>(a, stream);
}

}  // namespace attn
