// A chunk of new tokens of each sequence over a paged cache held in 4 bits (fp4.cuh), with more rows per
// key/value head than the few-row kernel (attn_paged_fp4.cu) takes.
//
// The kernel of chunks over the 16-bit cache (attn_fwd_two.cuh: two blocks an SM, 64-key steps, products on
// the tensor cores) whose two producer warps turn codes into f16 operands in shared memory instead of
// copying rows: code * scale is exact in f16, so nothing but the weights is rounded before a product.
#include "attn_paged.cuh"

namespace attn {

int launch_attn_fp4_chunk(const PagedArgs& a, const CacheFp4& c, cudaStream_t stream) {
  if (a.d == 64)
    return a.bf16 ? launch_paged_variant<64, true, true>(a, &c, stream)
                  : launch_paged_variant<64, false, true>(a, &c, stream);
  return a.bf16 ? launch_paged_variant<128, true, true>(a, &c, stream)
                : launch_paged_variant<128, false, true>(a, &c, stream);
}

int fp4_chunk_splits(int B, int Hq, int Hkv, int max_q, int max_k, int window, int sinks, int d) {
  return paged_split(B, Hq, Hkv, max_q, max_k, window, sinks, d).n_splits;
}

}  // namespace attn
