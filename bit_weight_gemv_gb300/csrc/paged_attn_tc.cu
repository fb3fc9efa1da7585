// The tensor-core attention kernel of lowbit_paged_attention.
#include "paged_attn_tc.cuh"

namespace lowbit {

// True where the kernel can run: heads of 64 or 128, pages that TMA can box.
bool attention_tc_fits(const AttnArgs& a, int D) { return D <= 128 && a.p.page_mask + 1 >= 16; }

cudaError_t launch_attention_tc(const AttnArgs& a, int D, bool fp8, bool pair, cudaStream_t s) {
  return launch_tc_by_dim(a, D, fp8, pair, s);
}

}  // namespace lowbit
