// The tensor-core attention kernel of lowbit_prefix_attention.
#include "paged_attn_tc.cuh"

namespace lowbit {

cudaError_t launch_attention_tc(const PrefixArgs& a, int D, bool fp8, bool pair, cudaStream_t s) {
  return launch_tc_by_dim(a, D, fp8, pair, s);
}

}  // namespace lowbit
