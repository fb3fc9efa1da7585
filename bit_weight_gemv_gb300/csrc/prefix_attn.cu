// lowbit_prefix_attention: attention of requests whose first pages are the same ones.
//
// With the keys of a row cut into the shared ones and its own, (m, l, o) of each part (paged_attn_mma.cuh) join
// as any two sets of keys do.  So the shared part is computed with all rows of a group as one request without
// a mask, which reads its keys and values once for the group, and the rows wait in the workspace, 4 (D + 2) bytes
// each; then the own part, whose way out joins them.  The same kernels and schedule as lowbit_paged_attention
// do both, each chosen by the rows that share a "request's" keys in its part.
#include "paged_attn_mma.cuh"

namespace lowbit {

cudaError_t launch_attention_mma(const PrefixArgs& a, int D, bool fp8, cudaStream_t s) { return launch_by_dim(a, D, fp8, s); }
cudaError_t launch_combine(const PrefixArgs& a, int D, cudaStream_t s) { return launch_join(a, D, s); }

}  // namespace lowbit

using namespace lowbit;

extern "C" {

size_t lowbit_prefix_attention_workspace_bytes(int T, int B, int Hq, int Hk, int D) {
  if (lowbit_paged_attention_workspace_bytes(T, B, Hq, Hk, D) == 0) return 0;
  return 2 * pieces_bytes(D) + (size_t)T * (size_t)Hq * (size_t)(D + 2) * sizeof(float);
}

lowbit_status lowbit_prefix_attention(const uint16_t* q, int64_t q_stride, int Hq, const lowbit_paged_batch* batch,
                                      const lowbit_paged_cache* cache, const int32_t* cu_groups,
                                      const int32_t* prefix_lens, int groups, float scale, int causal, uint16_t* out,
                                      float* lse, void* workspace, size_t ws_bytes, void* stream) {
  PrefixArgs a = {};
  const lowbit_status st = make_attn_args(q, q_stride, Hq, batch, cache, scale, causal, 0, out, lse, &a);
  if (st != LOWBIT_OK) return st;
  if (!cu_groups || !prefix_lens) return LOWBIT_ERR_INVALID_ARG;
  if (groups < 1 || groups > kMaxBatch) return LOWBIT_ERR_SHAPE;
  if (((uintptr_t)cu_groups | (uintptr_t)prefix_lens) & 3) return LOWBIT_ERR_ALIGN;
  if (a.p.T == 0) return LOWBIT_OK;
  const int D = cache->head_dim;
  if (!workspace || ws_bytes < lowbit_prefix_attention_workspace_bytes(a.p.T, a.p.B, Hq, cache->heads, D))
    return LOWBIT_ERR_WORKSPACE;
  if ((uintptr_t)workspace & 15) return LOWBIT_ERR_ALIGN;
  a.p.err = device_error_word();
  if (!a.p.err) return LOWBIT_ERR_CUDA;
  a.wide = (((uintptr_t)out | (uintptr_t)workspace) & 31) == 0;
  a.groups = groups;
  a.requests = a.p.B;
  a.cu_groups = cu_groups;
  a.prefix_lens = prefix_lens;
  a.base_o = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + 2 * pieces_bytes(D));
  a.base_ml = reinterpret_cast<float2*>(a.base_o + (size_t)a.p.T * (size_t)Hq * (size_t)D);
  const bool fp8 = cache->dtype == LOWBIT_CACHE_E4M3;
  cudaStream_t s = static_cast<cudaStream_t>(stream);

  PrefixArgs shared = a;
  shared.shared = true;
  shared.p.B = groups;
  shared.shape.causal = 0;
  use_pieces(&shared, workspace, D);
  cudaError_t e = launch_attention(shared, D, fp8, s);
  if (e != cudaSuccess) return LOWBIT_ERR_CUDA;
  use_pieces(&a, static_cast<uint8_t*>(workspace) + pieces_bytes(D), D);
  e = launch_attention(a, D, fp8, s);
  return e == cudaSuccess ? LOWBIT_OK : LOWBIT_ERR_CUDA;
}

}  // extern "C"
