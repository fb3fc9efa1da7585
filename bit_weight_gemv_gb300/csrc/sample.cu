// lowbit_sample: its checks; the kernel is in sample.cuh.
#include "sample.cuh"

using namespace lowbit;

extern "C" lowbit_status lowbit_sample(const void* logits, int dtype, int64_t row_stride, int M, int V,
                                       const float* temperature, const int32_t* top_k,
                                       const float* top_p, const float* min_p, const float* u,
                                       const int32_t* id_map, int32_t* ids, float* logprob,
                                       int32_t* kept, void* stream) {
  if (!logits || !u || !ids || (dtype != LOWBIT_LOGITS_FP32 && dtype != LOWBIT_LOGITS_BF16))
    return LOWBIT_ERR_INVALID_ARG;
  if (M < 1 || M > (1 << 24) || V < 1 || V > kMaxVocab || row_stride < V) return LOWBIT_ERR_SHAPE;
  const uintptr_t words = (uintptr_t)temperature | (uintptr_t)top_k | (uintptr_t)top_p | (uintptr_t)min_p |
                          (uintptr_t)u | (uintptr_t)id_map | (uintptr_t)ids | (uintptr_t)logprob | (uintptr_t)kept;
  if ((uintptr_t)logits & (dtype == LOWBIT_LOGITS_BF16 ? 1 : 3) || words & 3) return LOWBIT_ERR_ALIGN;
  const SampleArgs a = {logits, row_stride, M, V, 1, 0, 0, temperature, top_k, top_p, min_p, u, id_map, ids, logprob, kept};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = dtype == LOWBIT_LOGITS_BF16 ? launch_rows<true>(a, M, V, s) : launch_rows<false>(a, M, V, s);
  return e == cudaSuccess ? LOWBIT_OK : LOWBIT_ERR_CUDA;
}
