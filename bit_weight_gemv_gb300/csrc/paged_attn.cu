// lowbit_paged_attention: its checks, and its choice of kernel (paged_attn_mma.cuh, paged_attn_tc.cuh).
#include "paged_attn_mma.cuh"

namespace lowbit {

void attention_config(cudaLaunchConfig_t* cfg, cudaLaunchAttribute* attr, int ctas, int threads, int smem,
                      cudaStream_t s) {
  *cfg = {};
  cfg->gridDim = dim3((unsigned)ctas);
  cfg->blockDim = dim3((unsigned)threads);
  cfg->dynamicSmemBytes = (size_t)smem;
  cfg->stream = s;
  *attr = {};
  attr->id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr->val.programmaticStreamSerializationAllowed = 1;
  cfg->attrs = attr;
  cfg->numAttrs = 1;
}

bool encode_cache(CUtensorMap* map, const PagedArgs& p, void* at, int D, bool fp8, int keys) {
  // looked up once, on the first call
  static const PFN_cuTensorMapEncodeTiled_v12000 encode = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult qr;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &qr) != cudaSuccess ||
        qr != cudaDriverEntryPointSuccess)
      return static_cast<PFN_cuTensorMapEncodeTiled_v12000>(nullptr);
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  }();
  if (!encode) return false;
  const int ps = p.page_mask + 1, part = fp8 ? (D < 128 ? D : 128) : 64;
  const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)ps, (cuuint64_t)p.Hk, (cuuint64_t)p.pages};
  const cuuint64_t strides[3] = {(cuuint64_t)p.token_stride, (cuuint64_t)p.head_stride, (cuuint64_t)p.page_stride};
  const cuuint32_t box[4] = {(cuuint32_t)part, (cuuint32_t)(ps < keys ? ps : keys), 1, 1};
  const cuuint32_t step[4] = {1, 1, 1, 1};
  return encode(map, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, at, dims, strides, box,
                step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                fp8 && D < 128 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t launch_attention_mma(const AttnArgs& a, int D, bool fp8, cudaStream_t s) { return launch_by_dim(a, D, fp8, s); }
cudaError_t launch_combine(const AttnArgs& a, int D, cudaStream_t s) { return launch_join(a, D, s); }

lowbit_status make_attn_args(const uint16_t* q, int64_t q_stride, int Hq, const lowbit_paged_batch* batch,
                             const lowbit_paged_cache* cache, float scale, int causal, int window, uint16_t* out,
                             float* lse, AttnArgs* to) {
  AttnArgs& a = *to;
  const lowbit_status st = make_paged_args(batch, cache, &a.p);
  if (st != LOWBIT_OK) return st;
  if (a.p.T == 0) return LOWBIT_OK;  // the token arrays may then be null
  if (!q || !out || !(scale == scale)) return LOWBIT_ERR_INVALID_ARG;
  const int D = cache->head_dim;
  if (Hq < 1 || Hq > 65536 || Hq % cache->heads || window < 0 || q_stride < (int64_t)Hq * D ||
      (long long)a.p.T * (Hq / cache->heads) > 0x7FFFFF00LL ||
      ((long long)a.p.width << a.p.page_shift) > 0x7FFFFF00LL)
    return LOWBIT_ERR_SHAPE;
  if (((uintptr_t)q | (uintptr_t)out) & 15 || q_stride % 8 || ((uintptr_t)lse & 3)) return LOWBIT_ERR_ALIGN;
  const int G = Hq / cache->heads;
  a.shape = ItemShape{G, G > 1 ? (uint32_t)((1ull << 32) / G) : 0xFFFFFFFFu, 0, 0, 0, causal != 0, window};
  a.q = q;
  a.q_stride = q_stride;
  a.Hq = Hq;
  a.scale = scale;
  a.out = out;
  a.lse = lse;
  a.stall = debug_stall();
  return LOWBIT_OK;
}

}  // namespace lowbit

using namespace lowbit;

extern "C" {

size_t lowbit_paged_attention_workspace_bytes(int T, int B, int Hq, int Hk, int D) {
  if (T < 0 || T > kMaxTokens || B < 1 || B > kMaxBatch || Hk < 1 || Hk > 4096 || Hq < 1 || Hq > 65536 ||
      Hq % Hk || (D != 64 && D != 128 && D != 256))
    return 0;
  return pieces_bytes(D);
}

lowbit_status lowbit_paged_attention(const uint16_t* q, int64_t q_stride, int Hq,
                                     const lowbit_paged_batch* batch, const lowbit_paged_cache* cache,
                                     float scale, int causal, int window, uint16_t* out, float* lse,
                                     void* workspace, size_t ws_bytes, void* stream) {
  AttnArgs a = {};
  const lowbit_status st = make_attn_args(q, q_stride, Hq, batch, cache, scale, causal, window, out, lse, &a);
  if (st != LOWBIT_OK || a.p.T == 0) return st;
  const int D = cache->head_dim;
  if (!workspace || ws_bytes < lowbit_paged_attention_workspace_bytes(a.p.T, a.p.B, Hq, cache->heads, D))
    return LOWBIT_ERR_WORKSPACE;
  if ((uintptr_t)workspace & 15) return LOWBIT_ERR_ALIGN;
  a.p.err = device_error_word();
  if (!a.p.err) return LOWBIT_ERR_CUDA;
  use_pieces(&a, workspace, D);
  a.wide = (((uintptr_t)out | (uintptr_t)workspace) & 31) == 0;
  const cudaError_t e = launch_attention(a, D, cache->dtype == LOWBIT_CACHE_E4M3, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? LOWBIT_OK : LOWBIT_ERR_CUDA;
}

}  // extern "C"
