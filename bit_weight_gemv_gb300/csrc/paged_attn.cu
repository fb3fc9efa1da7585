// lowbit_paged_attention: its checks, and its choice of kernel (paged_attn_mma.cuh, paged_attn_tc.cuh).
#include "paged_attn_mma.cuh"

namespace lowbit {
namespace {

// Items that the cuts went through: blocks (j, *) finish the item that CTA j began and others went
// on with, a share of its rows each.  The attention's CTAs leave behind what there is to join: found
// again from the batch, as it once was, it took 11 of 34 us for one row of 30,000 keys per head.
// Bound by round trips to L2, so everything a row needs is asked for at once where its pieces are few
// (1,200 tokens over 4,000 keys, most items cut once: 80 us with the attention, 86 when the weights came
// first and then pieces by eights).  Four blocks an SM: most blocks have nothing to join, and with
// fewer at a time the others wait for them (16 tokens over 32,765 keys: 34.5 us, 35.4 with three).
template <int D>
struct Join {
  static constexpr int kPart = D >= 128 ? 4 : 2, kParts = D / (32 * kPart);  // a lane's elements of a row
  const AttnArgs& a;
  long long slot0, c0;  // pieces: slot0, and slot 2 (c0 + i) for i = 1..n
  int n, R, r0, h, row_base, lane;
  float vscale;

  __device__ __forceinline__ long long place(int i, int row) const { return (i ? 2 * (c0 + i) : slot0) * R + row; }
  __device__ __forceinline__ void load(int i, int row, float (&v)[kParts][kPart]) const {
    const float* src = a.piece_o + place(i, row) * D + lane * kPart;
#pragma unroll
    for (int q = 0; q < kParts; ++q) {
      if (kPart == 4) *reinterpret_cast<float4*>(v[q]) = *reinterpret_cast<const float4*>(src + q * 128);
      else *reinterpret_cast<float2*>(v[q]) = *reinterpret_cast<const float2*>(src);
    }
  }
  // The joined row (`all`: of all its pieces) leaves.
  __device__ __forceinline__ void store(int row, bool all, float m, float l, const float (&acc)[kParts][kPart]) const {
    const int G = a.shape.G, r = r0 + row, tok = token_of(a.shape, r);
    const long long orow = (long long)(row_base + tok) * a.Hq + h * G + (r - tok * G);
    if (!all) return;
    const float s = l > 0.0f ? vscale / l : (l == 0.0f ? 0.0f : l);
#pragma unroll
    for (int q = 0; q < kParts; ++q) {
      uint16_t* dst = a.out + orow * D + q * 128 + lane * kPart;
      const uint32_t lo = pack2<false>(acc[q][0] * s, acc[q][1] * s);
      if (kPart == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(lo, pack2<false>(acc[q][kPart - 2] * s, acc[q][kPart - 1] * s));
      else *reinterpret_cast<uint32_t*>(dst) = lo;
    }
    if (lane == 0 && a.lse) a.lse[orow] = l == 0.0f ? -INFINITY : m * 0.6931471805599453f + logf(l);
  }
  // ROWS rows of up to PIECES pieces, by one warp.
  template <int ROWS, int PIECES>
  __device__ __forceinline__ void few(int row, int end) const {
    float2 ml[ROWS][PIECES];
    float v[ROWS][PIECES][kParts][kPart];
#pragma unroll
    for (int e = 0; e < ROWS; ++e)
#pragma unroll
      for (int k = 0; k < PIECES; ++k) {  // past the last: it again, with weight 0
        ml[e][k] = a.piece_ml[place(min(k, n), min(row + e, end - 1))];
        load(min(k, n), min(row + e, end - 1), v[e][k]);
      }
#pragma unroll
    for (int e = 0; e < ROWS; ++e) {
      float m = ml[e][0].x, l = 0.0f, acc[kParts][kPart] = {};
      bool all = ml[e][0].y != kNoPiece;
#pragma unroll
      for (int k = 1; k < PIECES; ++k) m = fmaxf(m, ml[e][k].x), all &= ml[e][k].y != kNoPiece;
#pragma unroll
      for (int k = 0; k < PIECES; ++k) {
        if (k > n) break;
        const float f = m == -INFINITY ? 0.0f : ex2(ml[e][k].x - m);
        l += f * ml[e][k].y;
#pragma unroll
        for (int q = 0; q < kParts; ++q)
#pragma unroll
          for (int d = 0; d < kPart; ++d) acc[q][d] += f * v[e][k][q][d];
      }
      if (row + e < end) store(row + e, all, m, l, acc);
    }
  }
  // One row of any number of pieces: the lanes hold the pieces' (maximum, sum), 32 at a time.
  __device__ __forceinline__ void many(int row) const {
    float m = -INFINITY;
    for (int i = lane; i <= n; i += 32) m = fmaxf(m, a.piece_ml[place(i, row)].x);
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
    float l = 0.0f, acc[kParts][kPart] = {};
    bool all = true;
    for (int i0 = 0; i0 <= n; i0 += 32) {
      float f = 0.0f;
      if (i0 + lane <= n) {
        const float2 ml = a.piece_ml[place(i0 + lane, row)];
        all &= ml.y != kNoPiece;
        f = m == -INFINITY ? 0.0f : ex2(ml.x - m);
        l += f * ml.y;
      }
      const int k1 = min(32, n + 1 - i0);
      constexpr int kBatch = 8 / kParts;  // pieces asked for together
      for (int k = 0; k < k1; k += kBatch) {
        float v[kBatch][kParts][kPart];
#pragma unroll
        for (int e = 0; e < kBatch; ++e) load(min(i0 + k + e, n), row, v[e]);
#pragma unroll
        for (int e = 0; e < kBatch; ++e) {
          const float fk = __shfl_sync(~0u, f, k + e);
#pragma unroll
          for (int q = 0; q < kParts; ++q)
#pragma unroll
            for (int d = 0; d < kPart; ++d)
              if (k + e < k1) acc[q][d] += fk * v[e][q][d];
        }
      }
    }
    for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(~0u, l, o);
    store(row, __all_sync(~0u, all), m, l, acc);
  }
};
template <int D>
__global__ void __launch_bounds__(kJoinThreads, 4) attn_combine_kernel(const __grid_constant__ AttnArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int4 lo = reinterpret_cast<const int4*>(a.cuts + blockIdx.x)[0];
  const int n = lo.x;
  if (n == 0) return;
  const int4 hi = reinterpret_cast<const int4*>(a.cuts + blockIdx.x)[1];
  const int rows = lo.z, warp = threadIdx.x >> 5;
  const int ra = rows * blockIdx.y / gridDim.y, rb = rows * (blockIdx.y + 1) / gridDim.y;
  const Join<D> j = {a, lo.y, (long long)blockIdx.x, n, 1 << a.shape.r_shift, lo.w, hi.y, hi.x, (int)(threadIdx.x & 31),
                     a.p.v_scale ? __ldg(a.p.v_scale + hi.y) : 1.0f};
  constexpr int kWide = D == 256 ? 4 : 8;
  if (n < 2) {
    for (int row = ra + 2 * warp; row < rb; row += kJoinThreads / 16) j.template few<2, 2>(row, rb);
  } else if (n < kWide) {
    for (int row = ra + warp; row < rb; row += kJoinThreads / 32) j.template few<1, kWide>(row, rb);
  } else {
    for (int row = ra + warp; row < rb; row += kJoinThreads / 32) j.many(row);
  }
}

template <int D, bool FP8>
cudaError_t launch_rows(const AttnArgs& a, cudaStream_t s) {
  // Rows that share a request's keys, on average: the host knows the totals only.
  const long long rows = ((long long)a.p.T * a.shape.G + a.p.B - 1) / a.p.B;
  if (rows <= 8) return launch_row8<D, FP8>(a, s);
  if (rows <= 16) return launch_mma<D, 1, FP8>(a, s);
  if (rows <= 32) return launch_mma<D, 2, FP8>(a, s);
  return launch_mma<D, 4, FP8>(a, s);
}

}  // namespace

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

cudaError_t launch_attention_mma(const AttnArgs& a, int D, bool fp8, cudaStream_t s) {
  if (D == 64) return fp8 ? launch_rows<64, true>(a, s) : launch_rows<64, false>(a, s);
  if (D == 128) return fp8 ? launch_rows<128, true>(a, s) : launch_rows<128, false>(a, s);
  return fp8 ? launch_rows<256, true>(a, s) : launch_rows<256, false>(a, s);
}

cudaError_t launch_combine(const AttnArgs& a, int D, cudaStream_t s) {
  if (a.ctas < 2) return cudaSuccess;
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr;
  attention_config(&cfg, &attr, a.ctas - 1, kJoinThreads, 0, s);
  cfg.gridDim.y = a.shape.r_shift > 4 ? 1u << (a.shape.r_shift - 4) : 1;  // 16 rows of an item each
  if (D == 64) return cudaLaunchKernelEx(&cfg, attn_combine_kernel<64>, a);
  if (D == 128) return cudaLaunchKernelEx(&cfg, attn_combine_kernel<128>, a);
  return cudaLaunchKernelEx(&cfg, attn_combine_kernel<256>, a);
}
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
