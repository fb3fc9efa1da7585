// Rotary positions on the new tokens' queries and keys, and keys and values into a paged cache.
//
// Pair j of a head's first `rot` elements turns by the position's angle, whose cosine and sine
// come from a table row: a' = a cos - b sin, b' = b cos + a sin.  Every product and sum is
// rounded on its own (no fused multiply-add), so the stored bits are those of the formula in
// fp32 and do not depend on how a compiler contracts it.
//
// Bound: memory.  Each of q, k and v is read once and written once, plus 4 * rot bytes of table
// per token; nothing is shared between tokens, so a thread takes 16 elements of one head of one
// token: the two 8-element vectors that hold 8 whole pairs, as 16-byte accesses.  A block takes one
// token, or eight in long calls.  16,665 tokens of 32 + 8 + 8 heads of 128, bf16: 49.4 us, 261 MB,
// 5.3 TB/s of 6.8 copied (57 us with one token per block); 512 tokens into an e4m3 cache 3.9 us, one
// token 2.9 us, which is a launch and two dependent loads (the page, then the data).
#include "common.cuh"
#include "paged.cuh"
#include "ptx.cuh"

#include <cuda_fp8.h>

#include <algorithm>

namespace lowbit {
namespace {

struct AppendArgs {
  PagedArgs p;
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  long long q_stride, k_stride, v_stride;
  const float* rope;
  int rope_rows, rot, Hq;
  uint16_t* q_out;
};

__device__ __forceinline__ void unpack8(const uint4 w, float (&x)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(u[i] << 16);
    x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  return (uint32_t)float_to_bf16_bits(lo) | ((uint32_t)float_to_bf16_bits(hi) << 16);
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                    pack_bf16(x[6], x[7]));
}
__device__ __forceinline__ uint2 pack8_e4m3(const float (&x)[8], float scale) {
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    w[i >> 2] |= (uint32_t)__nv_cvt_float_to_fp8(__fdiv_rn(x[i], scale), __NV_SATFINITE, __NV_E4M3)
                 << (8 * (i & 3));
  return make_uint2(w[0], w[1]);
}

template <int D, bool FP8, bool INTER, int TOKENS>
__global__ void __launch_bounds__(256, 5) kv_append_kernel(const __grid_constant__ AppendArgs a) {
  constexpr int kPer = D / 16;  // threads per head
  const int t0 = blockIdx.x * TOKENS, tid = threadIdx.x, lane = tid & 31;
  __shared__ int s_pos[TOKENS], s_page[TOKENS];
  const PagedArgs& p = a.p;
  const int nq = a.q ? a.Hq : 0;
  const int units = (nq + 2 * p.Hk) * kPer;
  asm volatile("griddepcontrol.wait;" ::: "memory");

  // a warp looks up each token's place
  if (tid < 32 * TOKENS) {
    const int t = t0 + (tid >> 5);
    // its request: the first one whose rows it is among
    int b = p.B, row0 = 0, end = 0, kv = 0;
    for (int b0 = 0; b0 < p.B; b0 += 32) {
      int from = 0, to = 0, len = 0;
      if (b0 + lane < p.B) from = p.cu_q[b0 + lane], to = p.cu_q[b0 + lane + 1], len = p.kv_lens[b0 + lane];
      if (to < from) record_error(p.err, LOWBIT_ERR_INVALID_ARG);
      const uint32_t in = __ballot_sync(~0u, from <= t && t < to);
      if (in && b == p.B) {
        const int src = __ffs(in) - 1;
        b = b0 + src;
        row0 = __shfl_sync(~0u, from, src), end = __shfl_sync(~0u, to, src), kv = __shfl_sync(~0u, len, src);
      }
    }
    int pos = -1, page = -1;
    if (t < p.T && b < p.B) {
      const Request r = check_request(p, row0, end, kv);
      if (t - r.row0 < r.n) {
        pos = r.kv - r.n + (t - r.row0);
        const bool in = pos >= 0 && (a.rot == 0 || pos < a.rope_rows);
        if (in) page = p.table[(long long)b * p.table_stride + (pos >> p.page_shift)];
        if (!in || page < 0 || page >= p.pages) {
          record_error(p.err, LOWBIT_ERR_INVALID_ARG);
          pos = -1;
        }
      }
    }
    if (lane == 0) s_pos[tid >> 5] = pos, s_page[tid >> 5] = page;
  }
  __syncthreads();

#pragma unroll 2
  for (int i = tid; i < units * TOKENS; i += 256) {
    const int which = TOKENS == 1 ? 0 : i / units, u = TOKENS == 1 ? i : i - which * units;
    const int t = t0 + which, pos = s_pos[which];
    if (pos < 0) continue;
    const int head = u / kPer, j = u % kPer;
    const int kind = head < nq ? 0 : (head < nq + p.Hk ? 1 : 2);  // q, k, v
    const int h = kind == 0 ? head : (kind == 1 ? head - nq : head - nq - p.Hk);
    const uint16_t* src = (kind == 0 ? a.q + (long long)t * a.q_stride
                         : kind == 1 ? a.k + (long long)t * a.k_stride
                                     : a.v + (long long)t * a.v_stride) + (long long)h * D;
    const bool turn = kind != 2 && 16 * j < a.rot;
    const int ia = !INTER && turn ? 8 * j : 16 * j, ib = !INTER && turn ? a.rot / 2 + 8 * j : 16 * j + 8;
    float x[8], y[8];
    unpack8(*reinterpret_cast<const uint4*>(src + ia), x);
    unpack8(*reinterpret_cast<const uint4*>(src + ib), y);
    const long long slot = (long long)s_page[which] * p.page_stride + (long long)(pos & p.page_mask) * p.token_stride;
    const float* row = a.rope + (long long)pos * a.rot;
    if (turn) {
      float c[8], s[8];
      const float4* pc = reinterpret_cast<const float4*>(row + 8 * j);
      const float4* ps = reinterpret_cast<const float4*>(row + a.rot / 2 + 8 * j);
      *reinterpret_cast<float4*>(c) = __ldg(pc);
      *reinterpret_cast<float4*>(c + 4) = __ldg(pc + 1);
      *reinterpret_cast<float4*>(s) = __ldg(ps);
      *reinterpret_cast<float4*>(s + 4) = __ldg(ps + 1);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float& e = INTER ? (i < 4 ? x[2 * i] : y[2 * (i - 4)]) : x[i];
        float& f = INTER ? (i < 4 ? x[2 * i + 1] : y[2 * (i - 4) + 1]) : y[i];
        const float e0 = e, f0 = f;
        e = __fsub_rn(__fmul_rn(e0, c[i]), __fmul_rn(f0, s[i]));
        f = __fadd_rn(__fmul_rn(f0, c[i]), __fmul_rn(e0, s[i]));
      }
    }
    if (kind == 0) {
      uint16_t* dst = a.q_out + ((long long)t * a.Hq + h) * D;
      *reinterpret_cast<uint4*>(dst + ia) = pack8(x);
      *reinterpret_cast<uint4*>(dst + ib) = pack8(y);
      continue;
    }
    uint8_t* dst = (kind == 1 ? p.k : p.v) + slot + (long long)h * p.head_stride;
    if (FP8) {
      const float* sc = kind == 1 ? p.k_scale : p.v_scale;
      const float scale = sc ? __ldg(sc + h) : 1.0f;
      *reinterpret_cast<uint2*>(dst + ia) = pack8_e4m3(x, scale);
      *reinterpret_cast<uint2*>(dst + ib) = pack8_e4m3(y, scale);
    } else {
      *reinterpret_cast<uint4*>(dst + 2 * ia) = pack8(x);
      *reinterpret_cast<uint4*>(dst + 2 * ib) = pack8(y);
    }
  }
}

template <int D, int TOKENS>
cudaError_t launch(const AppendArgs& a, bool fp8, bool inter, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((a.p.T + TOKENS - 1) / TOKENS));
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (fp8)
    return inter ? cudaLaunchKernelEx(&cfg, kv_append_kernel<D, true, true, TOKENS>, a)
                 : cudaLaunchKernelEx(&cfg, kv_append_kernel<D, true, false, TOKENS>, a);
  return inter ? cudaLaunchKernelEx(&cfg, kv_append_kernel<D, false, true, TOKENS>, a)
               : cudaLaunchKernelEx(&cfg, kv_append_kernel<D, false, false, TOKENS>, a);
}
template <int D>
cudaError_t launch_tokens(const AppendArgs& a, bool fp8, bool inter, cudaStream_t s) {
  // One token per block finishes soonest while the blocks come in few waves of 760; eight share the lookup
  // and fill the block where a token has few units of 16 elements.  us with one / eight, bf16: 40 units a
  // token, 608 tokens 2.4 / 3.4, 1,216 3.8 / 3.5; 96 units, 1,216 4.1 / 4.1, 1,824 5.5 / 4.5; 192 units, 2,432
  // 8.5 / 9.1, 3,648 13.5 / 12.1; 256 units, 3,040 12.8 / 15.2, 4,864 19.0 / 19.6; 384 units, 1,824 12.3 / 17.1,
  // 3,648 20.9 / 21.1, 6,080 31.9 / 27.1; 640 units, 3,952 32.1 / 34.4, 4,864 38.3 / 37.8.
  const long long units = (long long)((a.q ? a.Hq : 0) + 2 * a.p.Hk) * (D / 16);
  return a.p.T > std::max(1000LL, std::min(16 * units, 4000LL)) ? launch<D, 8>(a, fp8, inter, s) : launch<D, 1>(a, fp8, inter, s);
}

inline bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
// True where the `bytes` bytes at `p` meet one of T rows of `row` bytes, `stride` bytes apart from `first` on.
inline bool meets(const void* p, __int128 bytes, const void* first, __int128 row, __int128 stride, int T) {
  const __int128 at = (__int128)(uintptr_t)p - (__int128)(uintptr_t)first;
  const __int128 t = at < row ? 0 : (at - row) / stride + 1;  // the first row that ends behind p
  return t < T && t * stride < at + bytes;
}

}  // namespace

lowbit_status make_paged_args(const lowbit_paged_batch* batch, const lowbit_paged_cache* cache,
                              PagedArgs* a) {
  if (!batch || !cache || !batch->cu_q || !batch->kv_lens || !batch->block_table || !cache->k ||
      !cache->v)
    return LOWBIT_ERR_INVALID_ARG;
  if (cache->dtype != LOWBIT_CACHE_BF16 && cache->dtype != LOWBIT_CACHE_E4M3) return LOWBIT_ERR_INVALID_ARG;
  if (cache->dtype == LOWBIT_CACHE_BF16 && (cache->k_scale || cache->v_scale)) return LOWBIT_ERR_INVALID_ARG;
  const int size = cache->dtype == LOWBIT_CACHE_E4M3 ? 1 : 2;
  const int ps = cache->page_size;
  if (batch->B < 1 || batch->B > kMaxBatch || batch->T < 0 || batch->T > kMaxTokens ||
      batch->width < 1 || batch->table_stride < batch->width || cache->num_pages < 1 || ps < 1 ||
      ps > kMaxPageSize || (ps & (ps - 1)) || cache->heads < 1 || cache->heads > 4096 ||
      (cache->head_dim != 64 && cache->head_dim != 128 && cache->head_dim != 256))
    return LOWBIT_ERR_SHAPE;
  if ((int64_t)ps * cache->head_dim * size < 128) return LOWBIT_ERR_SHAPE;  // a tensor copy's alignment
  const int64_t strides[3] = {cache->page_stride, cache->token_stride, cache->head_stride};
  for (const int64_t s : strides)
    if (s <= 0 || s >= (int64_t)1 << 39 || s * size % 16) return LOWBIT_ERR_ALIGN;
  if (!aligned16(cache->k) || !aligned16(cache->v) || ((uintptr_t)batch->cu_q & 3) ||
      ((uintptr_t)batch->kv_lens & 3) || ((uintptr_t)batch->block_table & 3) ||
      ((uintptr_t)cache->k_scale & 3) || ((uintptr_t)cache->v_scale & 3))
    return LOWBIT_ERR_ALIGN;
  *a = PagedArgs{batch->cu_q, batch->kv_lens, batch->block_table, batch->table_stride, batch->B,
                 batch->T, batch->width, static_cast<uint8_t*>(cache->k),
                 static_cast<uint8_t*>(cache->v), strides[0] * size, strides[1] * size,
                 strides[2] * size, cache->num_pages, __builtin_ctz(ps), ps - 1, cache->heads,
                 cache->k_scale, cache->v_scale, nullptr};
  return LOWBIT_OK;
}

}  // namespace lowbit

using namespace lowbit;

extern "C" lowbit_status lowbit_kv_append(const uint16_t* q, int64_t q_stride, const uint16_t* k,
                                          int64_t k_stride, const uint16_t* v, int64_t v_stride,
                                          int Hq, const float* rope, int rope_rows, int rot,
                                          int interleaved, const lowbit_paged_batch* batch,
                                          const lowbit_paged_cache* cache, uint16_t* q_out,
                                          void* stream) {
  AppendArgs a = {};
  const lowbit_status st = make_paged_args(batch, cache, &a.p);
  if (st != LOWBIT_OK) return st;
  if (a.p.T == 0) return LOWBIT_OK;  // the token arrays may then be null
  if (!k || !v || !q != !q_out) return LOWBIT_ERR_INVALID_ARG;
  const int D = cache->head_dim;
  if (rot < 0 || rot > D || rot % 16 || (q && (Hq < 1 || Hq > 65536))) return LOWBIT_ERR_SHAPE;
  if (rot ? (!rope || rope_rows < 1) : rope != nullptr) return LOWBIT_ERR_INVALID_ARG;
  if ((q && q_stride < (int64_t)Hq * D) || k_stride < (int64_t)cache->heads * D ||
      v_stride < (int64_t)cache->heads * D)
    return LOWBIT_ERR_SHAPE;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(rope) || !aligned16(q_out) ||
      (q && q_stride % 8) || k_stride % 8 || v_stride % 8)
    return LOWBIT_ERR_ALIGN;
  if (q) {  // a block that writes its token's queries must not meet what another one has yet to read
    const __int128 row = (__int128)Hq * D * 2, kv = (__int128)cache->heads * D * 2;
    const bool in_place = q_out == q && (a.p.T == 1 || q_stride == (int64_t)Hq * D);
    if ((!in_place && meets(q_out, row * a.p.T, q, row, (__int128)q_stride * 2, a.p.T)) ||
        meets(q_out, row * a.p.T, k, kv, (__int128)k_stride * 2, a.p.T) ||
        meets(q_out, row * a.p.T, v, kv, (__int128)v_stride * 2, a.p.T))
      return LOWBIT_ERR_INVALID_ARG;
  }
  a.p.err = device_error_word();
  if (!a.p.err) return LOWBIT_ERR_CUDA;
  a.q = q;
  a.k = k;
  a.v = v;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.rope = rope;
  a.rope_rows = rope_rows;
  a.rot = rot;
  a.Hq = Hq;
  a.q_out = q_out;
  const bool fp8 = cache->dtype == LOWBIT_CACHE_E4M3, inter = interleaved != 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = D == 64 ? launch_tokens<64>(a, fp8, inter, s)
                      : D == 128 ? launch_tokens<128>(a, fp8, inter, s)
                                 : launch_tokens<256>(a, fp8, inter, s);
  return e == cudaSuccess ? LOWBIT_OK : LOWBIT_ERR_CUDA;
}
