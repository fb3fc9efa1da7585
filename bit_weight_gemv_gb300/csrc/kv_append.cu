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
  const float* q_weight;  // of the norm (kv_append_norm_kernel alone)
  const float* k_weight;
  float eps;
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

// Where token t goes, found by a warp: its position and page, or position -1 for a row that belongs to no
// request or has no place (which the device error word then says).
struct Spot {
  int pos, page;
};
__device__ __forceinline__ Spot find_spot(const AppendArgs& a, int t, int lane) {
  const PagedArgs& p = a.p;
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
  Spot s = {-1, -1};
  if (t < p.T && b < p.B) {
    const Request r = check_request(p, row0, end, kv);
    if (t - r.row0 < r.n) {
      s.pos = r.kv - r.n + (t - r.row0);
      const bool in = s.pos >= 0 && (a.rot == 0 || s.pos < a.rope_rows);
      if (in) s.page = p.table[(long long)b * p.table_stride + (s.pos >> p.page_shift)];
      if (!in || s.page < 0 || s.page >= p.pages) {
        record_error(p.err, LOWBIT_ERR_INVALID_ARG);
        s.pos = -1;
      }
    }
  }
  return s;
}
// Eight pairs of a thread turned: (x[i], y[i]), or neighbours of x and then of y.
template <bool INTER>
__device__ __forceinline__ void turn8(float (&x)[8], float (&y)[8], const float (&c)[8], const float (&s)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float& e = INTER ? (i < 4 ? x[2 * i] : y[2 * (i - 4)]) : x[i];
    float& f = INTER ? (i < 4 ? x[2 * i + 1] : y[2 * (i - 4) + 1]) : y[i];
    const float e0 = e, f0 = f;
    e = __fsub_rn(__fmul_rn(e0, c[i]), __fmul_rn(f0, s[i]));
    f = __fadd_rn(__fmul_rn(f0, c[i]), __fmul_rn(e0, s[i]));
  }
}
// A thread's 16 elements of head h into the slot at byte `slot` of the keys or values.
// ONCE: to be read once at most before the next 100 MB of them (a hint to L2).
template <bool ONCE, class V>
__device__ __forceinline__ void store(uint8_t* at, V v) {
  if (ONCE) __stcs(reinterpret_cast<V*>(at), v);
  else *reinterpret_cast<V*>(at) = v;
}
template <bool FP8, bool ONCE = false>
__device__ __forceinline__ void store_cache(const PagedArgs& p, bool key, long long slot, int h, int ia, int ib,
                                            const float (&x)[8], const float (&y)[8]) {
  uint8_t* dst = (key ? p.k : p.v) + slot + (long long)h * p.head_stride;
  if (FP8) {
    const float* sc = key ? p.k_scale : p.v_scale;
    const float scale = sc ? __ldg(sc + h) : 1.0f;
    store<ONCE>(dst + ia, pack8_e4m3(x, scale));
    store<ONCE>(dst + ib, pack8_e4m3(y, scale));
  } else {
    store<ONCE>(dst + 2 * ia, pack8(x));
    store<ONCE>(dst + 2 * ib, pack8(y));
  }
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
    const Spot s = find_spot(a, t0 + (tid >> 5), lane);
    if (lane == 0) s_pos[tid >> 5] = s.pos, s_page[tid >> 5] = s.page;
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
      turn8<INTER>(x, y, c, s);
    }
    if (kind == 0) {
      uint16_t* dst = a.q_out + ((long long)t * a.Hq + h) * D;
      *reinterpret_cast<uint4*>(dst + ia) = pack8(x);
      *reinterpret_cast<uint4*>(dst + ib) = pack8(y);
      continue;
    }
    store_cache<FP8>(p, kind == 1, slot, h, ia, ib, x, y);
  }
}

// With a norm of each head of q and k before the rotation:
//   y = x * r * w,  r = 1 / sqrt(sum x^2 / D + eps),
// everything in fp32 from the bf16 elements to the one rounding of what is stored.
//
// WARPS warps take a token: 32 lanes hold 512 elements, D / 16 lanes a head, so that
// a head's sum of squares is a few exchanges between neighbouring lanes, the lane's part of the angles stays in
// registers over the token's heads, and no warp waits for another.  The first heads are asked for before the
// token's place is known.
//
// 16,396 tokens of 32 + 8 + 8 heads of 128, bf16: 74.5 us, 411 MB, 5.5 TB/s of 6.8 copied: HBM, reads and writes of
// short runs in turn.  One step at a time 88 us, four 92 (more registers, fewer warps), blocks of 256 threads 77.9,
// without the hints to L2 76.8, eight warps a token 128 (of 75.6 then).  Into an e4m3 cache 92 us, 378 MB, 4.1 TB/s: as many
// instructions a cycle (58% of the slots, with 24 warps an SM) but 23% more of them, for an exact quotient and a
// conversion of each element of k and v.  512 tokens into an e4m3 cache 4.5 us, one 4.0.
template <int WARPS>
constexpr int kNormThreads = WARPS < 8 ? 128 : 256;
template <int D, bool FP8, bool INTER, int WARPS>
__global__ void __launch_bounds__(kNormThreads<WARPS>, WARPS < 8 ? 6 : 3)
kv_append_norm_kernel(const __grid_constant__ AppendArgs a) {
  constexpr int kPer = D / 16, kHeads = 32 / kPer;  // lanes per head, heads per step of a warp
  constexpr bool kLong = WARPS == 1;
  constexpr int kBatch = WARPS <= 2 ? 2 : 1;            // steps asked for together
  const PagedArgs& p = a.p;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t = blockIdx.x * (kNormThreads<WARPS> / 32 / WARPS) + warp / WARPS, part = warp % WARPS;
  if (t >= p.T) return;
  const int j = lane % kPer, nq = a.q ? a.Hq : 0;
  const int q_steps = (nq + kHeads - 1) / kHeads, kv_steps = (p.Hk + kHeads - 1) / kHeads;
  const int steps = q_steps + 2 * kv_steps;
  const bool turned = 16 * j < a.rot;
  const int ia = !INTER && turned ? 8 * j : 16 * j, ib = !INTER && turned ? a.rot / 2 + 8 * j : 16 * j + 8;
  asm volatile("griddepcontrol.wait;" ::: "memory");

  // the steps' heads: first those of q, then of k, then of v
  struct Place {
    int kind, h;
    bool in;
  };
  auto locate = [&](int step) {
    Place w;
    w.kind = step < q_steps ? 0 : (step < q_steps + kv_steps ? 1 : 2);
    w.h = (step - (w.kind == 0 ? 0 : q_steps + (w.kind - 1) * kv_steps)) * kHeads + lane / kPer;
    w.in = step < steps && w.h < (w.kind == 0 ? nq : p.Hk);
    return w;
  };
  uint4 va[kBatch], vb[kBatch];
  auto load = [&](int step0) {
#pragma unroll
    for (int e = 0; e < kBatch; ++e) {
      const Place w = locate(step0 + e * WARPS);
      va[e] = vb[e] = make_uint4(0, 0, 0, 0);
      if (!w.in) continue;
      const uint16_t* src = (w.kind == 0 ? a.q + (long long)t * a.q_stride
                           : w.kind == 1 ? a.k + (long long)t * a.k_stride
                                         : a.v + (long long)t * a.v_stride) + (long long)w.h * D;
      va[e] = kLong ? __ldcs(reinterpret_cast<const uint4*>(src + ia)) : *reinterpret_cast<const uint4*>(src + ia);
      vb[e] = kLong ? __ldcs(reinterpret_cast<const uint4*>(src + ib)) : *reinterpret_cast<const uint4*>(src + ib);
    }
  };
  load(part);

  const Spot s = find_spot(a, t, lane);
  if (s.pos < 0) return;
  float c[8], sn[8];
  if (turned) {
    const float* row = a.rope + (long long)s.pos * a.rot + 8 * j;
    *reinterpret_cast<float4*>(c) = __ldg(reinterpret_cast<const float4*>(row));
    *reinterpret_cast<float4*>(c + 4) = __ldg(reinterpret_cast<const float4*>(row) + 1);
    *reinterpret_cast<float4*>(sn) = __ldg(reinterpret_cast<const float4*>(row + a.rot / 2));
    *reinterpret_cast<float4*>(sn + 4) = __ldg(reinterpret_cast<const float4*>(row + a.rot / 2) + 1);
  }
  const long long slot = (long long)s.page * p.page_stride + (long long)(s.pos & p.page_mask) * p.token_stride;

  for (int step0 = part; step0 < steps; step0 += WARPS * kBatch) {
    if (step0 != part) load(step0);
#pragma unroll
    for (int e = 0; e < kBatch; ++e) {
      const Place w = locate(step0 + e * WARPS);
      float x[8], y[8];
      unpack8(va[e], x);
      unpack8(vb[e], y);
      const float* weight = w.kind == 0 ? a.q_weight : (w.kind == 1 ? a.k_weight : nullptr);
      if (weight) {
        auto mean_square = [&](float eps) {
          float sum = 0.0f;
#pragma unroll
          for (int i = 0; i < 8; ++i) sum = fmaf(x[i], x[i], fmaf(y[i], y[i], sum));
#pragma unroll
          for (int o = kPer / 2; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
          return fmaf(sum, 1.0f / D, eps);
        };
        float mean = mean_square(a.eps);
        // Near the end of fp32's range squares lose their bits, and the mean does: such a head (elements up to 2^-41, so
        // that its squares stay finite) is multiplied by 2^100, which is exact, and eps by the square of that.
        const bool small = mean < 0x1p-90f;
        if (__any_sync(~0u, small)) {
          const float up = small ? 0x1p100f : 1.0f;
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] *= up, y[i] *= up;
          mean = mean_square(a.eps * up * up);
        }
        const float r = rsqrtf(mean);
#pragma unroll
        for (int i = 0; i < 8; i += 4) {
          const float4 wa = __ldg(reinterpret_cast<const float4*>(weight + ia + i));
          const float4 wb = __ldg(reinterpret_cast<const float4*>(weight + ib + i));
          // (x r first, which is at most sqrt(D): r w may be out of range where x r w is not)
          x[i] = x[i] * r * wa.x, x[i + 1] = x[i + 1] * r * wa.y, x[i + 2] = x[i + 2] * r * wa.z, x[i + 3] = x[i + 3] * r * wa.w;
          y[i] = y[i] * r * wb.x, y[i + 1] = y[i + 1] * r * wb.y, y[i + 2] = y[i + 2] * r * wb.z, y[i + 3] = y[i + 3] * r * wb.w;
        }
      }
      if (turned && w.kind != 2) turn8<INTER>(x, y, c, sn);
      if (!w.in) continue;
      if (w.kind == 0) {
        uint8_t* dst = reinterpret_cast<uint8_t*>(a.q_out + ((long long)t * a.Hq + w.h) * D);
        store<kLong>(dst + 2 * ia, pack8(x));
        store<kLong>(dst + 2 * ib, pack8(y));
      } else {
        store_cache<FP8, kLong>(p, w.kind == 1, slot, w.h, ia, ib, x, y);
      }
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


template <int D, int WARPS>
cudaError_t launch_norm(const AppendArgs& a, bool fp8, bool inter, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  constexpr int kTokens = kNormThreads<WARPS> / 32 / WARPS;
  cfg.gridDim = dim3((unsigned)((a.p.T + kTokens - 1) / kTokens));
  cfg.blockDim = dim3(kNormThreads<WARPS>);
  cfg.stream = s;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (fp8)
    return inter ? cudaLaunchKernelEx(&cfg, kv_append_norm_kernel<D, true, true, WARPS>, a)
                 : cudaLaunchKernelEx(&cfg, kv_append_norm_kernel<D, true, false, WARPS>, a);
  return inter ? cudaLaunchKernelEx(&cfg, kv_append_norm_kernel<D, false, true, WARPS>, a)
               : cudaLaunchKernelEx(&cfg, kv_append_norm_kernel<D, false, false, WARPS>, a);
}
template <int D>
cudaError_t launch_norm_warps(const AppendArgs& a, bool fp8, bool inter, cudaStream_t s) {
  // As many warps a token as fit on the GPU at a time, 24 an SM.  us with 8 / 4 / 2 / 1 warps, 32 + 8 + 8 heads of
  // 128, bf16: 304 tokens 4.0 / 4.2 / 5.4 / 8.1, 608 6.9 / 5.1 / 6.1 / 8.2, 1,216 9.7 / 8.3 / 7.4 / 9.5, 1,824 12.8 / 9.6 /
  // 9.4 / 11.2, 3,648 27 / 20 / 19 / 17, 7,296 60 / 45 / 40 / 36.
  const int T = a.p.T;
  return T <= 3 * 152 ? launch_norm<D, 8>(a, fp8, inter, s)
       : T <= 6 * 152 ? launch_norm<D, 4>(a, fp8, inter, s)
       : T <= 12 * 152 ? launch_norm<D, 2>(a, fp8, inter, s)
                       : launch_norm<D, 1>(a, fp8, inter, s);
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

namespace {
// The checks of both append calls; fills `a` (all but the norm's part).  LOWBIT_OK with T = 0: nothing to do.
lowbit_status make_append_args(const uint16_t* q, int64_t q_stride, const uint16_t* k, int64_t k_stride,
                               const uint16_t* v, int64_t v_stride, int Hq, const float* rope, int rope_rows, int rot,
                               const lowbit_paged_batch* batch, const lowbit_paged_cache* cache, uint16_t* q_out,
                               AppendArgs* out) {
  AppendArgs a = {};
  const lowbit_status st = make_paged_args(batch, cache, &a.p);
  if (st != LOWBIT_OK) return st;
  *out = a;
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
  *out = a;
  return LOWBIT_OK;
}
}  // namespace

}  // namespace lowbit

using namespace lowbit;

extern "C" {

lowbit_status lowbit_kv_append(const uint16_t* q, int64_t q_stride, const uint16_t* k, int64_t k_stride,
                               const uint16_t* v, int64_t v_stride, int Hq, const float* rope, int rope_rows,
                               int rot, int interleaved, const lowbit_paged_batch* batch,
                               const lowbit_paged_cache* cache, uint16_t* q_out, void* stream) {
  AppendArgs a = {};
  const lowbit_status st = make_append_args(q, q_stride, k, k_stride, v, v_stride, Hq, rope, rope_rows, rot, batch,
                                            cache, q_out, &a);
  if (st != LOWBIT_OK || a.p.T == 0) return st;
  a.p.err = device_error_word();
  if (!a.p.err) return LOWBIT_ERR_CUDA;
  const int D = cache->head_dim;
  const bool fp8 = cache->dtype == LOWBIT_CACHE_E4M3, inter = interleaved != 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = D == 64 ? launch_tokens<64>(a, fp8, inter, s)
                      : D == 128 ? launch_tokens<128>(a, fp8, inter, s)
                                 : launch_tokens<256>(a, fp8, inter, s);
  return e == cudaSuccess ? LOWBIT_OK : LOWBIT_ERR_CUDA;
}

lowbit_status lowbit_kv_append_norm(const uint16_t* q, int64_t q_stride, const uint16_t* k, int64_t k_stride,
                                    const uint16_t* v, int64_t v_stride, int Hq, const float* q_weight,
                                    const float* k_weight, float eps, const float* rope, int rope_rows, int rot,
                                    int interleaved, const lowbit_paged_batch* batch,
                                    const lowbit_paged_cache* cache, uint16_t* q_out, void* stream) {
  AppendArgs a = {};
  const lowbit_status st = make_append_args(q, q_stride, k, k_stride, v, v_stride, Hq, rope, rope_rows, rot, batch,
                                            cache, q_out, &a);
  if (st != LOWBIT_OK || a.p.T == 0) return st;
  if ((q_weight && !q) || !(eps >= 0.0f) || eps > 3.402823466e38f) return LOWBIT_ERR_INVALID_ARG;
  if (!aligned16(q_weight) || !aligned16(k_weight)) return LOWBIT_ERR_ALIGN;
  a.q_weight = q_weight;
  a.k_weight = k_weight;
  a.eps = eps;
  a.p.err = device_error_word();
  if (!a.p.err) return LOWBIT_ERR_CUDA;
  const int D = cache->head_dim;
  const bool fp8 = cache->dtype == LOWBIT_CACHE_E4M3, inter = interleaved != 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = D == 64 ? launch_norm_warps<64>(a, fp8, inter, s)
                      : D == 128 ? launch_norm_warps<128>(a, fp8, inter, s)
                                 : launch_norm_warps<256>(a, fp8, inter, s);
  return e == cudaSuccess ? LOWBIT_OK : LOWBIT_ERR_CUDA;
}

}  // extern "C"
