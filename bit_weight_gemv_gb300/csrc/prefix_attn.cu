// lowbit_prefix_attention: attention of requests whose first pages are the same ones.
//
// With the keys of a row cut into the shared ones and its own, (m, l, o) of each part (paged_attn_mma.cuh) join
// as any two sets of keys do.  So the shared part is computed with all rows of a group as one request without
// a mask, which reads its keys and values once for the group, the own part as ever, and a last step joins a row's
// pieces out of both.  The kernels and their schedule are lowbit_paged_attention's.
//
// Where one kernel suits both parts (few rows in the shared part; or many in the own one) one launch takes them,
// laid end to end in its schedule; else two, one after the other.
#include "paged_attn_mma.cuh"

namespace lowbit {
namespace {

constexpr int kPrefixJoinWarps = 8;

// The last of x[0..n), ascending, that is not above v, or 0: by a warp, so that it takes a round trip for
// every factor of 32 in n.
__device__ __forceinline__ int last_not_above(const int32_t* x, int n, int v, int lane) {
  int at = 0;
#pragma unroll 1
  while (n > 1) {
    const int step = (n + 31) / 32;
    const uint32_t in = __ballot_sync(~0u, lane * step < n && x[at + min(lane * step, n - 1)] <= v);
    const int k = in ? 31 - __clz(in) : 0;
    at += k * step;
    n = min(step, n - k * step);
  }
  return at;
}
// Request b with its group g as the header asks for them: inside the group's bounds and rows, and with what it
// shares computed.  False, and recorded, if not.
__device__ __forceinline__ bool request_of_group(const PrefixArgs& a, int b, int g, Request* own) {
  const int from = a.cu_groups[g], to = a.cu_groups[g + 1];
  const Request group = load_group(a, g);
  *own = load_own(a, b, g);
  if (own->n == 0) return false;
  const bool bounds = from >= 0 && to <= a.requests && b >= from && b < to;
  if (!bounds || own->row0 < a.p.cu_q[from] || own->row0 + own->n > a.p.cu_q[to] || (own->skip && group.n == 0)) {
    record_error(a.p.err, LOWBIT_ERR_INVALID_ARG);
    return false;
  }
  return true;
}

// The keys that row t shares where it is request b's, or -1 where it is not, or the request is not consistent.
__device__ __forceinline__ int shared_keys(const PrefixArgs& a, int b, int t) {
  Request own;
  if (a.p.cu_q[b] > t || t >= a.p.cu_q[b + 1] || !request_of_group(a, b, group_of(a, b), &own)) return -1;
  return own.skip;
}
// The same for whichever request has the row, -1 where none does: by a warp.  The search finds it where cu_q is
// ascending.  Offsets out of order hide consistent requests from it, so a row without one is asked of all requests, but
// for rows past cu_q[B], the padding of a captured graph, which are nobody's (asked as well they took 4,096 requests of a
// token and as many such rows from 231 to 355 us).
__device__ __forceinline__ int shared_keys_of_row(const PrefixArgs& a, int t, int lane) {
  int skip = shared_keys(a, last_not_above(a.p.cu_q, a.requests, t, lane), t);
  if (skip >= 0 || t >= a.p.cu_q[a.requests]) return skip;
#pragma unroll 1
  for (int b0 = 0; skip < 0 && b0 < a.requests; b0 += 32) {
    const int b = b0 + lane, from = b < a.requests ? a.p.cu_q[b] : 0, to = b < a.requests ? a.p.cu_q[b + 1] : 0;
    const uint32_t has = __ballot_sync(~0u, from >= 0 && from <= t && t < to && to <= a.p.T);
    if (has) skip = shared_keys(a, b0 + __ffs(has) - 1, t);
  }
  return skip;
}

// A warp joins a row's pieces: of the shared part, then of its own.  Bound by round trips: where they are and, meanwhile,
// the row's request and group; their statistics; the pieces.  Alone and cold 11 us for 256 rows, 22 for 20,992 (36 MB).
// (Looking the request up before the wait would take 1 us off, but what earlier kernels wrote is promised to be seen
// only behind it.)
template <int D>
__global__ void __launch_bounds__(kPrefixJoinWarps * 32)
prefix_join_kernel(const __grid_constant__ PrefixArgs a, const float* own_o, const float2* own_ml) {
  constexpr int kPart = D >= 128 ? 4 : 2, kParts = D / (32 * kPart), kBatch = 8 / kParts;
  const int lane = threadIdx.x & 31, h = blockIdx.y * kPrefixJoinWarps + (threadIdx.x >> 5), t = blockIdx.x;
  if (h >= a.Hq) return;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const long long row = (long long)t * a.Hq + h;
  int4 f0 = a.found[row];  // read only where the request shares anything
  const int4 f1 = a.found[a.rows + row];
  const int skip = shared_keys_of_row(a, t, lane);
  if (skip < 0) return;
  if (!skip) f0.x = kInBase;
  if (f0.x == kLost || f1.x == kLost) return;
  const int n0 = skip ? max(f0.x, 0) + 1 : 0, n = n0 + max(f1.x, 0) + 1;
  // where piece i is
  auto locate = [&](int i, const float2*& ml, const float*& o) {
    const bool second = i >= n0;
    const int4 f = second ? f1 : f0;
    const int k = second ? i - n0 : i;
    if (f.x == kInBase) {
      const long long place = row + (second ? a.rows : 0);
      ml = a.base_ml + place, o = a.base_o + place * D;
    } else {
      long long place = k ? (long long)f.z + (long long)(k - 1) * f.w : f.y;
      place = min(max(place, 0LL), (long long)kMaxPieceRows - 1);
      ml = (second ? own_ml : a.piece_ml) + place, o = (second ? own_o : a.piece_o) + place * D;
    }
  };
  float m = -INFINITY, l = 0.0f, acc[kParts][kPart] = {};
  bool all = true;
  for (int i0 = 0; i0 < n; i0 += 32) {  // the lanes hold the pieces' statistics, 32 at a time
    float2 ml = make_float2(-INFINITY, 0.0f);
    const float2* at_ml;
    const float* at_o = nullptr;
    if (i0 + lane < n) {
      locate(i0 + lane, at_ml, at_o);
      ml = *at_ml;
      all &= ml.y != kNoPiece;
    }
    float top = ml.x;
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
    top = fmaxf(top, m);
    const float before = top == -INFINITY ? 0.0f : ex2(m - top), f = top == -INFINITY ? 0.0f : ex2(ml.x - top);
    m = top;
    float sum = f * ml.y;
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
    l = l * before + sum;
#pragma unroll
    for (int q = 0; q < kParts; ++q)
#pragma unroll
      for (int d = 0; d < kPart; ++d) acc[q][d] *= before;
    const int k1 = min(32, n - i0);
    for (int k = 0; k < k1; k += kBatch) {  // asked for together
      float v[kBatch][kParts][kPart];
#pragma unroll
      for (int e = 0; e < kBatch; ++e) {
        const float* src = reinterpret_cast<const float*>(
                               __shfl_sync(~0u, (unsigned long long)reinterpret_cast<uintptr_t>(at_o), min(k + e, k1 - 1))) + lane * kPart;
#pragma unroll
        for (int q = 0; q < kParts; ++q) {
          if (kPart == 4) *reinterpret_cast<float4*>(v[e][q]) = *reinterpret_cast<const float4*>(src + q * 128);
          else *reinterpret_cast<float2*>(v[e][q]) = *reinterpret_cast<const float2*>(src);
        }
      }
#pragma unroll
      for (int e = 0; e < kBatch; ++e) {
        const float fk = __shfl_sync(~0u, f, min(k + e, 31));
        if (k + e >= k1) continue;
#pragma unroll
        for (int q = 0; q < kParts; ++q)
#pragma unroll
          for (int d = 0; d < kPart; ++d) acc[q][d] += fk * v[e][q][d];
      }
    }
  }
  if (!__all_sync(~0u, all)) return;
  const float vscale = a.p.v_scale ? __ldg(a.p.v_scale + h / a.shape.G) : 1.0f;
  const float s = l > 0.0f ? vscale / l : (l == 0.0f ? 0.0f : l);
#pragma unroll
  for (int q = 0; q < kParts; ++q) {
    uint16_t* dst = a.out + row * D + q * 128 + lane * kPart;
    const uint32_t lo = pack2<false>(acc[q][0] * s, acc[q][1] * s);
    if (kPart == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(lo, pack2<false>(acc[q][kPart - 2] * s, acc[q][kPart - 1] * s));
    else *reinterpret_cast<uint32_t*>(dst) = lo;
  }
  if (lane == 0 && a.lse) a.lse[row] = l == 0.0f ? -INFINITY : m * 0.6931471805599453f + logf(l);
}

// Records what the join step would have recorded.
__global__ void __launch_bounds__(256) prefix_check_kernel(const __grid_constant__ PrefixArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int i = blockIdx.x * 256 + threadIdx.x;
  Request own;
  if (i < a.groups) load_group(a, i);
  if (i < a.requests) request_of_group(a, i, group_of(a, i), &own);
}

// Rows a request, on average, up to which a request's own part is computed apart (measured below).
constexpr long long kOwnRowsTc = 96, kOwnRowsMma = 48;

// The kernels by rows an item.
enum Kind { kRow8, kMma16, kMma32, kMma64, kTc128, kTc256 };
Kind kind_of(const AttnArgs& a, int D, long long rows, long long pair) {
  if (rows > (D == 64 ? 48 : 32) && attention_tc_fits(a, D)) return rows > pair ? kTc256 : kTc128;
  return rows <= 8 ? kRow8 : (rows <= 16 ? kMma16 : (rows <= 32 ? kMma32 : kMma64));
}
template <int D, bool FP8>
cudaError_t launch_ring_kind(const PrefixArgs& a, Kind kind, cudaStream_t s) {
  if (kind == kRow8) return launch_row8<D, FP8>(a, s);
  if (kind == kMma16) return launch_mma<D, 1, FP8>(a, s);
  if (kind == kMma32) return launch_mma<D, 2, FP8>(a, s);
  return launch_mma<D, 4, FP8>(a, s);
}
cudaError_t launch_kind(const PrefixArgs& a, int D, bool fp8, Kind kind, cudaStream_t s) {
  if (kind >= kTc128) return launch_attention_tc(a, D, fp8, kind == kTc256, s);
  if (D == 64) return fp8 ? launch_ring_kind<64, true>(a, kind, s) : launch_ring_kind<64, false>(a, kind, s);
  if (D == 128) return fp8 ? launch_ring_kind<128, true>(a, kind, s) : launch_ring_kind<128, false>(a, kind, s);
  return fp8 ? launch_ring_kind<256, true>(a, kind, s) : launch_ring_kind<256, false>(a, kind, s);
}

}  // namespace
}  // namespace lowbit

using namespace lowbit;

extern "C" {

size_t lowbit_prefix_attention_workspace_bytes(int T, int B, int Hq, int Hk, int D) {
  if (lowbit_paged_attention_workspace_bytes(T, B, Hq, Hk, D) == 0) return 0;
  // Calls of more rows a request leave none to the join; those of fewer rows or requests need no more than this.
  const long long most = (D <= 128 ? kOwnRowsTc : kOwnRowsMma) * B * Hk;
  const size_t rows = (size_t)std::min((long long)T * Hq, most);
  return 2 * pieces_bytes(D) + rows * 2 * ((size_t)(D + 2) * sizeof(float) + sizeof(int4));
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
  const int D = cache->head_dim, B = a.p.B;
  if (!workspace || ws_bytes < lowbit_prefix_attention_workspace_bytes(a.p.T, B, Hq, cache->heads, D))
    return LOWBIT_ERR_WORKSPACE;
  if ((uintptr_t)workspace & 15) return LOWBIT_ERR_ALIGN;
  a.p.err = device_error_word();
  if (!a.p.err) return LOWBIT_ERR_CUDA;
  a.wide = (((uintptr_t)out | (uintptr_t)workspace) & 31) == 0;
  a.groups = groups;
  a.requests = B;
  a.cu_groups = cu_groups;
  a.prefix_lens = prefix_lens;
  a.rows = (long long)a.p.T * Hq;
  a.base_o = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + 2 * pieces_bytes(D));
  a.found = reinterpret_cast<int4*>(a.base_o + 2 * (size_t)a.rows * (size_t)D);
  a.base_ml = reinterpret_cast<float2*>(a.found + 2 * a.rows);
  const bool fp8 = cache->dtype == LOWBIT_CACHE_E4M3;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  use_pieces(&a, workspace, D);

  // By the rows that share keys, on average, in either part (the host knows the totals only, not the lengths).
  // From about 100 rows a request on, its own tiles are full and its keys come out of L2 for the requests that
  // follow: the plain call is as fast, and has no second part to join.  us here / plain, heads of 128, bf16:
  // 6 requests behind 12,345 keys, 128 rows each 65 / 52, 256 rows 97 / 89, 1,024 rows 305 / 303; 24 behind
  // 3,000, 256 rows 151 / 97; with 64 rows, 48 behind 16,000 215 / 377, 24 behind 3,000 53 / 53, 8 behind 8,000
  // 46 / 44; with four, 64 behind 16,384 69 / 279, 16 behind 4,000 20 / 25, 8 16 / 16, 64 behind 500 46 / 34.
  // On the warp-level MMA, whose items have 64 rows at most, from 50 on (heads of 256, 16 requests behind 6,000
  // keys, 64 rows each 89 / 82, 32 rows 54 / 55).
  const long long all = (long long)a.p.T * a.shape.G, shared_rows = (all + groups - 1) / groups, own_rows = (all + B - 1) / B;
  // Short requests are as quick on their own, too.  Their lengths the host knows a bound of, the block table's: us with
  // one row tile shared / on their own, bf16, 100 keys each behind 256, 1,024 and 2,048: 8 of four rows 12 / 8, 14 / 10,
  // 16 / 12, 32 22 / 12, 24 / 18, 24 / 26, 128 45 / 26, 49 / 49, 50 / 82; 16 of 64 rows 26 / 13, 29 / 24, 33 / 30, 128
  // 115 / 64, 139 / 107, 173 / 164.  Groups of 16 and less under 2,048 slots so, too, unless there are many: 42 of 32
  // rows in ten groups, e4m3, 42 / 32, 36 in nine 30 / 27, 22 of five rows in two 16 / 11; 64 of four rows in four
  // groups, behind 960 keys 52 / 54, 1,920 37 / 65. Under 1,024 slots it stays so with any number of requests (512 of
  // four rows behind 448 keys 185 / 127, 512 216 / 192, 960 192 / 227; heads of 64, 8 rows each 56 / 31, 65 / 39, 55 /
  // 44), but where reading a request's keys takes the plain kernels long: many few-row items over e4m3 (512 of four rows
  // 81 / 95, 125 / 138, 93 / 158, heads of 64 64 / 73, 94 / 105, 67 / 122; 2,048 with two heads 99 / 110, 140 / 156, 107
  // / 174; 256 56 / 54, 82 / 75, 56 / 86; eight rows each 69 / 58, 96 / 80, 76 / 91), and heads of 256 in bf16 (128 of
  // four rows 64 / 90, 102 / 139, 71 / 165; over e4m3 73 / 50, 119 / 70, 82 / 79).
  const long long reach = (long long)a.p.width << a.p.page_shift, items = (long long)B * cache->heads;
  const bool slow_alone = own_rows <= 4 && (D == 256 ? !fp8 && items >= 1024 : fp8 && items >= 4096);
  const bool brief = (reach <= 1024 && !slow_alone) ||
                     (reach <= 2048 && (own_rows > 32 || (B <= 16LL * groups && items * reach < 1 << 20)));
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr;
  cudaError_t e;
  if (brief || own_rows > (attention_tc_fits(a, D) ? kOwnRowsTc : kOwnRowsMma)) {
    attention_config(&cfg, &attr, (std::max(B, groups) + 255) / 256, 256, 0, s);
    e = cudaLaunchKernelEx(&cfg, prefix_check_kernel, a);
    if (e == cudaSuccess) e = launch_attention(a, D, fp8, s);
    return e == cudaSuccess ? LOWBIT_OK : LOWBIT_ERR_CUDA;
  }
  // 256 rows an item in the shared part read its keys half as often, but leave more of an item empty in the own part if
  // one launch takes both, and of the last one.  So they pay behind long prefixes, whose length the host knows a bound of,
  // the block table's.  us with 256 / 128, bf16, 16,000 keys shared: 12 requests of 64 rows 67 / 72, 24 112 / 131, 48 in four
  // groups 209 / 276, 5 48 / 41; 8,000 keys: 48 in four groups 145 / 157, 16 61 / 59; 4,000: 48 104 / 94, in four groups with
  // 1,500 keys of their own 153 / 139.  With a launch for each part, 256 requests of 16 rows 312 / 370 behind 16,000, 225 / 223
  // behind 4,000, 64 of 32 rows 168 / 167 and 122 / 98 (behind 6,000); over e4m3, 128 of 16 rows 194 / 213 behind 10,000, 136 /
  // 140 behind 6,000, 64 of 32 rows 187 / 198 behind 16,000, 125 / 121 behind 6,000.
  const Kind own_kind = kind_of(a, D, own_rows, 1024);
  const bool tall = shared_rows > 600 && (own_kind >= kTc128 ? reach > 8192
                                          : fp8             ? own_rows <= 16 || reach > 8192
                                                            : all * reach > 1 << 25);
  const Kind shared_kind = kind_of(a, D, shared_rows, tall ? 1 : 1 << 30);
  // One launch where the shared part's kernel suits the own part, which then costs no start of its own: where rows
  // fill an item half or more, items are few, or (128 rows an item) tiles need no conversion.  us in one / in
  // two launches: 32 requests of 32 rows behind 10,000 keys 74 / 88 (e4m3 85 / 93), 16 of 4 behind 4,000 20 / 22, 48 of
  // 64 behind 16,000 215 / 228; 64 of 4 behind 16,384 61 / 79 (e4m3 77 / 67), behind 500 52 / 54 (56 / 37), 128 of 4
  // behind 4,000 61 / 66 (70 / 51).
  const bool together = shared_kind == own_kind || shared_kind <= kMma64 || own_kind >= kTc128 ||
                        (shared_kind == kTc128 && (!fp8 || own_rows > 16 || (long long)B * cache->heads <= 152));
  PrefixArgs part = a;
  part.p.B = together ? groups + B : groups;
  e = launch_kind(part, D, fp8, shared_kind, s);
  if (e == cudaSuccess && !together) {
    part.p.B = B;
    part.first = groups;
    use_pieces(&part, static_cast<uint8_t*>(workspace) + pieces_bytes(D), D);
    e = launch_kind(part, D, fp8, own_kind, s);
  }
  if (e != cudaSuccess) return LOWBIT_ERR_CUDA;
  attention_config(&cfg, &attr, a.p.T, kPrefixJoinWarps * 32, 0, s);
  cfg.gridDim.y = (unsigned)((Hq + kPrefixJoinWarps - 1) / kPrefixJoinWarps);
  const float* own_o = part.piece_o;
  const float2* own_ml = part.piece_ml;
  e = D == 64 ? cudaLaunchKernelEx(&cfg, prefix_join_kernel<64>, a, own_o, own_ml)
    : D == 128 ? cudaLaunchKernelEx(&cfg, prefix_join_kernel<128>, a, own_o, own_ml)
               : cudaLaunchKernelEx(&cfg, prefix_join_kernel<256>, a, own_o, own_ml);
  return e == cudaSuccess ? LOWBIT_OK : LOWBIT_ERR_CUDA;
}

}  // extern "C"
