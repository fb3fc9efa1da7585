// Drafted tokens against the target's probabilities, from given uniform numbers.
//
// Draft d of a row is accepted where u q(d) < p(d); behind the accepted ones the next token comes from
//   max(p - q, 0), up to a factor,   after a rejection,   or from p where all were accepted,
// which leaves the tokens distributed as sampling from p alone would (p: the target's row under the request's
// settings, q: the drafter's).
//
// Two steps.  sample_kernel (sample.cuh), in the form that keeps a row's settled state instead of drawing
// from it, takes every row of the target and of the drafter: the largest logit, the cut that top-k, top-p and
// min-p come to, and the mass of what stays, in 32 bytes, with a list of the target's tokens that stay where
// they are few.  Then a cluster of CTAs per request looks up the drafted tokens' shares, which needs two logits
// each, finds the first rejection, and draws once: from the list, or it sums the differences of its
// slices, and the CTA that holds the aim takes its own apart again, as in lowbit_sample.
//
// Differences are taken in fp32 of the two probabilities, each product and the difference rounded by
// itself, and become whole numbers (2^-40 each) before they are summed, so the sums are exact, in any order.
//
// Bound: few rows by round trips (15 drafts of one request proposed with certainty, 16 rows of 248,320: 20.6 us, of which
// the states take some 13 and the draw from a list the rest; the rows at the copy rate 2.4), many by the instructions of
// rows that sum masses (480 drafts of 32 requests under settings of all kinds, 574 MB: 204 to 248 us with the settings; 85 at
// the copy rate).  Where nothing is cut off and the next token comes from a difference, the draw weighs two rows of the
// vocabulary in 16 CTAs: 7 drafts of each of four requests against full drafter rows 34 us, 30 MB.  The states are a kernel
// of their own because they are the same for every row, whoever needs them, and spread over all SMs; the draw, which
// needs one row of a request, would leave most idle if it began from the logits.
#include "sample.cuh"

namespace lowbit {
namespace {

struct VerifyArgs {
  const void* logits;
  const void* draft_logits;  // NULL: the drafter proposes its token with certainty
  long long row_stride, draft_stride;
  int B, N, M, V, Vd, cluster;
  int per_warp;  // elements of a warp's segment, a multiple of 512
  int aligned, draft_aligned, index_aligned;  // rows (the index) start on 16-byte boundaries
  const int32_t* cu_drafts;
  const int32_t* drafts;
  const int32_t* draft_index;  // column of draft_logits by token, or NULL: the token itself
  const float* u;
  const float* v;
  const RowState* target;
  const RowState* draft;
  const u64* lists;  // [target row][kList]
  int32_t* n_accept;
  int32_t* ids;
  float* accept;
  int* err;
};

__device__ __forceinline__ float logit_at(const void* row, bool bf16, int i) {
  return bf16 ? bf16_bits_to_float(__ldg(static_cast<const uint16_t*>(row) + i)) : __ldg(static_cast<const float*>(row) + i);
}
// A row's state in the form that a token is tested in: its weight counts where the logit is above cut, or equal to
// it with an index up to `last`, and the weight is at least `least`, which leaves out those that min-p drops and
// those without mass (where a cut through such tokens falls depends on the way that it was found).
struct Kept {
  float top, rate, cut, least;
  uint32_t last;
  __device__ __forceinline__ explicit Kept(const RowState& s) : top(s.top), rate(s.rate) {
    const uint32_t key = (uint32_t)(s.cut >> 32);
    cut = !s.total ? INFINITY : (key == 0xFFFFFFFFu ? -INFINITY : key_logit(key));
    last = s.total ? (uint32_t)s.cut : 0u;
    least = s.total ? fmaxf(s.floor_w, __uint_as_float(__float_as_uint(kLeast) + 1)) : INFINITY;
  }
  // The logit as it was given: clipped to 0..1, the weight of an infinity is that of the largest number, which it is
  // also ordered as (a NaN comes to no weight before its place in the order counts).
  __device__ __forceinline__ float weight(float z, int i) const {
    const float w = __saturatef(weight_of(z, top, rate));
    z = fminf(z, 3.402823466e38f);
    return (z > cut || (z == cut && (uint32_t)i <= last)) && w >= least ? w : 0.0f;
  }
  // Of four neighbours, from token i on; a row that nothing is cut off takes the short way.
  __device__ __forceinline__ void weights4(const float (&z)[4], int i, float (&w)[4]) const {
#pragma unroll
    for (int e = 0; e < 4; e += 2) {
      const float2 x = mul2(add2(make_float2(z[e], z[e + 1]), both(-top)), both(rate));
      w[e] = __saturatef(expf(x.x)), w[e + 1] = __saturatef(expf(x.y));
    }
    if (cut == -INFINITY) {
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] = w[e] >= least ? w[e] : 0.0f;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float c = fminf(z[e], 3.402823466e38f);
        w[e] = (c > cut || (c == cut && (uint32_t)(i + e) <= last)) && w[e] >= least ? w[e] : 0.0f;
      }
    }
  }
};
// A thousand threads a CTA, so that few requests, which have 16 CTAs each at most, keep their SMs busy.
constexpr int kDrawThreads = 1024, kDrawWarps = kDrawThreads / 32;

struct VerifyShared {
  u64 warp_mass[kDrawWarps], rank_mass[2][kMaxCluster];
  u64 token[kList], mass[kList];  // a listed row's
  u64 aim;
  RowState p, q;  // of the rows that the next token comes from
  float ip, iq;
  int first, refused;  // the first draft that is not accepted, and its token
};

template <bool BF16, bool DRAFT_BF16>
__global__ void __launch_bounds__(kDrawThreads, 1) verify_draw_kernel(const __grid_constant__ VerifyArgs a) {
  __shared__ VerifyShared s;
  constexpr int kSize = BF16 ? 2 : 4, kDraftSize = DRAFT_BF16 ? 2 : 4;
  const int C = a.cluster, rank = blockIdx.x % C, b = blockIdx.x / C;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int seg_from = warp * a.per_warp, seg_to = seg_from + a.per_warp;
  const int index0 = rank * kDrawWarps * a.per_warp;
  cluster_arrive();  // this CTA runs: the others may write its shared memory
  if (tid == 0) s.first = INT32_MAX;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int c0 = a.cu_drafts[b], c1 = a.cu_drafts[b + 1];
  const bool fits = request_fits(b, c0, c1, a.N, a.M);
  const int n = fits ? c1 - c0 : 0;
  const uint8_t* const rows = static_cast<const uint8_t*>(a.logits);
  const uint8_t* const draft_rows = static_cast<const uint8_t*>(a.draft_logits);
  // What a draft is judged by, beside the rows' states: every CTA finds out for itself.
  struct Judged {
    int d, col;
    float z, y, u;
  };
  auto look = [&](int i) {
    const int r = c0 + i;
    Judged g = {a.drafts[r], -1, -INFINITY, -INFINITY, a.u[r]};
    if (g.d < 0 || g.d >= a.V) return g;
    g.z = logit_at(rows + (long long)(r + b) * a.row_stride * kSize, BF16, g.d);
    if (!draft_rows) return g;
    g.col = a.draft_index ? a.draft_index[g.d] : g.d;
    if (g.col >= a.Vd) g.col = -1;
    if (g.col >= 0) g.y = logit_at(draft_rows + (long long)r * a.draft_stride * kDraftSize, DRAFT_BF16, g.col);
    return g;
  };
  // (asked for together; the last thread has the state of the row behind all drafts)
  const float v = a.v[b];
  RowState p_seen = {}, q_seen = {};
  if (fits && (tid < n || tid == kDrawThreads - 1)) p_seen = a.target[c0 + b + min(tid, n)];
  if (tid < n && draft_rows) q_seen = a.draft[c0 + tid];
  Judged mine = {};
  if (tid < n) mine = look(tid);
  __syncthreads();
  if (!fits) {
    if (rank == 0 && tid == 0) {
      record_error(a.err, LOWBIT_ERR_INVALID_ARG);
      a.n_accept[b] = 0;
    }
    cluster_wait();
    return;
  }

  // ---- which drafts are accepted
  for (int i = tid; i < n; i += kDrawThreads) {
    const Judged g = i == tid ? mine : look(i);
    const int r = c0 + i;
    const RowState p = i == tid ? p_seen : a.target[r + b];
    double share = 0.0, given = draft_rows ? 0.0 : 1.0;
    if (g.d >= 0 && g.d < a.V && p.total) share = (double)mass_of(Kept(p).weight(g.z, g.d)) / (double)p.total;
    if (g.col >= 0) {
      const RowState q = i == tid ? q_seen : a.draft[r];
      if (q.total) given = (double)mass_of(Kept(q).weight(g.y, g.col)) / (double)q.total;
    }
    const float u = g.u >= 0.0f ? fminf(g.u, 1.0f) : 0.0f;
    if (!((double)u * given < share)) atomicMin(&s.first, i);
    if (rank == 0 && a.accept) a.accept[r] = given > 0.0 ? (float)fmin(share / given, 1.0) : (share > 0.0 ? 1.0f : 0.0f);
  }
  __syncthreads();
  const int j = min(s.first, n), t = c0 + b + j;  // the row that the next token comes from
  const bool rejected = j < n;
  // Its states, from the thread that has them, and 2^40 / S of both, what a weight is multiplied by to become
  // a probability: in the lanes of one warp, since 64-bit floating point is slow here (two a clock and SM).
  const int who = n >= kDrawThreads ? 0 : (rejected ? j : kDrawThreads - 1);
  if (n >= kDrawThreads && tid == 0) {
    p_seen = a.target[t];
    q_seen = rejected && draft_rows ? a.draft[c0 + j] : RowState{};
    mine.d = rejected ? a.drafts[c0 + j] : -1;
  }
  if (warp == who >> 5) {
    const u64 sp = __shfl_sync(~0u, p_seen.total, who & 31), sq = __shfl_sync(~0u, q_seen.total, who & 31);
    const u64 total = lane == 0 ? sp : sq;
    const float x = total ? (float)(0x1p40 / (double)total) : 0.0f;
    if (lane == 0) s.ip = x;
    if (lane == 1) s.iq = x;
    if (lane == (who & 31)) s.p = p_seen, s.q = q_seen, s.refused = mine.d;
  }
  __syncthreads();
  const RowState p = s.p, q = s.q;
  if (rank == 0) {
    for (int i = tid; i <= n; i += kDrawThreads)
      if (i != j) a.ids[c0 + b + i] = i < j ? a.drafts[c0 + i] : -1;
    if (tid == 0) {
      a.n_accept[b] = j;
      if (!p.total) a.ids[t] = -1;
    }
  }
  if (!p.total) {  // no finite logit; the whole cluster agrees
    cluster_wait();
    return;
  }
  if (p.listed && rank != 0) {  // the first CTA does it alone, and the whole cluster agrees
    cluster_wait();
    return;
  }
  const int out = rejected && !draft_rows ? s.refused : -1;  // proposed with certainty
  const float ip = s.ip, iq = s.iq;
  const uint8_t* const draft_row = draft_rows + (long long)(c0 + j) * a.draft_stride * kDraftSize;
  const Kept by_p(p), by_q(q);
  // What is left of a token's probability once the drafter's is taken off.
  auto left_of = [&](float w, float drafted) { return fmaxf(__fsub_rn(__fmul_rn(w, ip), __fmul_rn(drafted, iq)), 0.0f); };

  if (p.listed) {
    cluster_wait();
    const u64 entry = tid < p.listed ? a.lists[(long long)t * kList + tid] : 0;
    const int token = (int)(uint32_t)entry;
    float w = 0.0f, x = 0.0f;
    if (tid < p.listed) {
      w = by_p.weight(key_logit((uint32_t)(entry >> 32)), token);
      x = w;
      if (rejected && draft_rows) {
        const int col = a.draft_index ? __ldg(a.draft_index + token) : token;
        x = left_of(w, col >= 0 && col < a.Vd ? by_q.weight(logit_at(draft_row, DRAFT_BF16, col), col) : 0.0f);
      } else if (rejected) {
        x = token == out ? 0.0f : __fmul_rn(w, ip);
      }
    }
    u64 mine = mass_of(x);
    if (rejected && !__syncthreads_or(mine != 0)) mine = mass_of(w);
    if (tid < kList) s.token[tid] = token, s.mass[tid] = mine;
    const u64 sum = warp_sum(mine);
    if (lane == 0) s.warp_mass[warp] = sum;
    __syncthreads();
    if (warp == 0) {
      const u64 all = warp_sum(s.warp_mass[lane]);
      const u64 aim = aim_of(v, all);
      if (lane == 0) s.aim = aim;
    }
    __syncthreads();
    if (!mine) return;
    u64 before = 0;  // of the tokens with lower indices
    for (int i = 0; i < p.listed; ++i) before += s.token[i] < (u64)token ? s.mass[i] : 0;
    if (s.aim >= before && s.aim < before + mine) a.ids[t] = token;
    return;
  }

  const Slice<BF16, false> z_of = {rows + (long long)t * a.row_stride * kSize + (long long)index0 * kSize,
                                   max(0, a.V - index0), a.aligned};
  const Slice<DRAFT_BF16, false> y_of = {draft_row + (long long)index0 * kDraftSize, max(0, a.Vd - index0), a.draft_aligned};

  // What four neighbouring tokens are drawn with, in units of 1: false where all of it is zero.
  bool differ = rejected;  // else p itself
  auto values = [&](int i, const float (&z)[4], float (&x)[4]) {
    const float most = fmaxf(fmaxf(z[0], z[1]), fmaxf(z[2], z[3]));
    if (!(most >= by_p.cut) || (most - p.top) * p.rate < -kReach) return false;
    by_p.weights4(z, index0 + i, x);
    if (!differ) return true;
    if (draft_rows) {
      if (!a.draft_index) {
        float y[4], w[4];
        y_of.load4(i, y);  // -inf past the row
        by_q.weights4(y, index0 + i, w);
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = left_of(x[e], w[e]);
      } else {
        int col[4];
        if (a.index_aligned && index0 + i + 4 <= a.V) {
          *reinterpret_cast<int4*>(col) = __ldg(reinterpret_cast<const int4*>(a.draft_index + index0 + i));
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) col[e] = index0 + i + e < a.V ? __ldg(a.draft_index + index0 + i + e) : -1;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float w = 0.0f;
          if (x[e] > 0.0f && col[e] >= 0 && col[e] < a.Vd) w = by_q.weight(logit_at(draft_row, DRAFT_BF16, col[e]), col[e]);
          x[e] = left_of(x[e], w);
        }
      }
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = index0 + i + e == out ? 0.0f : __fmul_rn(x[e], ip);
    }
    return true;
  };
  auto sum_of = [&](int from, int to) {
    uint32_t hi = 0, lo = 0, parts = 0;
    z_of.template each4<false>(from, to, [&](int i, float (&z)[4]) {
      float x[4];
      if (!values(i, z, x)) return false;
      parts += 4;
      add_masses2(make_float2(x[0], x[1]), hi, lo);
      add_masses2(make_float2(x[2], x[3]), hi, lo);
      return false;
    });
    return warp_sum(join_mass(hi, lo, parts));
  };

  // ---- the mass of every CTA's slice; where the differences come to nothing, that of p
  u64 total = 0, before = 0;
  cluster_wait();
#pragma unroll 1
  for (int turn = 0; turn < 2; ++turn) {
    const u64 mine = sum_of(seg_from, seg_to);
    __syncthreads();  // warp_mass of the turn before has been read
    if (lane == 0) s.warp_mass[warp] = mine;
    __syncthreads();
    if (warp == 0) {
      const u64 sum = warp_sum(s.warp_mass[lane]);
      if (lane < C) st_dsmem_u64(map_to_rank(smem_addr(&s.rank_mass[turn][rank]), lane), sum);
    }
    cluster_sync();
    for (int r = 0; r < C; ++r) {
      if (r == rank) before = total;
      total += s.rank_mass[turn][r];
    }
    if (total || !differ) break;
    differ = false;
  }
  if (warp == 0) {
    const u64 at = aim_of(v, total);
    if (lane == 0) s.aim = at;
  }
  __syncthreads();
  const u64 aim = s.aim;
  const u64 slice = s.rank_mass[rejected && !differ ? 1 : 0][rank];
  if (aim < before || aim >= before + slice) return;

  // ---- the warp's segment that holds the aim, of its parts the one that does, then the token
  int from = seg_from, to = seg_to;
#pragma unroll 1
  for (int level = 0; level < 2; ++level) {
    int owner = 0;
    for (; owner < kDrawWarps; ++owner) {
      if (aim < before + s.warp_mass[owner]) break;
      before += s.warp_mass[owner];
    }
    if (level == 1) {
      if (owner != warp) return;
      break;
    }
    const int each = ((a.per_warp / 128 + kDrawWarps - 1) / kDrawWarps) * 128;
    to = (owner + 1) * a.per_warp;
    from = min(owner * a.per_warp + warp * each, to);
    to = min(from + each, to);
    const u64 mine = sum_of(from, to);
    __syncthreads();
    if (lane == 0) s.warp_mass[warp] = mine;
    __syncthreads();
  }
  z_of.template each4<false>(from, to, [&](int i, float (&z)[4]) {
    float x[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    u64 m[4], sum = 0;
    const bool some = values(i, z, x);
#pragma unroll
    for (int e = 0; e < 4; ++e) m[e] = some ? mass_of(x[e]) : 0, sum += m[e];
    const u64 incl = warp_incl(sum, lane);
    u64 at = before + incl - sum;
    const uint32_t hit = __ballot_sync(~0u, before + incl > aim);
    if (hit) {
      if (lane == __ffs(hit) - 1) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (aim >= at && aim < at + m[e]) a.ids[t] = index0 + i + e;
          at += m[e];
        }
      }
      return true;
    }
    before += __shfl_sync(~0u, incl, 31);
    return false;
  });
}

template <bool BF16, bool DRAFT_BF16>
cudaError_t launch_draw(VerifyArgs a, cudaStream_t s) {
  // Slices of up to 16,384 elements where the CTAs, one an SM, fit at a time, else longer ones, by two CTAs a request at least
  // (one where 16,384 hold the row).
  int C = 1;
  while (C < kMaxCluster && (long long)C * 16384 < a.V) C *= 2;
  while (C > 2 && (long long)a.B * C > 152) C /= 2;
  a.cluster = C;
  a.per_warp = ((a.V + C * kDrawWarps - 1) / (C * kDrawWarps) + 511) / 512 * 512;
  a.aligned = ((uintptr_t)a.logits & 15) == 0 && (a.row_stride * (BF16 ? 2 : 4)) % 16 == 0;
  a.draft_aligned = ((uintptr_t)a.draft_logits & 15) == 0 && (a.draft_stride * (DRAFT_BF16 ? 2 : 4)) % 16 == 0;
  a.index_aligned = ((uintptr_t)a.draft_index & 15) == 0;
  static std::atomic<int> ready[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!ready[dev].load(std::memory_order_relaxed)) {
    e = cudaFuncSetAttribute(verify_draw_kernel<BF16, DRAFT_BF16>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    ready[dev].store(1, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.B * C));
  cfg.blockDim = dim3(kDrawThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[2] = {};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)C;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, verify_draw_kernel<BF16, DRAFT_BF16>, a);
}

cudaError_t launch_state(const StatePair& a, int V, bool bf16, cudaStream_t s) {
  const int M = a.part[0].M + a.part[1].M;
  return bf16 ? launch_rows<true>(a, M, V, s) : launch_rows<false>(a, M, V, s);
}
// What a call reads or writes: the cluster's CTAs find out about a request each for itself, so what one of them
// writes must not be what another one reads.
struct Span {
  const void* at;
  __int128 bytes;
};
bool meet(const Span& x, const Span& y) {
  const __int128 a = (__int128)(uintptr_t)x.at, b = (__int128)(uintptr_t)y.at;
  return x.at && y.at && x.bytes && y.bytes && a < b + y.bytes && b < a + x.bytes;
}
bool known(int dtype) { return dtype == LOWBIT_LOGITS_FP32 || dtype == LOWBIT_LOGITS_BF16; }

}  // namespace
}  // namespace lowbit

using namespace lowbit;

extern "C" {

size_t lowbit_verify_drafts_workspace_bytes(int M, int N) {
  if (M < 1 || M > 1 << 24 || N < 0 || N > 1 << 24) return 0;
  return ((size_t)M + (size_t)N) * sizeof(RowState) + (size_t)M * kList * sizeof(u64);
}

lowbit_status lowbit_verify_drafts(const lowbit_row_settings* target, const lowbit_row_settings* draft, int B, int N,
                                   const int32_t* cu_drafts, const int32_t* drafts, const int32_t* draft_index,
                                   const float* u, const float* v, int32_t* n_accept, int32_t* ids, float* accept,
                                   void* workspace, size_t ws_bytes, void* stream) {
  if (!target || !target->logits || !known(target->dtype) || !cu_drafts || !v || !n_accept || !ids || (N > 0 && (!drafts || !u)) ||
      (draft && N > 0 && (!draft->logits || !known(draft->dtype))) || (draft_index && !draft))
    return LOWBIT_ERR_INVALID_ARG;
  if (B < 1 || B > 1 << 16 || N < 0 || N > 1 << 24 || target->rows < 1 || target->rows > 1 << 24 || target->V < 1 ||
      target->V > kMaxVocab || target->row_stride < target->V)
    return LOWBIT_ERR_SHAPE;
  if (draft && (draft->V < 1 || draft->V > kMaxVocab || draft->row_stride < draft->V || draft->rows != N)) return LOWBIT_ERR_SHAPE;
  uintptr_t words = (uintptr_t)cu_drafts | (uintptr_t)drafts | (uintptr_t)draft_index | (uintptr_t)u | (uintptr_t)v |
                    (uintptr_t)n_accept | (uintptr_t)ids | (uintptr_t)accept;
  for (const lowbit_row_settings* r : {target, draft}) {
    if (!r) continue;
    words |= (uintptr_t)r->temperature | (uintptr_t)r->top_k | (uintptr_t)r->top_p | (uintptr_t)r->min_p |
             ((uintptr_t)r->logits & (r->dtype == LOWBIT_LOGITS_BF16 ? 1 : 3)) << (r->dtype == LOWBIT_LOGITS_BF16 ? 1 : 0);
  }
  if (words & 3) return LOWBIT_ERR_ALIGN;
  if (!workspace || ws_bytes < lowbit_verify_drafts_workspace_bytes(target->rows, N)) return LOWBIT_ERR_WORKSPACE;
  if ((uintptr_t)workspace & 15) return LOWBIT_ERR_ALIGN;
  const Span written[] = {{n_accept, (__int128)B * 4}, {ids, (__int128)target->rows * 4}, {accept, (__int128)N * 4},
                          {workspace, (__int128)lowbit_verify_drafts_workspace_bytes(target->rows, N)}};
  Span read[16] = {{cu_drafts, (__int128)(B + 1) * 4}, {drafts, (__int128)N * 4}, {draft_index, (__int128)target->V * 4},
                   {u, (__int128)N * 4}, {v, (__int128)B * 4}};
  int reads = 5;
  for (const lowbit_row_settings* r : {target, draft}) {
    if (!r) continue;
    const __int128 size = r->dtype == LOWBIT_LOGITS_BF16 ? 2 : 4;
    read[reads++] = {r->logits, r->rows < 1 ? 0 : ((__int128)(r->rows - 1) * r->row_stride + r->V) * size};
    for (const void* x : {(const void*)r->temperature, (const void*)r->top_k, (const void*)r->top_p, (const void*)r->min_p})
      read[reads++] = {x, (__int128)B * 4};
  }
  for (int i = 0; i < 4; ++i) {
    for (int k = 0; k < reads; ++k)
      if (meet(written[i], read[k])) return LOWBIT_ERR_INVALID_ARG;
    for (int k = 0; k < i; ++k)
      if (meet(written[i], written[k])) return LOWBIT_ERR_INVALID_ARG;
  }
  int* const err = device_error_word();
  if (!err) return LOWBIT_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  RowState* const states = static_cast<RowState*>(workspace);
  u64* const lists = reinterpret_cast<u64*>(states + target->rows + N);
  const bool drafter = draft && N > 0;

  auto rows_of = [&](const lowbit_row_settings* r) {
    StateArgs st = {};
    st.logits = r->logits;
    st.row_stride = r->row_stride;
    st.M = r->rows;
    st.V = r->V;
    st.temperature = r->temperature;
    st.top_k = r->top_k;
    st.top_p = r->top_p;
    st.min_p = r->min_p;
    st.state = r == target ? states : states + target->rows;
    st.lists = r == target ? lists : nullptr;
    st.cu_drafts = cu_drafts;
    st.B = B;
    st.N = N;
    st.rows = target->rows;
    st.extra = r == target;
    return st;
  };
  const bool bf16 = target->dtype == LOWBIT_LOGITS_BF16, draft_bf16 = draft && draft->dtype == LOWBIT_LOGITS_BF16;
  StatePair pair = {};
  pair.part[0] = rows_of(target);
  if (drafter) {
    // Both in one launch, so that the short rows fill the gaps of the long ones (28 drafts of four requests 34 us, 40
    // one after the other; with the settings of one seed, 67 of nine with a trimmed vocabulary 59 and 67; 480 of 32 206 and 218).
    if (bf16 == draft_bf16) {
      pair.part[1] = rows_of(draft);
    } else {
      StatePair alone = {};
      alone.part[0] = rows_of(draft);
      if (launch_state(alone, draft->V, draft_bf16, s) != cudaSuccess) return LOWBIT_ERR_CUDA;
    }
  }
  if (launch_state(pair, pair.part[1].M ? std::max(target->V, draft->V) : target->V, bf16, s) != cudaSuccess) return LOWBIT_ERR_CUDA;
  VerifyArgs a = {};
  a.logits = target->logits;
  a.row_stride = target->row_stride;
  a.B = B;
  a.N = N;
  a.M = target->rows;
  a.V = target->V;
  if (draft) {
    a.draft_logits = draft->logits;
    a.draft_stride = draft->row_stride;
    a.Vd = draft->V;
  }
  a.cu_drafts = cu_drafts;
  a.drafts = drafts;
  a.draft_index = draft_index;
  a.u = u;
  a.v = v;
  a.target = states;
  a.draft = states + target->rows;
  a.lists = lists;
  a.n_accept = n_accept;
  a.ids = ids;
  a.accept = accept;
  a.err = err;
  const cudaError_t e = bf16 ? (draft_bf16 ? launch_draw<true, true>(a, s) : launch_draw<true, false>(a, s))
                             : (draft_bf16 ? launch_draw<false, true>(a, s) : launch_draw<false, false>(a, s));
  return e == cudaSuccess ? LOWBIT_OK : LOWBIT_ERR_CUDA;
}

}  // extern "C"
