// Drafted tokens against the target's probabilities, from given uniform numbers.
//
// Draft d of a row is accepted where u q(d) < p(d); behind the accepted ones the next token comes from
//   max(p - q, 0), up to a factor,   after a rejection,   or from p where all were accepted,
// which leaves the tokens distributed as sampling from p alone would (p: the target's row under the request's
// settings, q: the drafter's).
//
// Two steps.  sample_kernel (sample.cuh), in the form that keeps a row's settled state instead of drawing
// from it, takes every row of the target and of the drafter: the largest logit, the cut that top-k, top-p and
// min-p come to, and the mass of what stays, in 32 bytes.  Then a cluster of CTAs per request looks up the
// drafted tokens' shares, which needs two logits each, finds the first rejection, and draws once: it sums
// the differences of its slice, the CTA that holds the aim takes it apart again, as in lowbit_sample.
//
// Differences are taken in fp32 of the two probabilities, each product and the difference rounded by
// itself, and become whole numbers (2^-40 each) before they are summed, so the sums are exact, in any order.
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
  int32_t* n_accept;
  int32_t* ids;
  float* accept;
  int* err;
};

__device__ __forceinline__ float logit_at(const void* row, bool bf16, int i) {
  return clean(bf16 ? bf16_bits_to_float(__ldg(static_cast<const uint16_t*>(row) + i)) : __ldg(static_cast<const float*>(row) + i));
}
// The weight of a token that the row's settings leave, 0 of another and of one without mass (where a cut through
// such tokens falls depends on the way that it was found).
__device__ __forceinline__ float kept_weight(const RowState& s, float z, int i) {
  const float w = weight_of(z, s.top, s.rate);
  return (((u64)down_key(z) << 32) | (uint32_t)i) <= s.cut && w > kLeast && !(w < s.floor_w) && s.total ? w : 0.0f;
}
// 2^40 / total: what a weight is multiplied by to become a probability.
__device__ __forceinline__ float inverse(const RowState& s) {
  return s.total ? (float)(0x1p40 / (double)s.total) : 0.0f;
}

struct VerifyShared {
  u64 warp_mass[kWarps], rank_mass[2][kMaxCluster];
  int first;
};

template <bool BF16, bool DRAFT_BF16>
__global__ void __launch_bounds__(kThreads, 2) verify_draw_kernel(const __grid_constant__ VerifyArgs a) {
  __shared__ VerifyShared s;
  constexpr int kSize = BF16 ? 2 : 4, kDraftSize = DRAFT_BF16 ? 2 : 4;
  const int C = a.cluster, rank = blockIdx.x % C, b = blockIdx.x / C;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int seg_from = warp * a.per_warp, seg_to = seg_from + a.per_warp;
  const int index0 = rank * kWarps * a.per_warp;
  cluster_arrive();  // this CTA runs: the others may write its shared memory
  if (tid == 0) s.first = INT32_MAX;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int c0 = a.cu_drafts[b], c1 = a.cu_drafts[b + 1];
  __syncthreads();
  if (!request_fits(b, c0, c1, a.N, a.M)) {
    if (rank == 0 && tid == 0) {
      record_error(a.err, LOWBIT_ERR_INVALID_ARG);
      a.n_accept[b] = 0;
    }
    cluster_wait();
    return;
  }
  const int n = c1 - c0;
  const uint8_t* const rows = static_cast<const uint8_t*>(a.logits);
  const uint8_t* const draft_rows = static_cast<const uint8_t*>(a.draft_logits);

  // ---- which drafts are accepted: every CTA finds out for itself
  for (int i = tid; i < n; i += kThreads) {
    const int r = c0 + i, d = a.drafts[r];
    const bool inside = d >= 0 && d < a.V;
    double share = 0.0, given = 1.0;
    if (inside) {
      const RowState p = a.target[r + b];
      const float z = logit_at(rows + (long long)(r + b) * a.row_stride * kSize, BF16, d);
      share = p.total ? (double)mass_of(kept_weight(p, z, d)) / (double)p.total : 0.0;
    }
    if (draft_rows) {
      given = 0.0;
      const int col = inside ? (a.draft_index ? a.draft_index[d] : d) : -1;
      if (col >= 0 && col < a.Vd) {
        const RowState q = a.draft[r];
        const float z = logit_at(draft_rows + (long long)r * a.draft_stride * kDraftSize, DRAFT_BF16, col);
        if (q.total) given = (double)mass_of(kept_weight(q, z, col)) / (double)q.total;
      }
    }
    float u = a.u[r];
    u = u >= 0.0f ? fminf(u, 1.0f) : 0.0f;
    if (!((double)u * given < share)) atomicMin(&s.first, i);
    if (rank == 0 && a.accept) a.accept[r] = given > 0.0 ? (float)fmin(share / given, 1.0) : (share > 0.0 ? 1.0f : 0.0f);
  }
  __syncthreads();
  const int j = min(s.first, n), t = c0 + b + j;  // the row that the next token comes from
  const RowState p = a.target[t];
  const bool rejected = j < n;
  if (rank == 0) {
    for (int i = tid; i <= n; i += kThreads)
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
  RowState q = {};
  if (rejected && draft_rows) q = a.draft[c0 + j];
  const int out = rejected && !draft_rows ? a.drafts[c0 + j] : -1;  // proposed with certainty
  const float ip = inverse(p), iq = inverse(q);
  // tokens below it have no mass, or are cut off
  const float cut_z = (uint32_t)(p.cut >> 32) == 0xFFFFFFFFu ? -INFINITY : key_logit((uint32_t)(p.cut >> 32));

  const Slice<BF16, false> z_of = {rows + (long long)t * a.row_stride * kSize + (long long)index0 * kSize,
                                   max(0, a.V - index0), a.aligned};
  const uint8_t* const draft_row = draft_rows + (long long)(c0 + j) * a.draft_stride * kDraftSize;
  const Slice<DRAFT_BF16, false> y_of = {draft_row + (long long)index0 * kDraftSize, max(0, a.Vd - index0), a.draft_aligned};

  // What four neighbouring tokens are drawn with, in units of 1: false where all of it is zero.
  bool differ = rejected;  // else p itself
  auto values = [&](int i, const float (&z)[4], float (&x)[4]) {
    const float most = fmaxf(fmaxf(z[0], z[1]), fmaxf(z[2], z[3]));
    if (!(most >= cut_z) || (most - p.top) * p.rate < -kReach) return false;
    bool any = false;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[e] = kept_weight(p, z[e], index0 + i + e);
      any |= x[e] > 0.0f;
    }
    if (!differ || !any) return any;
    if (draft_rows) {
      if (!a.draft_index) {
        float y[4];
        y_of.load4(i, y);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float w = index0 + i + e < a.Vd ? kept_weight(q, clean(y[e]), index0 + i + e) : 0.0f;
          x[e] = fmaxf(__fsub_rn(__fmul_rn(x[e], ip), __fmul_rn(w, iq)), 0.0f);
        }
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
          if (x[e] > 0.0f && col[e] >= 0 && col[e] < a.Vd) w = kept_weight(q, logit_at(draft_row, DRAFT_BF16, col[e]), col[e]);
          x[e] = fmaxf(__fsub_rn(__fmul_rn(x[e], ip), __fmul_rn(w, iq)), 0.0f);
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
    z_of.each4(from, to, [&](int i, float (&z)[4]) {
      float x[4];
      if (!values(i, z, x)) return false;
      parts += 4;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        uint32_t h, l;
        split_mass(x[e], h, l);
        hi += h, lo += l;
      }
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
      const u64 sum = warp_sum(lane < kWarps ? s.warp_mass[lane] : 0);
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
  const u64 aim = aim_of(a.v[b], total);
  const u64 slice = s.rank_mass[rejected && !differ ? 1 : 0][rank];
  if (aim < before || aim >= before + slice) return;

  // ---- the warp's segment that holds the aim, its sixteenth, then the token
  int from = seg_from, to = seg_to;
#pragma unroll 1
  for (int level = 0; level < 2; ++level) {
    int owner = 0;
    for (; owner < kWarps; ++owner) {
      if (aim < before + s.warp_mass[owner]) break;
      before += s.warp_mass[owner];
    }
    if (level == 1) {
      if (owner != warp) return;
      break;
    }
    const int each = ((a.per_warp / 128 + kWarps - 1) / kWarps) * 128;
    to = (owner + 1) * a.per_warp;
    from = min(owner * a.per_warp + warp * each, to);
    to = min(from + each, to);
    const u64 mine = sum_of(from, to);
    __syncthreads();
    if (lane == 0) s.warp_mass[warp] = mine;
    __syncthreads();
  }
  z_of.each4(from, to, [&](int i, float (&z)[4]) {
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
  // Slices of 16,384 elements and more, and no more CTAs than fit at a time.
  int C = 1;
  while (C < kMaxCluster && (long long)C * 16384 < a.V) C *= 2;
  while (C > 4 && (long long)a.B * C > 256) C /= 2;
  a.cluster = C;
  a.per_warp = ((a.V + C * kWarps - 1) / (C * kWarps) + 511) / 512 * 512;
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
  cfg.blockDim = dim3(kThreads);
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

cudaError_t launch_state(const StateArgs& a, bool bf16, cudaStream_t s) {
  return bf16 ? launch_rows<true>(a, s) : launch_rows<false>(a, s);
}
bool known(int dtype) { return dtype == LOWBIT_LOGITS_FP32 || dtype == LOWBIT_LOGITS_BF16; }

}  // namespace
}  // namespace lowbit

using namespace lowbit;

extern "C" {

size_t lowbit_verify_drafts_workspace_bytes(int M, int N) {
  if (M < 1 || M > 1 << 24 || N < 0 || N > 1 << 24) return 0;
  return ((size_t)M + (size_t)N) * sizeof(RowState);
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
  int* const err = device_error_word();
  if (!err) return LOWBIT_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  RowState* const states = static_cast<RowState*>(workspace);

  for (const lowbit_row_settings* r : {draft, target}) {
    if (!r || (r == draft && N == 0)) continue;
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
    st.cu_drafts = cu_drafts;
    st.B = B;
    st.N = N;
    st.rows = target->rows;
    st.extra = r == target;
    if (launch_state(st, r->dtype == LOWBIT_LOGITS_BF16, s) != cudaSuccess) return LOWBIT_ERR_CUDA;
  }
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
  a.n_accept = n_accept;
  a.ids = ids;
  a.accept = accept;
  a.err = err;
  const bool bf16 = target->dtype == LOWBIT_LOGITS_BF16, draft_bf16 = draft && draft->dtype == LOWBIT_LOGITS_BF16;
  const cudaError_t e = bf16 ? (draft_bf16 ? launch_draw<true, true>(a, s) : launch_draw<true, false>(a, s))
                             : (draft_bf16 ? launch_draw<false, true>(a, s) : launch_draw<false, false>(a, s));
  return e == cudaSuccess ? LOWBIT_OK : LOWBIT_ERR_CUDA;
}

}  // extern "C"
