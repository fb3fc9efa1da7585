// One token per row of logits under temperature, top-k, top-p and min-p, from a given uniform
// number (see include/lowbit.h for the definition).
//
// A weight w = exp((z - max) / T) becomes a whole number, w * 2^40 rounded, so every sum below is
// a 64-bit integer: exact, the same in any order, and free to be taken with atomics.
// Truncation is a prefix of the order (larger logit, then lower index): it is described by a
// threshold key and the number r of tokens equal to it that stay, the lowest r of them.  The
// prefix is found by histograms of counts and masses, first over 2048 equal steps of
// (max - z) / T -- 28.5 covers every weight that does not round to zero -- then over the digits of
// the key within the step that holds the cut.  The draw itself goes in index order over
// contiguous segments, so it needs only their kept masses and a walk through one of them.
//
// A cluster of CTAs takes one row, each a contiguous slice.
#include <atomic>

#include "common.cuh"
#include "ptx.cuh"

namespace lowbit {
namespace {

using namespace ptx;

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr int kMaxCluster = 8;
constexpr float kReach = 28.5f;  // 2^-41 = exp(-28.42)
constexpr int kMaxVocab = 1 << 19;

struct SampleArgs {
  const void* logits;
  long long row_stride;
  int M, V, cluster;
  const float* temperature;
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  const float* u;
  const int32_t* id_map;
  int32_t* ids;
  float* logprob;
  int32_t* kept;
};

template <bool BF16>
__device__ __forceinline__ float load_logit(const void* row, int i) {
  float z;
  if (BF16) z = bf16_bits_to_float(__ldg(static_cast<const uint16_t*>(row) + i));
  else z = __ldg(static_cast<const float*>(row) + i);
  if (!(z >= -INFINITY)) z = -INFINITY;  // NaN
  return fminf(z, 3.402823466e38f) + 0.0f;  // -0 becomes +0
}
// Ascending with descending z.
__device__ __forceinline__ uint32_t down_key(float z) {
  const uint32_t b = __float_as_uint(z);
  return (b & 0x80000000u) ? b : ~(b | 0x80000000u);
}
__device__ __forceinline__ float weight_of(float z, float top, float rate) {
  return z == -INFINITY ? 0.0f : expf((z - top) * rate);
}
__device__ __forceinline__ unsigned long long mass_of(float w) {
  return (unsigned long long)__float2ll_rn(w * 1099511627776.0f);
}
__device__ __forceinline__ int step_of(float z, float top, float steps) {
  return z == -INFINITY ? kBins - 1 : (int)fminf((top - z) * steps, (float)(kBins - 1));
}

struct Shared {
  uint32_t count[kBins], lo[kBins], hi[kBins];  // this CTA's histogram; the mass in two words
  uint32_t all_count[kBins];                    // the cluster's
  unsigned long long all_mass[kBins];
  unsigned long long warp_mass[kWarps];
  uint32_t warp_count[kWarps], warp_ties[kWarps];
  float rank_max[kMaxCluster];
  unsigned long long warp_tie[kWarps], rank_tie[kMaxCluster];  // mass of one token at the cut
  unsigned long long rank_mass[kMaxCluster];
  uint32_t rank_count[kMaxCluster], rank_ties[kMaxCluster];
  // the bin that a search found, and what precedes it
  int bin;
  uint32_t count_before;
  unsigned long long mass_before;
  float top;
};

__device__ __forceinline__ void st_dsmem_u64(uint32_t addr, unsigned long long v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}
__device__ __forceinline__ unsigned long long warp_incl(unsigned long long v, int lane) {
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long x = __shfl_up_sync(~0u, v, o);
    if (lane >= o) v += x;
  }
  return v;
}
__device__ __forceinline__ uint32_t warp_incl32(uint32_t v, int lane) {
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t x = __shfl_up_sync(~0u, v, o);
    if (lane >= o) v += x;
  }
  return v;
}

// Sums the CTAs' histograms into every CTA's all_count / all_mass.
__device__ void merge_histograms(Shared& s, int C, int rank) {
  cluster_sync();
  const int each = kBins / C;
  for (int i = threadIdx.x; i < each; i += kThreads) {
    const int bin = rank * each + i;
    uint32_t c = 0;
    unsigned long long m = 0;
    for (int r = 0; r < C; ++r) {
      c += ld_dsmem_u32(smem_addr(&s.count[bin]), r);
      m += ld_dsmem_u32(smem_addr(&s.lo[bin]), r) + ((unsigned long long)ld_dsmem_u32(smem_addr(&s.hi[bin]), r) << 32);
    }
    for (int r = 0; r < C; ++r) {
      st_dsmem_u32(map_to_rank(smem_addr(&s.all_count[bin]), r), c);
      st_dsmem_u64(map_to_rank(smem_addr(&s.all_mass[bin]), r), m);
    }
  }
  cluster_sync();
}
__device__ void clear_histogram(Shared& s) {
  for (int i = threadIdx.x; i < kBins; i += kThreads) s.count[i] = s.lo[i] = s.hi[i] = 0;
}
__device__ __forceinline__ void add_to_bin(Shared& s, int bin, unsigned long long mass) {
  atomicAdd(&s.count[bin], 1u);
  const uint32_t lo = (uint32_t)mass;
  uint32_t up = (uint32_t)(mass >> 32);
  if (lo && atomicAdd(&s.lo[bin], lo) > 0xFFFFFFFFu - lo) ++up;  // carry
  if (up) atomicAdd(&s.hi[bin], up);
}
// The first bin with (count up to it) >= k, or with (mass up to it) >= limit; s.bin = kBins if
// there is none.  All threads; the results are ready after it.
__device__ void find_bin(Shared& s, bool by_mass, uint32_t k, unsigned long long limit) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t c0 = s.all_count[2 * tid], c1 = s.all_count[2 * tid + 1];
  const unsigned long long m0 = s.all_mass[2 * tid], m1 = s.all_mass[2 * tid + 1];
  const uint32_t ci = warp_incl32(c0 + c1, lane);
  const unsigned long long mi = warp_incl(m0 + m1, lane);
  if (tid == 0) s.bin = kBins;
  if (lane == 31) s.warp_count[warp] = ci, s.warp_mass[warp] = mi;
  __syncthreads();
  uint32_t cb = ci - c0 - c1;
  unsigned long long mb = mi - m0 - m1;
  for (int w = 0; w < warp; ++w) cb += s.warp_count[w], mb += s.warp_mass[w];
  const bool pre = by_mass ? mb < limit : cb < k;
  const bool in0 = by_mass ? mb + m0 >= limit : cb + c0 >= k;
  const bool in1 = by_mass ? mb + m0 + m1 >= limit : cb + c0 + c1 >= k;
  if (pre && in1) {
    s.bin = in0 ? 2 * tid : 2 * tid + 1;
    s.count_before = in0 ? cb : cb + c0;
    s.mass_before = in0 ? mb : mb + m0;
  }
  __syncthreads();
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads, 1) sample_kernel(const SampleArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  Shared& s = *reinterpret_cast<Shared*>(smem);
  const int C = a.cluster, rank = blockIdx.x % C, m = blockIdx.x / C;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const void* row = static_cast<const uint8_t*>(a.logits) + (long long)m * a.row_stride * (BF16 ? 2 : 4);

  const float temp = a.temperature ? a.temperature[m] : 1.0f;
  const bool greedy = !(temp >= 1e-6f);
  const float rate = __frcp_rn(greedy ? 1.0f : fminf(temp, 1e6f));
  const int k_arg = a.top_k ? a.top_k[m] : 0;
  const uint32_t k = greedy ? 1u : (k_arg <= 0 || k_arg > a.V ? (uint32_t)a.V : (uint32_t)k_arg);
  const float p = a.top_p ? a.top_p[m] : 1.0f;
  const float min_p = a.min_p ? a.min_p[m] : 0.0f;
  const float floor_w = min_p > 0.0f ? fminf(min_p, 1.0f) : 0.0f;
  const float steps = rate * ((float)kBins / kReach);

  // segments: warp by warp, slice by slice, in index order
  const int per_warp = ((a.V + C * kWarps - 1) / (C * kWarps) + 31) / 32 * 32;
  const int i0 = (rank * kWarps + warp) * per_warp, i1 = min(a.V, i0 + per_warp);

  // ---- the largest logit
  float top = -INFINITY;
  for (int i = i0 + lane; i < i1; i += 32) top = fmaxf(top, load_logit<BF16>(row, i));
  for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
  if (lane == 0) s.warp_mass[warp] = __float_as_uint(top);
  clear_histogram(s);
  cluster_sync();  // every CTA of the cluster runs before its shared memory is written
  if (warp == 0) {
    top = __uint_as_float((uint32_t)s.warp_mass[lane]);
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
    if (lane < C) st_dsmem_f32(map_to_rank(smem_addr(&s.rank_max[rank]), lane), top);
  }
  cluster_sync();
  top = -INFINITY;
  for (int r = 0; r < C; ++r) top = fmaxf(top, s.rank_max[r]);
  if (top == -INFINITY) {  // no finite logit; the whole cluster agrees
    if (rank == 0 && tid == 0) {
      a.ids[m] = -1;
      if (a.logprob) a.logprob[m] = -INFINITY;
      if (a.kept) a.kept[m] = 0;
    }
    return;
  }

  // ---- the cut: tokens with key < cut stay, and the first r with key == cut
  uint32_t cut = 0xFFFFFFFFu, r_keep = 0xFFFFFFFFu;
  if (k < (uint32_t)a.V || !(p >= 1.0f)) {
    for (int i = i0 + lane; i < i1; i += 32) {
      const float z = load_logit<BF16>(row, i);
      const int bin = step_of(z, top, steps);
      if (bin < kBins - 1) add_to_bin(s, bin, mass_of(weight_of(z, top, rate)));
    }
    merge_histograms(s, C, rank);
    unsigned long long total = 0;
    // what lies past the last step has no mass: a cut there cuts nothing
    bool mass_turn = false;
    unsigned long long limit = 0;
    for (int turn = 0; turn < 2; ++turn) {
      if (turn == 0) {
        find_bin(s, false, k, 0);
      } else {
        if (p >= 1.0f) break;
        // ceil(p * S), at least 1: the mass that must precede what is dropped
        const double want = ceil((double)p * (double)total);
        limit = want >= 1.0 ? (unsigned long long)want : 1ull;
        mass_turn = true;
        find_bin(s, true, 0, limit);
      }
      const int bin = turn == 0 && k >= (uint32_t)a.V ? kBins : s.bin;
      uint32_t count_before = s.count_before;
      unsigned long long mass_before = s.mass_before;
      __syncthreads();
      if (bin == kBins) {  // nothing is cut (turn 0: fewer than k tokens have mass)
        if (turn == 0) {
          for (int i = lane; i < kBins; i += 32) total += s.all_mass[i];
          for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(~0u, total, o);
        }
        __syncthreads();
        continue;
      }
      // digits of the key among the tokens of that step: 11, 11 and 10 bits
      uint32_t prefix = 0;
      unsigned long long one = 0;  // mass of one token at the cut
      // level 0 of the histogram is needed again by the second turn: the digits use a copy
      for (int level = 0; level < 3; ++level) {
        const int shift = level == 0 ? 21 : (level == 1 ? 10 : 0);
        const uint32_t mask = level == 2 ? 1023u : 2047u;
        clear_histogram(s);
        __syncthreads();
        for (int i = i0 + lane; i < i1; i += 32) {
          const float z = load_logit<BF16>(row, i);
          if (step_of(z, top, steps) != bin) continue;
          const uint32_t key = down_key(z);
          if (level && (key >> (shift + (level == 2 ? 10 : 11))) != prefix) continue;
          add_to_bin(s, (key >> shift) & mask, mass_of(weight_of(z, top, rate)));
        }
        merge_histograms(s, C, rank);
        find_bin(s, mass_turn, k > count_before ? k - count_before : 0, limit - mass_before);
        const int d = s.bin;
        count_before += s.count_before;
        mass_before += s.mass_before;
        const uint32_t here = s.all_count[d];
        if (level == 2) one = s.all_mass[d] / here;  // equal keys, equal masses
        prefix = (prefix << (level == 2 ? 10 : 11)) | (uint32_t)d;
        __syncthreads();
      }
      cut = prefix;
      if (!mass_turn) {
        r_keep = k - count_before;
        total = mass_before + (unsigned long long)r_keep * one;
      } else {
        r_keep = (uint32_t)((limit - mass_before + one - 1) / one);
      }
      if (turn == 0 && !(p >= 1.0f)) {  // the first histogram again, for the second turn
        clear_histogram(s);
        __syncthreads();
        for (int i = i0 + lane; i < i1; i += 32) {
          const float z = load_logit<BF16>(row, i);
          const int bn = step_of(z, top, steps);
          if (bn < kBins - 1) add_to_bin(s, bn, mass_of(weight_of(z, top, rate)));
        }
        merge_histograms(s, C, rank);
      }
    }
  }

  // ---- kept mass of every segment
  unsigned long long mass = 0, tie_mass = 0;
  uint32_t count = 0, ties = 0;
  for (int i = i0 + lane; i < i1; i += 32) {
    const float z = load_logit<BF16>(row, i);
    const uint32_t key = down_key(z);
    if (key > cut) continue;
    const float w = weight_of(z, top, rate);
    const unsigned long long q = w >= floor_w ? mass_of(w) : 0;
    if (key == cut) ++ties, tie_mass = q;
    else mass += q, count += q != 0;
  }
  for (int o = 16; o; o >>= 1) {
    mass += __shfl_xor_sync(~0u, mass, o);
    count += __shfl_xor_sync(~0u, count, o);
    ties += __shfl_xor_sync(~0u, ties, o);
    const unsigned long long x = __shfl_xor_sync(~0u, tie_mass, o);
    tie_mass = x > tie_mass ? x : tie_mass;
  }
  if (lane == 0) {
    s.warp_mass[warp] = mass;
    s.warp_count[warp] = count;
    s.warp_ties[warp] = ties;
    s.warp_tie[warp] = tie_mass;
  }
  __syncthreads();
  if (warp == 0) {
    unsigned long long ms = s.warp_mass[lane], tm = s.warp_tie[lane];
    uint32_t cs = s.warp_count[lane], ts = s.warp_ties[lane];
    for (int o = 16; o; o >>= 1) {
      ms += __shfl_xor_sync(~0u, ms, o);
      cs += __shfl_xor_sync(~0u, cs, o);
      ts += __shfl_xor_sync(~0u, ts, o);
      const unsigned long long x = __shfl_xor_sync(~0u, tm, o);
      tm = x > tm ? x : tm;
    }
    if (lane < C) {
      st_dsmem_u64(map_to_rank(smem_addr(&s.rank_mass[rank]), lane), ms);
      st_dsmem_u32(map_to_rank(smem_addr(&s.rank_count[rank]), lane), cs);
      st_dsmem_u32(map_to_rank(smem_addr(&s.rank_ties[rank]), lane), ts);
      st_dsmem_u64(map_to_rank(smem_addr(&s.rank_tie[rank]), lane), tm);
    }
  }
  cluster_sync();  // the last exchange: no CTA touches another's memory after it
  unsigned long long total = 0, before = 0, one = 0;
  uint32_t kept = 0, ties_before = 0, seen = 0;
  for (int r = 0; r < C; ++r) one = s.rank_tie[r] > one ? s.rank_tie[r] : one;
  for (int r = 0; r < C; ++r) {
    if (r == rank) before = total, ties_before = seen;
    const uint32_t left = r_keep > seen ? r_keep - seen : 0;
    const uint32_t stay = s.rank_ties[r] < left ? s.rank_ties[r] : left;
    total += s.rank_mass[r] + stay * one;
    kept += s.rank_count[r] + (one ? stay : 0);
    seen += s.rank_ties[r];
  }
  float u = a.u[m];
  u = u >= 0.0f ? fminf(u, 1.0f) : 0.0f;
  const double want = floor((double)u * (double)total);
  unsigned long long aim = (unsigned long long)want;
  if (aim > total - 1) aim = total - 1;

  // ---- the segment that holds the aim, then the token
  for (int w = 0; w < warp; ++w) {
    const uint32_t left = r_keep > ties_before ? r_keep - ties_before : 0;
    const uint32_t stay = s.warp_ties[w] < left ? s.warp_ties[w] : left;
    before += s.warp_mass[w] + stay * one;
    ties_before += s.warp_ties[w];
  }
  {
    const uint32_t left = r_keep > ties_before ? r_keep - ties_before : 0;
    const uint32_t stay = s.warp_ties[warp] < left ? s.warp_ties[warp] : left;
    if (aim < before || aim >= before + s.warp_mass[warp] + stay * one) return;
  }
  for (int b = i0; b < i1; b += 32) {
    const int i = b + lane;
    unsigned long long q = 0;
    uint32_t key = 0xFFFFFFFFu;
    if (i < i1) {
      const float z = load_logit<BF16>(row, i);
      key = down_key(z);
      const float w = weight_of(z, top, rate);
      if (key <= cut && w >= floor_w) q = mass_of(w);
    }
    const uint32_t tie = __ballot_sync(~0u, i < i1 && key == cut);
    if (key == cut && ties_before + __popc(tie & ((1u << lane) - 1)) >= r_keep) q = 0;
    ties_before += __popc(tie);
    const unsigned long long incl = warp_incl(q, lane);
    const uint32_t hit = __ballot_sync(~0u, before + incl > aim);
    if (hit) {
      if (lane == __ffs(hit) - 1) {
        a.ids[m] = a.id_map ? a.id_map[i] : i;
        if (a.logprob) a.logprob[m] = logf((float)((double)q / (double)total));
        if (a.kept) a.kept[m] = (int32_t)kept;
      }
      return;
    }
    before += __shfl_sync(~0u, incl, 31);
  }
}

template <bool BF16>
cudaError_t launch(SampleArgs a, cudaStream_t s) {
  a.cluster = a.V > 65536 ? 8 : (a.V > 16384 ? 4 : 1);
  static std::atomic<int> ready[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!ready[dev].load(std::memory_order_relaxed)) {
    e = cudaFuncSetAttribute(sample_kernel<BF16>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Shared));
    if (e != cudaSuccess) return e;
    ready[dev].store(1, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.M * a.cluster));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = sizeof(Shared);
  cfg.stream = s;
  cudaLaunchAttribute attr[2] = {};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)a.cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, sample_kernel<BF16>, a);
}

}  // namespace
}  // namespace lowbit

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
  const SampleArgs a = {logits, row_stride, M, V, 1, temperature, top_k, top_p, min_p, u, id_map, ids, logprob, kept};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = dtype == LOWBIT_LOGITS_BF16 ? launch<true>(a, s) : launch<false>(a, s);
  return e == cudaSuccess ? LOWBIT_OK : LOWBIT_ERR_CUDA;
}
