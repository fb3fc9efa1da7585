// One token per row of logits under temperature, top-k, top-p and min-p, from a given uniform
// number (see include/lowbit.h for the definition).
//
// A weight w = exp((z - max) / T) becomes a whole number, w * 2^40 rounded, so every sum below is
// a 64-bit integer: exact, the same in any order, and free to be taken with atomics.
//
// A cluster of CTAs takes one row, each a contiguous slice that stays in its shared memory, so the
// row is read once.  Truncation keeps a prefix of the order (larger logit, then lower index):
//   1. the largest logit, over the cluster;
//   2. with top-p alone, the whole mass S.  What stays ends among the weights above (1 - p) S / V,
//      since the others sum to (1 - p) S at most, so only those are looked at further;
//   3. a histogram over 1024 equal steps of (max - z) / T (28.5 covers every weight that does not
//      round to zero) of counts, or of counts and masses, merged over the cluster: the step in
//      which the prefix ends, and how many tokens (n) lie up to it;
//   4. n <= 2048, nearly always: those tokens go to the first CTA, which sorts them (grouped by
//      step already, so a token is only compared with its own step's) and finishes the row;
//      else the cut is narrowed down by the key's digits to a threshold key and the number of
//      tokens equal to it that stay, and the draw walks the segments that the warps own.
#include <algorithm>
#include <atomic>

#include "common.cuh"
#include "ptx.cuh"

namespace lowbit {
namespace {

using namespace ptx;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 1024;
constexpr int kCap = 2048;       // candidates that the first CTA can finish
constexpr int kMaxCluster = 16;
constexpr float kReach = 28.5f;  // 2^-41 = exp(-28.42)
constexpr int kMaxVocab = 1 << 19;
typedef unsigned long long u64;

struct SampleArgs {
  const void* logits;
  long long row_stride;
  int M, V, cluster;
  int per_warp;   // elements of a warp's segment, a multiple of 128
  int aligned;    // every row starts on a 16-byte boundary
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

__device__ __forceinline__ float clean(float z) {
  if (!(z >= -INFINITY)) z = -INFINITY;     // NaN
  return fminf(z, 3.402823466e38f) + 0.0f;  // -0 becomes +0
}
// Ascending with descending z, and back.
__device__ __forceinline__ uint32_t down_key(float z) {
  const uint32_t b = __float_as_uint(z);
  return (b & 0x80000000u) ? b : ~(b | 0x80000000u);
}
__device__ __forceinline__ float key_logit(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? k : ~k & 0x7FFFFFFFu);
}
__device__ __forceinline__ float weight_of(float z, float top, float rate) {
  return z == -INFINITY ? 0.0f : expf((z - top) * rate);
}
// w * 2^40 rounded, as hi * 2^20 + lo: both parts are taken by adding 1.5 * 2^23, which leaves the
// rounded integer in the low bits; the remainder between them is exact.
constexpr float kMagic = 12582912.0f;
constexpr uint32_t kMagicBits = 0x4B400000u;
__device__ __forceinline__ void split_mass(float w, uint32_t& hi, uint32_t& lo) {
  const float f = w * 1048576.0f, t = f + kMagic;
  hi = __float_as_uint(t) - kMagicBits;
  lo = __float_as_uint(fmaf(f - (t - kMagic), 1048576.0f, kMagic)) - kMagicBits;  // signed
}
__device__ __forceinline__ u64 mass_of(float w) {
  uint32_t hi, lo;
  split_mass(w, hi, lo);
  return (u64)(((long long)(int)hi << 20) + (int)lo);
}
__device__ __forceinline__ int step_of(float z, float top, float steps) {
  return z == -INFINITY ? kBins - 1 : (int)fminf((top - z) * steps, (float)(kBins - 1));
}

struct Shared {
  uint32_t count[kBins], lo[kBins], hi[kBins];  // this CTA's histogram; the mass in two words
  uint32_t all_count[kBins];                    // the cluster's
  u64 all_mass[kBins];
  u64 cand[kCap];                               // first CTA: key << 32 | index, grouped by step
  u64 warp_mass[kWarps], warp_tie[kWarps];
  uint32_t warp_count[kWarps], warp_ties[kWarps];
  float warp_max[kWarps], rank_max[kMaxCluster];
  u64 rank_mass[kMaxCluster], rank_tie[kMaxCluster], rank_total[kMaxCluster];
  uint32_t rank_count[kMaxCluster], rank_ties[kMaxCluster];
  // the bin that a search found, and what precedes it
  int bin, found;
  uint32_t count_before, kept;
  u64 mass_before, total, kept_mass;
};

__device__ __forceinline__ void st_dsmem_u64(uint32_t addr, u64 v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}
__device__ __forceinline__ u64 warp_incl(u64 v, int lane) {
  for (int o = 1; o < 32; o <<= 1) {
    const u64 x = __shfl_up_sync(~0u, v, o);
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
__device__ __forceinline__ u64 warp_sum(u64 v) {
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  return v;
}

// Sums the CTAs' histograms into every CTA's all_count / all_mass.
__device__ __noinline__ void merge_histograms(Shared& s, int C, int rank, bool masses) {
  cluster_sync();
  const int each = kBins / C;
  // a bin's words of all CTAs lie with neighbouring threads, so that their loads overlap
  for (int i = threadIdx.x; i < each * C; i += kThreads) {
    const int bin = rank * each + i / C, r = i % C;  // C divides 32
    uint32_t c = ld_dsmem_u32(smem_addr(&s.count[bin]), r);
    u64 m = 0;
    if (masses) m = ld_dsmem_u32(smem_addr(&s.lo[bin]), r) + ((u64)ld_dsmem_u32(smem_addr(&s.hi[bin]), r) << 32);
    for (int o = C / 2; o; o >>= 1) {
      c += __shfl_xor_sync(~0u, c, o);
      if (masses) m += __shfl_xor_sync(~0u, m, o);
    }
    st_dsmem_u32(map_to_rank(smem_addr(&s.all_count[bin]), r), c);
    if (masses) st_dsmem_u64(map_to_rank(smem_addr(&s.all_mass[bin]), r), m);
  }
  cluster_sync();
}
__device__ __forceinline__ void clear_histogram(Shared& s) {
  for (int i = threadIdx.x; i < kBins; i += kThreads) s.count[i] = s.lo[i] = s.hi[i] = 0;
}
__device__ __forceinline__ void add_mass(Shared& s, int bin, u64 mass) {
  const uint32_t lo = (uint32_t)mass;
  uint32_t up = (uint32_t)(mass >> 32);
  if (lo && atomicAdd(&s.lo[bin], lo) > 0xFFFFFFFFu - lo) ++up;  // carry
  if (up) atomicAdd(&s.hi[bin], up);
}
// The first bin with (count up to it) >= k, or with (mass up to it) >= limit, and what precedes
// it; s.bin = kBins if there is none, with the whole count and mass.  Turns all_count into the
// counts that precede each bin when `prefix`.  All threads; the results are ready after it.
__device__ __noinline__ void find_bin(Shared& s, bool by_mass, uint32_t k, u64 limit, bool prefix) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t c0 = s.all_count[2 * tid], c1 = s.all_count[2 * tid + 1];
  const u64 m0 = by_mass ? s.all_mass[2 * tid] : 0, m1 = by_mass ? s.all_mass[2 * tid + 1] : 0;
  const uint32_t ci = warp_incl32(c0 + c1, lane);
  const u64 mi = by_mass ? warp_incl(m0 + m1, lane) : 0;
  if (lane == 31) s.warp_count[warp] = ci, s.warp_mass[warp] = mi;
  if (tid == 0) s.bin = kBins;
  __syncthreads();
  uint32_t cb = ci - c0 - c1;
  u64 mb = mi - m0 - m1;
  for (int w = 0; w < warp; ++w) cb += s.warp_count[w], mb += s.warp_mass[w];
  const bool pre = by_mass ? mb < limit : cb < k;
  const bool in0 = by_mass ? mb + m0 >= limit : cb + c0 >= k;
  const bool in1 = by_mass ? mb + m0 + m1 >= limit : cb + c0 + c1 >= k;
  if (pre && in1) {
    s.bin = in0 ? 2 * tid : 2 * tid + 1;
    s.count_before = in0 ? cb : cb + c0;
    s.mass_before = in0 ? mb : mb + m0;
    s.found = in0 ? c0 : c1;
  } else if (tid == kThreads - 1 && !in1) {
    s.count_before = cb + c0 + c1;
    s.mass_before = mb + m0 + m1;
    s.found = 0;
  }
  if (prefix) s.all_count[2 * tid] = cb, s.all_count[2 * tid + 1] = cb + c0;
  __syncthreads();
}

// ceil(p * S), at least 1: the mass that must precede what top-p drops.
__device__ __forceinline__ u64 top_p_limit(float p, u64 total) {
  const double want = ceil((double)p * (double)total);
  return want >= 1.0 ? (u64)want : 1ull;
}
// floor(u * S), below S.
__device__ __forceinline__ u64 aim_of(float u, u64 total) {
  u = u >= 0.0f ? fminf(u, 1.0f) : 0.0f;
  const u64 aim = (u64)floor((double)u * (double)total);
  return aim < total ? aim : total - 1;
}
__device__ __forceinline__ void finish(const SampleArgs& a, int m, int i, u64 mass, u64 total, uint32_t kept) {
  a.ids[m] = a.id_map ? a.id_map[i] : i;
  if (a.logprob) a.logprob[m] = logf((float)((double)mass / (double)total));
  if (a.kept) a.kept[m] = (int32_t)kept;
}

template <bool BF16>
struct Slice;
template <>
struct Slice<false> {
  const float* at;
  __device__ __forceinline__ void get4(int i, float (&z)[4]) const {
    const float4 v = *reinterpret_cast<const float4*>(at + i);
    z[0] = v.x, z[1] = v.y, z[2] = v.z, z[3] = v.w;
  }
};
template <>
struct Slice<true> {
  const uint16_t* at;
  __device__ __forceinline__ void get4(int i, float (&z)[4]) const {
    const uint2 v = *reinterpret_cast<const uint2*>(at + i);
    z[0] = clean(__uint_as_float(v.x << 16)), z[1] = clean(__uint_as_float(v.x & 0xFFFF0000u));
    z[2] = clean(__uint_as_float(v.y << 16)), z[3] = clean(__uint_as_float(v.y & 0xFFFF0000u));
  }
};

// The first CTA's end of a row: n candidates, grouped by step (all_count holds where each step
// begins), of which top-k, top-p and min-p keep a part; then the draw in index order.
__device__ __forceinline__ void finish_candidates(const SampleArgs& a, Shared& s, ulonglong2* sorted, int m, uint32_t n,
                                                  int last_bin, uint32_t k, float p, u64 whole, float floor_w,
                                                  float top, float rate, float steps, float u) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // rank inside the step, then the sorted place
  for (uint32_t i = tid; i < n; i += kThreads) {
    const u64 c = s.cand[i];
    const float z = key_logit((uint32_t)(c >> 32));
    const int bin = step_of(z, top, steps);
    const uint32_t from = s.all_count[bin], to = bin == last_bin ? n : s.all_count[bin + 1];
    uint32_t r = from;
    for (uint32_t j = from; j < to; ++j) r += s.cand[j] < c;
    sorted[r] = make_ulonglong2(c, mass_of(weight_of(z, top, rate)));
  }
  for (int i = tid; i < kBins; i += kThreads) s.lo[i] = s.hi[i] = 0;
  __syncthreads();
  // masses before each place; a thread takes four places in a row
  constexpr int kOwn = kCap / kThreads;
  u64 c[kOwn], q[kOwn], sum = 0;
#pragma unroll
  for (int e = 0; e < kOwn; ++e) {
    const uint32_t i = tid * kOwn + e;
    const ulonglong2 v = i < n ? sorted[i] : make_ulonglong2(0, 0);
    c[e] = v.x, q[e] = i < k ? v.y : 0;
    sum += q[e];
  }
  const u64 incl = warp_incl(sum, lane);
  if (lane == 31) s.warp_mass[warp] = incl;
  __syncthreads();
  u64 before = incl - sum, total = 0;
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += s.warp_mass[w];
    total += s.warp_mass[w];
  }
  if (k >= (uint32_t)a.V) total = whole;  // top-p of the whole row's mass
  const u64 limit = p >= 1.0f ? ~0ull : top_p_limit(p, total);
  const int shift = max(0, 32 - __clz(a.V - 1) - 10);  // 1024 buckets of indices
  uint32_t kept = 0;
  u64 mine = 0;
#pragma unroll
  for (int e = 0; e < kOwn; ++e) {
    const u64 at = before;
    before += q[e];
    if (at >= limit || (floor_w > 0.0f && weight_of(key_logit((uint32_t)(c[e] >> 32)), top, rate) < floor_w)) q[e] = 0;
    if (q[e]) ++kept, mine += q[e], add_mass(s, (int)((uint32_t)c[e] >> shift), q[e]);
  }
  mine = warp_sum(mine);
  for (int o = 16; o; o >>= 1) kept += __shfl_xor_sync(~0u, kept, o);
  __syncthreads();  // warp_mass has been read
  if (lane == 0) s.warp_mass[warp] = mine, s.warp_count[warp] = kept;
  __syncthreads();
  total = 0, kept = 0;
  for (int w = 0; w < kWarps; ++w) total += s.warp_mass[w], kept += s.warp_count[w];
  const u64 aim = aim_of(u, total);
  // the bucket that holds the aim
  {
    const u64 m0 = s.lo[2 * tid] + ((u64)s.hi[2 * tid] << 32), m1 = s.lo[2 * tid + 1] + ((u64)s.hi[2 * tid + 1] << 32);
    const u64 bi = warp_incl(m0 + m1, lane);
    if (lane == 31) s.warp_tie[warp] = bi;
    if (tid == 0) s.found = 0;
    __syncthreads();
    u64 b = bi - m0 - m1;
    for (int w = 0; w < warp; ++w) b += s.warp_tie[w];
    if (aim >= b && aim < b + m0 + m1) {
      const bool second = aim >= b + m0;
      s.bin = 2 * tid + second;
      s.mass_before = second ? b + m0 : b;
    }
    __syncthreads();
  }
  // its kept tokens (at most 2^19 / 1024), then the one whose share holds the aim
  const int bucket = s.bin;
  const u64 base = s.mass_before;
#pragma unroll
  for (int e = 0; e < kOwn; ++e)
    if (q[e] && (int)((uint32_t)c[e] >> shift) == bucket)
      sorted[atomicAdd(&s.found, 1)] = make_ulonglong2(c[e] & 0xFFFFFFFFu, q[e]);
  __syncthreads();
  const int found = s.found;
  for (int i = tid; i < found; i += kThreads) {
    const ulonglong2 v = sorted[i];
    u64 b = base;
    for (int j = 0; j < found; ++j) b += sorted[j].x < v.x ? sorted[j].y : 0;
    if (aim >= b && aim < b + v.y) finish(a, m, (int)v.x, v.y, total, kept);
  }
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const __grid_constant__ SampleArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  Shared& s = *reinterpret_cast<Shared*>(smem);
  uint8_t* const store = smem + (sizeof(Shared) + 15) / 16 * 16;
  constexpr int kSize = BF16 ? 2 : 4;
  const int C = a.cluster, rank = blockIdx.x % C, m = blockIdx.x / C;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int local = warp * a.per_warp + lane * 4;              // this lane's first place in the slice
  const int local_end = (warp + 1) * a.per_warp;
  const int index0 = rank * kWarps * a.per_warp;               // of the slice's first element
  asm volatile("griddepcontrol.wait;" ::: "memory");

  // the row's settings, asked for before the slice
  const float temp = a.temperature ? a.temperature[m] : 1.0f;
  const bool greedy = !(temp >= 1e-6f);
  const float rate = __frcp_rn(greedy ? 1.0f : fminf(temp, 1e6f));
  const int k_arg = a.top_k ? a.top_k[m] : 0;
  const uint32_t k = greedy ? 1u : (k_arg <= 0 || k_arg > a.V ? (uint32_t)a.V : (uint32_t)k_arg);
  const float p = a.top_p ? a.top_p[m] : 1.0f;
  const float min_p = a.min_p ? a.min_p[m] : 0.0f;
  const float floor_w = min_p > 0.0f ? fminf(min_p, 1.0f) : 0.0f;
  const float u = a.u[m];
  const float steps = rate * ((float)kBins / kReach);

  // ---- the slice comes in, and its largest logit; places past the row hold -inf
  float top = -INFINITY;
  {
    const uint8_t* row = static_cast<const uint8_t*>(a.logits) + (long long)m * a.row_stride * kSize;
    constexpr int kVec = 16 / kSize;                           // elements of a 16-byte load
    const int first = warp * a.per_warp;
    if (a.aligned) {
#pragma unroll 4
      for (int i = first + lane * kVec; i < local_end; i += 32 * kVec) {
        const int at = index0 + i;
        uint4 v;
        if (at + kVec <= a.V) {
          v = ld_stream(reinterpret_cast<const uint4*>(row + (long long)at * kSize));
        } else {
          uint32_t w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if (BF16) {
              const uint32_t x = at + 2 * e < a.V ? reinterpret_cast<const uint16_t*>(row)[at + 2 * e] : 0xFF80u;
              const uint32_t y = at + 2 * e + 1 < a.V ? reinterpret_cast<const uint16_t*>(row)[at + 2 * e + 1] : 0xFF80u;
              w[e] = x | y << 16;
            } else {
              w[e] = at + e < a.V ? reinterpret_cast<const uint32_t*>(row)[at + e] : 0xFF800000u;
            }
          }
          v = make_uint4(w[0], w[1], w[2], w[3]);
        }
        uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (BF16) {
            top = fmaxf(top, fmaxf(clean(__uint_as_float(w[e] << 16)), clean(__uint_as_float(w[e] & 0xFFFF0000u))));
          } else {
            const float z = clean(__uint_as_float(w[e]));
            top = fmaxf(top, z);
            w[e] = __float_as_uint(z);
          }
        }
        *reinterpret_cast<uint4*>(store + (size_t)i * kSize) = make_uint4(w[0], w[1], w[2], w[3]);
      }
    } else {
#pragma unroll 8
      for (int i = first + lane; i < local_end; i += 32) {
        const int at = index0 + i;
        if (BF16) {
          const uint16_t x = at < a.V ? reinterpret_cast<const uint16_t*>(row)[at] : 0xFF80u;
          top = fmaxf(top, clean(bf16_bits_to_float(x)));
          reinterpret_cast<uint16_t*>(store)[i] = x;
        } else {
          const float z = at < a.V ? clean(reinterpret_cast<const float*>(row)[at]) : -INFINITY;
          top = fmaxf(top, z);
          reinterpret_cast<float*>(store)[i] = z;
        }
      }
    }
  }
  Slice<BF16> z_of;
  z_of.at = reinterpret_cast<decltype(z_of.at)>(store);
  for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
  if (lane == 0) s.warp_max[warp] = top;
  clear_histogram(s);

  cluster_sync();  // every CTA of the cluster runs before its shared memory is written
  if (warp == 0) {
    top = lane < kWarps ? s.warp_max[lane] : -INFINITY;
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
    if (lane < C) st_dsmem_f32(map_to_rank(smem_addr(&s.rank_max[rank]), lane), top);
  }
  cluster_sync();
  top = lane < C ? s.rank_max[lane] : -INFINITY;
  for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
  if (top == -INFINITY) {  // no finite logit; the whole cluster agrees
    if (rank == 0 && tid == 0) {
      a.ids[m] = -1;
      if (a.logprob) a.logprob[m] = -INFINITY;
      if (a.kept) a.kept[m] = 0;
    }
    return;
  }

  // Kept mass of this warp's segment when tokens with key < cut stay, and those equal to it are
  // counted apart; floor_min drops smaller weights.
  u64 seg_mass, seg_tie;
  uint32_t seg_count, seg_ties;
  auto segment = [&](uint32_t cut, float floor_min) {
    uint32_t hi = 0, count = 0, ties = 0;
    int lo = 0;
    u64 tie = 0;
#pragma unroll 1
    for (int i = local; i < local_end; i += 128) {
      float z[4];
      z_of.get4(i, z);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t key = down_key(z[e]);
        const float w = weight_of(z[e], top, rate);
        uint32_t h, l;
        split_mass(w, h, l);
        if (key > cut || w < floor_min) h = l = 0;
        if (key == cut) {
          ++ties;
          tie = (u64)(((long long)(int)h << 20) + (int)l);
        } else {
          hi += h, lo += (int)l, count += (h | l) != 0;  // at most 2^9 tokens per lane: 32 bits hold the sums
        }
      }
    }
    seg_mass = warp_sum((u64)(((long long)hi << 20) + lo));
    for (int o = 16; o; o >>= 1) {
      count += __shfl_xor_sync(~0u, count, o);
      ties += __shfl_xor_sync(~0u, ties, o);
      const u64 x = __shfl_xor_sync(~0u, tie, o);
      tie = x > tie ? x : tie;
    }
    seg_count = count, seg_ties = ties, seg_tie = tie;
  };

  uint32_t cut = 0xFFFFFFFFu, r_keep = 0xFFFFFFFFu;  // tokens past the row have this key, and no mass
  const bool by_count = k < (uint32_t)a.V;
  if (by_count || !(p >= 1.0f)) {
    // ---- the whole mass, where top-p alone cuts
    u64 whole = 0, limit = 0;
    float low = -INFINITY;  // logits below it are not looked at
    if (!by_count) {
      segment(0xFFFFFFFEu, 0.0f);
      if (lane == 0) s.warp_mass[warp] = seg_mass;
      __syncthreads();
      if (warp == 0) {
        const u64 sum = warp_sum(lane < kWarps ? s.warp_mass[lane] : 0);
        if (lane < C) st_dsmem_u64(map_to_rank(smem_addr(&s.rank_total[rank]), lane), sum);
      }
      cluster_sync();
      for (int r = 0; r < C; ++r) whole += s.rank_total[r];
      limit = top_p_limit(p, whole);
      // weights up to (1 - p) S / V: half of it, for the roundings on the way
      const float tau = 0.5f * (1.0f - p) * ((float)whole * 0x1p-40f) / (float)a.V;
      low = top + logf(fmaxf(tau, 1e-30f)) / rate;
      if (!(low < top)) low = -INFINITY;
    }

    // ---- the step in which the prefix ends
#pragma unroll 1
    for (int i = local; i < local_end; i += 128) {
      float z[4];
      z_of.get4(i, z);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (!(z[e] >= low)) continue;
        const int bin = step_of(z[e], top, steps);
        if (bin >= kBins - 1) continue;  // no mass past the last step: a cut there cuts nothing
        atomicAdd(&s.count[bin], 1u);
        if (!by_count) add_mass(s, bin, mass_of(weight_of(z[e], top, rate)));
      }
    }
    merge_histograms(s, C, rank, !by_count);
    find_bin(s, !by_count, k, limit, true);
    int bin = s.bin;
    uint32_t count_before = s.count_before;
    u64 mass_before = s.mass_before;
    const uint32_t n = count_before + s.found;
    if (n <= kCap) {
      // ---- the candidates go to the first CTA
      const int last = bin < kBins ? bin : kBins - 2;
      for (int i = tid; i < kBins; i += kThreads) s.hi[i] = 0;  // the first CTA's: taken places of a step
      cluster_sync();
      const uint32_t taken = map_to_rank(smem_addr(s.hi), 0), cand = map_to_rank(smem_addr(s.cand), 0);
#pragma unroll 1
      for (int i = local; i < local_end; i += 128) {
        float z[4];
        z_of.get4(i, z);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (!(z[e] >= low)) continue;
          const int b = step_of(z[e], top, steps);
          if (b > last) continue;
          uint32_t place;
          asm volatile("atom.shared::cluster.add.u32 %0, [%1], 1;" : "=r"(place) : "r"(taken + 4 * b) : "memory");
          place += s.all_count[b];
          if (place < kCap) st_dsmem_u64(cand + 8 * place, ((u64)down_key(z[e]) << 32) | (uint32_t)(index0 + i + e));
        }
      }
      cluster_sync();  // the last exchange: no CTA touches another's memory after it
      if (rank == 0)
        finish_candidates(a, s, reinterpret_cast<ulonglong2*>(store), m, n, last, k, p, whole, floor_w, top, rate, steps, u);
      return;
    }

    // ---- too many: narrow the cut down by digits of the key
    u64 total = whole;
#pragma unroll 1
    for (int turn = by_count ? 0 : 1; turn < 2; ++turn) {
      if (turn == 1) {
        if (p >= 1.0f) break;
        if (by_count) {  // masses of the steps, which top-k did not need
          limit = top_p_limit(p, total);
          clear_histogram(s);
          __syncthreads();
#pragma unroll 1
          for (int i = local; i < local_end; i += 128) {
            float z[4];
            z_of.get4(i, z);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int b = step_of(z[e], top, steps);
              if (b < kBins - 1) atomicAdd(&s.count[b], 1u), add_mass(s, b, mass_of(weight_of(z[e], top, rate)));
            }
          }
          merge_histograms(s, C, rank, true);
          find_bin(s, true, 0, limit, false);
          bin = s.bin, count_before = s.count_before, mass_before = s.mass_before;
        }
      }
      if (bin == kBins) {  // fewer than k tokens have mass: top-k cuts nothing
        __syncthreads();
        if (turn == 0 && !(p >= 1.0f)) {
          segment(0xFFFFFFFEu, 0.0f);
          if (lane == 0) s.warp_mass[warp] = seg_mass;
          __syncthreads();
          if (warp == 0) {
            const u64 sum = warp_sum(lane < kWarps ? s.warp_mass[lane] : 0);
            if (lane < C) st_dsmem_u64(map_to_rank(smem_addr(&s.rank_total[rank]), lane), sum);
          }
          cluster_sync();
          total = 0;
          for (int r = 0; r < C; ++r) total += s.rank_total[r];
        }
        continue;
      }
      // among the tokens of the step: digits of 10, 10, 10 and 2 bits
      uint32_t prefix = 0;
      u64 one = 0;  // mass of one token at the cut
#pragma unroll 1
      for (int level = 0; level < 4; ++level) {
        const int shift = level < 3 ? 22 - 10 * level : 0, bits = level < 3 ? 10 : 2;
        __syncthreads();
        clear_histogram(s);
        __syncthreads();
#pragma unroll 1
        for (int i = local; i < local_end; i += 128) {
          float z[4];
          z_of.get4(i, z);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if (step_of(z[e], top, steps) != bin) continue;
            const uint32_t key = down_key(z[e]);
            if (level && (key >> (shift + bits)) != prefix) continue;
            const int d = (int)((key >> shift) & ((1u << bits) - 1));
            atomicAdd(&s.count[d], 1u);
            add_mass(s, d, mass_of(weight_of(z[e], top, rate)));
          }
        }
        merge_histograms(s, C, rank, true);
        find_bin(s, turn == 1, k > count_before ? k - count_before : 0, limit - mass_before, false);
        const int d = s.bin;
        count_before += s.count_before;
        if (turn == 1) mass_before += s.mass_before;
        if (level == 3) one = s.all_mass[d] / s.all_count[d];  // equal keys, equal masses
        prefix = (prefix << bits) | (uint32_t)d;
      }
      cut = prefix;
      if (turn == 0) {
        r_keep = k - count_before;
        // S of what top-k leaves
        segment(cut, 0.0f);
        if (lane == 0) s.warp_mass[warp] = seg_mass;
        __syncthreads();
        if (warp == 0) {
          const u64 sum = warp_sum(lane < kWarps ? s.warp_mass[lane] : 0);
          if (lane < C) st_dsmem_u64(map_to_rank(smem_addr(&s.rank_total[rank]), lane), sum);
        }
        cluster_sync();
        total = 0;
        for (int r = 0; r < C; ++r) total += s.rank_total[r];
        total += (u64)r_keep * one;
      } else {
        r_keep = (uint32_t)((limit - mass_before + one - 1) / one);
      }
    }
  }

  // ---- kept mass of every segment
  segment(cut, floor_w);
  if (lane == 0) {
    s.warp_mass[warp] = seg_mass;
    s.warp_count[warp] = seg_count;
    s.warp_ties[warp] = seg_ties;
    s.warp_tie[warp] = seg_tie;
  }
  __syncthreads();
  if (warp == 0) {
    const bool in = lane < kWarps;
    const u64 ms = warp_sum(in ? s.warp_mass[lane] : 0);
    u64 tm = in ? s.warp_tie[lane] : 0;
    uint32_t cs = in ? s.warp_count[lane] : 0, ts = in ? s.warp_ties[lane] : 0;
    for (int o = 16; o; o >>= 1) {
      cs += __shfl_xor_sync(~0u, cs, o);
      ts += __shfl_xor_sync(~0u, ts, o);
      const u64 x = __shfl_xor_sync(~0u, tm, o);
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
  u64 total = 0, before = 0, one = 0;
  uint32_t kept = 0, ties_before = 0, seen = 0;
  for (int r = 0; r < C; ++r) one = s.rank_tie[r] > one ? s.rank_tie[r] : one;
  auto staying = [&](uint32_t ties, uint32_t passed) {  // of `ties` tokens at the cut after `passed` others
    const uint32_t left = r_keep > passed ? r_keep - passed : 0;
    return ties < left ? ties : left;
  };
  for (int r = 0; r < C; ++r) {
    if (r == rank) before = total, ties_before = seen;
    const uint32_t stay = staying(s.rank_ties[r], seen);
    total += s.rank_mass[r] + stay * one;
    kept += s.rank_count[r] + (one ? stay : 0);
    seen += s.rank_ties[r];
  }
  const u64 aim = aim_of(u, total);

  // ---- the segment that holds the aim, then the token
  for (int w = 0; w < warp; ++w) {
    before += s.warp_mass[w] + staying(s.warp_ties[w], ties_before) * one;
    ties_before += s.warp_ties[w];
  }
  if (aim < before || aim >= before + s.warp_mass[warp] + staying(s.warp_ties[warp], ties_before) * one) return;
#pragma unroll 1
  for (int i = local; i < local_end; i += 128) {
    float z[4];
    z_of.get4(i, z);
    u64 q[4], sum = 0;
    uint32_t at_cut = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) at_cut += down_key(z[e]) == cut;
    const uint32_t ties_incl = warp_incl32(at_cut, lane);
    uint32_t passed = ties_before + ties_incl - at_cut;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t key = down_key(z[e]);
      const float w = weight_of(z[e], top, rate);
      q[e] = key <= cut && !(w < floor_w) ? mass_of(w) : 0;
      if (key == cut && passed++ >= r_keep) q[e] = 0;
      sum += q[e];
    }
    const u64 incl = warp_incl(sum, lane);
    u64 b = before + incl - sum;
    const uint32_t hit = __ballot_sync(~0u, before + incl > aim);
    if (hit) {
      if (lane == __ffs(hit) - 1) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (aim >= b && aim < b + q[e]) finish(a, m, index0 + i + e, q[e], total, kept);
          b += q[e];
        }
      }
      return;
    }
    before += __shfl_sync(~0u, incl, 31);
    ties_before += __shfl_sync(~0u, ties_incl, 31);
  }
}

template <bool BF16>
cudaError_t launch(SampleArgs a, cudaStream_t s) {
  // Slices of up to 32,768 elements (128 KB in fp32), and of about 8,192 and more while the row
  // is large enough: the phases between the exchanges then take about as long as the exchanges.
  int C = 1;
  while (C < kMaxCluster && (long long)C * 16384 < a.V) C *= 2;
  a.cluster = C;
  a.per_warp = ((a.V + C * kWarps - 1) / (C * kWarps) + 127) / 128 * 128;
  a.aligned = ((uintptr_t)a.logits & 15) == 0 && (a.row_stride * (BF16 ? 2 : 4)) % 16 == 0;
  const size_t bytes = (sizeof(Shared) + 15) / 16 * 16 +
                       std::max((size_t)kWarps * a.per_warp * (BF16 ? 2 : 4), (size_t)kCap * 16);
  static std::atomic<int> ready[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!ready[dev].load(std::memory_order_relaxed)) {
    e = cudaFuncSetAttribute(sample_kernel<BF16>, cudaFuncAttributeMaxDynamicSharedMemorySize, 220 * 1024);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(sample_kernel<BF16>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    ready[dev].store(1, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.M * a.cluster));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = bytes;
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
  const SampleArgs a = {logits, row_stride, M, V, 1, 0, 0, temperature, top_k, top_p, min_p, u, id_map, ids, logprob, kept};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = dtype == LOWBIT_LOGITS_BF16 ? launch<true>(a, s) : launch<false>(a, s);
  return e == cudaSuccess ? LOWBIT_OK : LOWBIT_ERR_CUDA;
}
