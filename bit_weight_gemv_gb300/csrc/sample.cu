// One token per row of logits under temperature, top-k, top-p and min-p, from a given uniform
// number (see include/lowbit.h for the definition).
//
// A weight w = exp((z - max) / T) becomes a whole number, w * 2^40 rounded, so every sum below is
// a 64-bit integer: exact, the same in any order, and free to be taken with atomics.
//
// A cluster of CTAs takes one row, each a contiguous slice, held in its shared memory where two such
// CTAs share an SM (the row is then read once), else read again from L2, which holds the rows in
// flight.  Truncation keeps a prefix of the order (larger logit, then lower index):
//   1. the largest logit, over the cluster;
//   2. a bound from the lanes' own maxima, of which k (or 512, for top-p alone) lie above it: a count of
//      them in 1024 equal steps of (max - z) / T (28.5 covers every weight that does not round to
//      zero).  The tokens down to that step, little more than k, go to the first CTA; for top-p the same
//      pass takes the whole mass S.  Where they hold all that stays, the first CTA sorts them and
//      finishes the row;
//   3. else a histogram over 1024 steps, of counts for top-k and of masses for top-p, merged over the
//      cluster: the step in which the prefix ends, and for top-k how many tokens (n) lie up to it.  For
//      top-p alone the steps are laid below the list of 2, down to the weight (1 - p) S / V: what lies
//      below sums to (1 - p) S at most, so the prefix ends above it;
//   4. top-k with n <= 2048: those tokens go to the first CTA as in 2; else only the tokens of that step
//      do, which gives the threshold key and the number of tokens equal to it that stay, and the draw
//      walks the segments that the warps own.  (A step with more than 2048 tokens, such as a row of
//      equal logits, is narrowed down by its keys' digits.)
//
// Few rows wait on latency: one row of 248,320 takes 14.9 us with top-k 20 and top-p 0.95, of which the
// merges and exchanges over 16 CTAs take 9, and 9.7 us without truncation.  Many rows are bound by
// instructions, about 30 for each weight that is summed: 192 rows of mixed settings take 145 us, 28
// of them for reading the logits once at the copy rate.
#include <algorithm>
#include <atomic>
#include <type_traits>

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
  int per_warp;   // elements of a warp's segment, a multiple of 128, or of 512 read from L2
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
  return fminf(fmaxf(z, -INFINITY), 3.402823466e38f);  // NaN to -inf
}
// Ascending with descending z, and back.
__device__ __forceinline__ uint32_t down_key(float z) {
  const uint32_t b = __float_as_uint(z + 0.0f);  // -0 to +0
  return (b & 0x80000000u) ? b : ~(b | 0x80000000u);
}
__device__ __forceinline__ float key_logit(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? k : ~k & 0x7FFFFFFFu);
}
__device__ __forceinline__ float weight_of(float z, float top, float rate) {
  return expf((z - top) * rate);  // top is finite: -inf gives 0
}
// w * 2^40 rounded, as hi * 2^20 + lo (signed): both parts are taken by adding 1.5 * 2^23, which leaves
// the rounded integer in the low bits; the remainder between them is exact.  Both words come with the
// bits of 1.5 * 2^23 on them, which a sum takes off once at its end.
constexpr float kMagic = 12582912.0f;
constexpr uint32_t kMagicBits = 0x4B400000u;
__device__ __forceinline__ void split_mass(float w, uint32_t& hi, uint32_t& lo) {
  const float f = w * 1048576.0f, t = f + kMagic;
  hi = __float_as_uint(t);
  lo = __float_as_uint(fmaf(f - (t - kMagic), 1048576.0f, kMagic));
}
__device__ __forceinline__ u64 join_mass(uint32_t hi, uint32_t lo, uint32_t parts) {
  return (u64)(((long long)(hi - parts * kMagicBits) << 20) + (int)(lo - parts * kMagicBits));
}
__device__ __forceinline__ u64 mass_of(float w) {
  uint32_t hi, lo;
  split_mass(w, hi, lo);
  return join_mass(hi, lo, 1);
}
constexpr float kLeast = 0x1p-41f;  // weights up to it have no mass
__device__ __forceinline__ int step_of(float z, float origin, float steps) {
  return z == -INFINITY ? kBins - 1 : (int)fminf(fmaxf((origin - z) * steps, 0.0f), (float)(kBins - 1));
}

struct Shared {
  uint32_t count[kBins], lo[kBins], hi[kBins];  // this CTA's histogram; the mass in two words
  uint32_t all_count[kBins];                    // the cluster's
  u64 all_mass[kBins];
  u64 cand[kCap];                               // key << 32 | index: this CTA's, then in the first one all
  u64 warp_mass[kWarps], warp_tie[kWarps];
  uint32_t warp_count[kWarps], warp_ties[kWarps];
  float warp_max[kWarps], rank_max[kMaxCluster];
  u64 rank_mass[kMaxCluster], rank_tie[kMaxCluster], rank_total[kMaxCluster];
  uint32_t rank_count[kMaxCluster], rank_ties[kMaxCluster], rank_cand[kMaxCluster];
  // the bin that a search found, and what precedes it
  int bin, found;
  uint32_t count_before, cut, stay;
  u64 mass_before, one;
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
// it; s.bin = kBins if there is none, with the whole count and mass.  All threads; the results are
// ready after it.
__device__ __noinline__ void find_bin(Shared& s, bool by_mass, uint32_t k, u64 limit) {
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

// Four neighbouring logits of a slice, by their place in it: from shared memory (places past the
// row hold -inf), or from the row itself.
template <bool BF16, bool HELD>
struct Slice {
  const uint8_t* at;   // HELD: the slice in shared memory; else the slice in the row
  int end;             // places of the slice inside the row
  int aligned;
  __device__ __forceinline__ void vector4(int i, float (&z)[4]) const {
    if (BF16) {
      const uint2 v = HELD ? *reinterpret_cast<const uint2*>(at + 2 * i) : __ldg(reinterpret_cast<const uint2*>(at + 2 * i));
      z[0] = __uint_as_float(v.x << 16), z[1] = __uint_as_float(v.x & 0xFFFF0000u);
      z[2] = __uint_as_float(v.y << 16), z[3] = __uint_as_float(v.y & 0xFFFF0000u);
    } else {
      const float4 v = HELD ? *reinterpret_cast<const float4*>(at + 4 * i) : __ldg(reinterpret_cast<const float4*>(at + 4 * i));
      z[0] = v.x, z[1] = v.y, z[2] = v.z, z[3] = v.w;
    }
  }
  __device__ __forceinline__ void load4(int i, float (&z)[4]) const {
    if (HELD || (aligned && i + 4 <= end)) {
      vector4(i, z);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        z[e] = -INFINITY;
        if (i + e < end)
          z[e] = BF16 ? bf16_bits_to_float(__ldg(reinterpret_cast<const uint16_t*>(at) + i + e))
                      : __ldg(reinterpret_cast<const float*>(at) + i + e);
      }
    }
  }
  __device__ __forceinline__ void clean4(float (&z)[4]) const {
    if constexpr (BF16 || !HELD) {  // else clean already
#pragma unroll
      for (int e = 0; e < 4; ++e) z[e] = clean(z[e]);
    }
  }
  // f(place, logits) for every fourth place of from..to (a multiple of 128 apart) and the lane's, until
  // it returns true.  Out of L2 four loads of a lane are under way at a time (top-k 20, 128 fp32 rows
  // of 248,320: 63 us, 72 with two, 79 with one); the loop over shared memory stays short, since few
  // rows spend their time on instructions read for the first time.
  template <class F>
  __device__ __forceinline__ void each4(int from, int to, F&& f) const {
    const int lane4 = (threadIdx.x & 31) * 4;
    if constexpr (!HELD) {
      const int whole = aligned ? min(to, end) : 0;
#pragma unroll 1
      for (; from + 512 <= whole; from += 512) {
        float z[4][4];
#pragma unroll
        for (int j = 0; j < 4; ++j) vector4(from + lane4 + 128 * j, z[j]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          clean4(z[j]);
          if (f(from + lane4 + 128 * j, z[j])) return;
        }
      }
    }
#pragma unroll 1
    for (; from < to; from += 128) {
      float z[4];
      load4(from + lane4, z);
      clean4(z);
      if (f(from + lane4, z)) return;
    }
  }
};

// One exchange of a bitonic sort between lanes `half` apart: the value that stays here.
__device__ __forceinline__ u64 keep_of_pair(u64 x, int half, bool lower) {
  const u64 y = __shfl_xor_sync(~0u, x, half);
  return (x < y) == lower ? x : y;
}
// Sorts the first n of s.cand (larger logit, then lower index, first), by all threads: bitonic, runs
// that ascend where bit `run` of a place is clear.  A warp does the exchanges within 64 places in
// registers, two places a lane, and wider ones go through shared memory (about 2,048 candidates with
// the search of the cut in them: 13.7 us, 19.7 with every exchange in shared memory).
__device__ __noinline__ void sort_candidates(Shared& s, uint32_t n) {
  const uint32_t lane = threadIdx.x & 31;
  uint32_t size = 64;
  while (size < n) size *= 2;
  for (uint32_t i = n + threadIdx.x; i < size; i += kThreads) s.cand[i] = ~0ull;
  __syncthreads();
#pragma unroll 1
  for (uint32_t run = 64; run <= size; run *= 2) {
#pragma unroll 1
    for (uint32_t half = run / 2; half > 32; half /= 2) {
      for (uint32_t t = threadIdx.x; t < size / 2; t += kThreads) {
        const uint32_t i = 2 * t - (t & (half - 1));
        const u64 x = s.cand[i], y = s.cand[i + half];
        if ((x > y) == ((i & run) == 0)) s.cand[i] = y, s.cand[i + half] = x;
      }
      __syncthreads();
    }
#pragma unroll 1
    for (uint32_t base = (threadIdx.x & ~31u) * 2; base < size; base += 2 * kThreads) {
      u64 x = s.cand[base + lane], y = s.cand[base + lane + 32];
#pragma unroll 1
      for (uint32_t r = run == 64 ? 2 : run; r <= run; r *= 2) {
        if (r >= 64) {
          const bool up = (base & r) == 0;
          if ((x > y) == up) {
            const u64 t = x;
            x = y, y = t;
          }
        }
#pragma unroll 1
        for (uint32_t half = r < 64 ? r / 2 : 16; half; half /= 2) {
          const bool low = (lane & half) == 0;
          x = keep_of_pair(x, half, low == (((base + lane) & r) == 0));
          y = keep_of_pair(y, half, low == (((base + lane + 32) & r) == 0));
        }
      }
      s.cand[base + lane] = x, s.cand[base + lane + 32] = y;
    }
    __syncthreads();
  }
}

// The first CTA's end of a row: n sorted candidates, of which top-k, top-p and min-p keep a part;
// then the draw in index order.
__device__ __forceinline__ void finish_candidates(const SampleArgs& a, Shared& s, ulonglong2* list, int m, uint32_t n,
                                                  uint32_t k, float p, u64 whole, float floor_w, float top, float rate,
                                                  float u) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  for (int i = tid; i < kBins; i += kThreads) s.lo[i] = s.hi[i] = 0;
  // masses before each place; a thread takes four places in a row
  constexpr int kOwn = kCap / kThreads;
  u64 c[kOwn], q[kOwn], sum = 0;
#pragma unroll
  for (int e = 0; e < kOwn; ++e) {
    const uint32_t i = tid * kOwn + e;
    c[e] = i < n ? s.cand[i] : 0;
    q[e] = i < n && i < k ? mass_of(weight_of(key_logit((uint32_t)(c[e] >> 32)), top, rate)) : 0;
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
      list[atomicAdd(&s.found, 1)] = make_ulonglong2(c[e] & 0xFFFFFFFFu, q[e]);
  __syncthreads();
  const int found = s.found;
  for (int i = tid; i < found; i += kThreads) {
    const ulonglong2 v = list[i];
    u64 b = base;
    for (int j = 0; j < found; ++j) b += list[j].x < v.x ? list[j].y : 0;
    if (aim >= b && aim < b + v.y) finish(a, m, (int)v.x, v.y, total, kept);
  }
}

template <bool BF16, bool HELD>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const __grid_constant__ SampleArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  Shared& s = *reinterpret_cast<Shared*>(smem);
  uint8_t* const store = smem + (sizeof(Shared) + 15) / 16 * 16;
  constexpr int kSize = BF16 ? 2 : 4;
  const int C = a.cluster, rank = blockIdx.x % C, m = blockIdx.x / C;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int seg_from = warp * a.per_warp, seg_to = seg_from + a.per_warp;  // this warp's places in the slice
  const int index0 = rank * kWarps * a.per_warp;               // of the slice's first element
  cluster_arrive();  // this CTA runs: the others may write its shared memory
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
  float steps = rate * ((float)kBins / kReach);

  // ---- the slice comes in, and its largest logit; places past the row hold -inf
  float top = -INFINITY;
  const uint8_t* const row = static_cast<const uint8_t*>(a.logits) + (long long)m * a.row_stride * kSize;
  const Slice<BF16, HELD> z_of = {HELD ? store : row + (long long)index0 * kSize, max(0, a.V - index0), a.aligned};
  if (!HELD) {
    z_of.each4(seg_from, seg_to, [&](int, float (&z)[4]) {
      top = fmaxf(fmaxf(fmaxf(top, z[0]), z[1]), fmaxf(z[2], z[3]));
      return false;
    });
  } else {
    constexpr int kVec = 16 / kSize;                           // elements of a 16-byte load
    if (a.aligned) {
#pragma unroll 4
      for (int i = seg_from + lane * kVec; i < seg_to; i += 32 * kVec) {
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
      for (int i = seg_from + lane; i < seg_to; i += 32) {
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
  const float lane_max = top;
  for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
  if (lane == 0) s.warp_max[warp] = top;
  clear_histogram(s);

  __syncthreads();
  if (warp == 0) {
    top = lane < kWarps ? s.warp_max[lane] : -INFINITY;
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
  }
  cluster_wait();
  if (warp == 0 && lane < C) st_dsmem_f32(map_to_rank(smem_addr(&s.rank_max[rank]), lane), top);
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

  // Kept mass of the places from..to: without a cut, or of the tokens with key < cut, those equal to
  // it counted apart; floor_min drops smaller weights.
  u64 seg_mass, seg_tie;
  uint32_t seg_count, seg_ties;
  auto segment = [&](auto with_cut, int from, int to, uint32_t cut, float floor_min) {
    constexpr bool kCut = decltype(with_cut)::value == 1, kWhole = decltype(with_cut)::value == 2;
    uint32_t hi = 0, lo = 0, parts = 0, count = 0, ties = 0;
    u64 tie = 0;
    // below this exponent the mass is zero, or the weight under the floor (expf and logf are good to
    // 2 ulp, a part in 2^21)
    const float least = !kWhole && floor_min > 0.0f ? fmaxf(logf(floor_min) - 1e-3f, -kReach) : -kReach;
    z_of.each4(from, to, [&](int, float (&z)[4]) {
      if ((fmaxf(fmaxf(z[0], z[1]), fmaxf(z[2], z[3])) - top) * rate < least) return false;
      parts += 4;  // at most 2^8 tokens per lane: 32 bits hold the sums
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float w = weight_of(z[e], top, rate);
        if (!kWhole && w < floor_min) w = 0.0f;
        if (kCut) {
          const uint32_t key = down_key(z[e]);
          if (key == cut) ++ties, tie = mass_of(w);
          if (key >= cut) w = 0.0f;
        }
        uint32_t h, l;
        split_mass(w, h, l);
        hi += h, lo += l;
        if (!kWhole) count += w > kLeast;
      }
      return false;
    });
    seg_mass = warp_sum(join_mass(hi, lo, parts));
    seg_count = 0, seg_ties = 0, seg_tie = 0;
    if (!kWhole) seg_count = __reduce_add_sync(~0u, count);
    if (kCut) {
      seg_ties = __reduce_add_sync(~0u, ties);
      for (int o = 16; o; o >>= 1) {
        const u64 x = __shfl_xor_sync(~0u, tie, o);
        tie = x > tie ? x : tie;
      }
      seg_tie = tie;
    }
  };
  using Plain = std::integral_constant<int, 0>;
  using WithCut = std::integral_constant<int, 1>;
  using Whole = std::integral_constant<int, 2>;  // every token, and no count
  // The cluster's sum of seg_mass; once per row.
  auto cluster_mass = [&]() {
    if (lane == 0) s.warp_mass[warp] = seg_mass;
    __syncthreads();
    if (warp == 0) {
      const u64 sum = warp_sum(lane < kWarps ? s.warp_mass[lane] : 0);
      if (lane < C) st_dsmem_u64(map_to_rank(smem_addr(&s.rank_total[rank]), lane), sum);
    }
    cluster_sync();
    u64 sum = 0;
    for (int r = 0; r < C; ++r) sum += s.rank_total[r];
    return sum;
  };
  // Tokens of steps from..to (logits >= low) into the first CTA's list; their number.  With more
  // than kCap the list is not used.  With masses, also the cluster's whole mass and that of the list.
  u64 whole = 0, listed = 0;
  float origin = top;  // where the steps begin
  auto gather = [&](auto with_masses, int from, int to, float low) {
    constexpr bool kMasses = decltype(with_masses)::value;
    // a step's width below the last one's end, and above the first one's start
    low = fmaxf(low, origin - (float)(to + 2) / steps);
    const float high = from ? origin - (float)(from - 1) / steps : INFINITY;
    uint32_t hi = 0, lo = 0, parts = 0;
    __syncthreads();  // s.found has been read
    if (tid == 0) s.found = 0;
    __syncthreads();
    z_of.each4(seg_from, seg_to, [&](int i, float (&z)[4]) {
      const float most = fmaxf(fmaxf(z[0], z[1]), fmaxf(z[2], z[3]));
      if (kMasses && (most - top) * rate >= -kReach) {  // as in `segment`
        parts += 4;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint32_t h, l;
          split_mass(weight_of(z[e], top, rate), h, l);
          hi += h, lo += l;
        }
      }
      if (most >= low) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (!(z[e] >= low && z[e] <= high)) continue;
          const int b = step_of(z[e], origin, steps);
          if (b < from || b > to) continue;
          const uint32_t at = atomicAdd(&s.found, 1);
          if (at < kCap) s.cand[at] = ((u64)down_key(z[e]) << 32) | (uint32_t)(index0 + i + e);
        }
      }
      return false;
    });
    __syncthreads();
    const uint32_t mine = (uint32_t)s.found;
    if (kMasses) {
      u64 own = 0;
#pragma unroll 1
      for (uint32_t i = tid; i < min(mine, (uint32_t)kCap); i += kThreads)
        own += mass_of(weight_of(key_logit((uint32_t)(s.cand[i] >> 32)), top, rate));
      own = warp_sum(own);
      const u64 sum = warp_sum(join_mass(hi, lo, parts));
      if (lane == 0) s.warp_mass[warp] = sum, s.warp_tie[warp] = own;
      __syncthreads();
    }
    if (warp == 0) {
      const u64 sum = kMasses ? warp_sum(lane < kWarps ? s.warp_mass[lane] : 0) : 0;
      const u64 part = kMasses ? warp_sum(lane < kWarps ? s.warp_tie[lane] : 0) : 0;
      if (lane < C) {
        st_dsmem_u32(map_to_rank(smem_addr(&s.rank_cand[rank]), lane), mine);
        if (kMasses) {
          st_dsmem_u64(map_to_rank(smem_addr(&s.rank_total[rank]), lane), sum);
          st_dsmem_u64(map_to_rank(smem_addr(&s.rank_mass[rank]), lane), part);
        }
      }
    }
    cluster_sync();
    uint32_t at = 0, n = 0;
    for (int r = 0; r < C; ++r) {
      if (r == rank) at = n;
      n += s.rank_cand[r];
      if (kMasses) whole += s.rank_total[r], listed += s.rank_mass[r];
    }
    if (rank && n <= kCap) {
      const uint32_t cand = map_to_rank(smem_addr(s.cand), 0);
      for (uint32_t i = tid; i < mine; i += kThreads) st_dsmem_u64(cand + 8 * (at + i), s.cand[i]);
    }
    cluster_sync();
    return n;
  };

  // Four tokens' masses, those with logits >= low, into the histogram; the additions to the low words
  // are all under way before the first one's carry is looked at (128 rows with top-p 0.9 that keep 90,000
  // tokens each: 226 us, 236 one after another).
  auto add_masses = [&](const float (&z)[4], float low) {
    if (!(fmaxf(fmaxf(z[0], z[1]), fmaxf(z[2], z[3])) >= low)) return;
    int bin[4];
    uint32_t lo[4], up[4], old[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      bin[e] = step_of(z[e], origin, steps);
      const u64 mass = z[e] >= low && bin[e] < kBins - 1 ? mass_of(weight_of(z[e], top, rate)) : 0;
      lo[e] = (uint32_t)mass, up[e] = (uint32_t)(mass >> 32), old[e] = 0;
      if (lo[e]) old[e] = atomicAdd(&s.lo[bin[e]], lo[e]);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (lo[e] && old[e] > 0xFFFFFFFFu - lo[e]) ++up[e];
      if (up[e]) atomicAdd(&s.hi[bin[e]], up[e]);
    }
  };

  // In the first CTA: of its n candidates only those down to the step in which their mass reaches
  // `limit`, still unsorted; their number.
  auto trim = [&](uint32_t n, u64 limit) {
    constexpr int kOwn = kCap / kThreads;
    clear_histogram(s);
    __syncthreads();
    u64 c[kOwn];
    int step[kOwn];
#pragma unroll
    for (int e = 0; e < kOwn; ++e) {
      const uint32_t i = tid + e * kThreads;
      c[e] = i < n ? s.cand[i] : 0;
      step[e] = kBins;
      if (i < n) {
        const float x = key_logit((uint32_t)(c[e] >> 32));
        step[e] = step_of(x, origin, steps);
        add_mass(s, step[e], mass_of(weight_of(x, top, rate)));
      }
    }
    __syncthreads();
    for (int i = tid; i < kBins; i += kThreads) s.all_count[i] = 0, s.all_mass[i] = s.lo[i] + ((u64)s.hi[i] << 32);
    __syncthreads();
    find_bin(s, true, 0, limit);
    const int last = s.bin;
    if (tid == 0) s.found = 0;
    __syncthreads();
#pragma unroll
    for (int e = 0; e < kOwn; ++e)
      if (step[e] <= last && step[e] < kBins) s.cand[atomicAdd(&s.found, 1)] = c[e];
    __syncthreads();
    return (uint32_t)s.found;
  };

  uint32_t cut = 0xFFFFFFFFu, r_keep = 0xFFFFFFFFu;  // a key that no token has
  const bool by_count = k < (uint32_t)a.V;
  if (by_count || !(p >= 1.0f)) {
    // ---- the lanes' own maxima first: at least k tokens lie in the steps down to the k-th largest
    // of them, and with k up to half the lanes not many more.  Where they number kCap at most and
    // hold all that top-k or top-p leaves, they finish the row, and no histogram of it is taken (one
    // row of 248,320 with top-k 20: 14.9 us, 17.5 by the histogram; with top-p 0.8: 19.8 and 25.7).  For
    // top-p the bound is that of 512 lanes (16 rows with top-p 0.8: 29 us, 46 with 256 and 30 with 1,024;
    // 192 rows of mixed settings 145, 147 and 152).
    const uint32_t reach = min(C * kThreads / 2, kCap / 2);
    u64 limit = 0;
    bool have_whole = false, beyond = false;
    if (!by_count || k <= reach) {
      const int own = step_of(lane_max, origin, steps);
      if (own < kBins - 1) atomicAdd(&s.count[own], 1u);
      merge_histograms(s, C, rank, false);
      find_bin(s, false, by_count ? k : min(reach, 512u), 0);
      const int bin = min(s.bin, kBins - 2);
      uint32_t n = kCap + 1;
      bool all = true;
      if (by_count) {
        if (s.bin < kBins) n = gather(std::false_type(), 0, bin, -INFINITY);
      } else {
        n = gather(std::true_type(), 0, bin, -INFINITY);
        have_whole = true;
        limit = top_p_limit(p, whole);
        all = listed >= limit;
        beyond = n <= kCap && !all;
      }
      if (n <= kCap && all) {
        if (rank == 0) {
          if (!by_count && n > 64) n = trim(n, limit);
          sort_candidates(s, n);
          finish_candidates(a, s, reinterpret_cast<ulonglong2*>(store), m, n, k, p, whole, floor_w, top, rate, u);
        }
        return;
      }
      clear_histogram(s);
      __syncthreads();
    }
    float low = -INFINITY;  // logits below it are not looked at
    if (have_whole) {
      // Tokens of weights up to (1 - p) S / V sum to (1 - p) S at most.  Less a thousandth for expf and
      // logf, half a unit of 2^-40 for each mass's rounding, and a few ulps of the logits.
      const float tau = 0.999f * (1.0f - p) * ((float)whole * 0x1p-40f) / (float)a.V - 0x1p-41f;
      const float deep = logf(fmaxf(tau, 1e-30f)) / rate;
      low = top + deep - 4e-7f * (fabsf(top) + fabsf(deep));
      // the prefix ends between it and the list's last step: the steps are laid there, which leaves
      // a sixth of the tokens in the one that is searched (T = 1.5, p = 0.9)
      const float from = top - (float)min(s.bin, kBins - 2) / steps;
      if (beyond && low < from) {
        origin = from;
        steps = (float)(kBins - 4) / (from - low);
      } else if (!(low < top)) {
        low = -INFINITY;
      }
    }

    // ---- the step in which the prefix ends
    z_of.each4(seg_from, seg_to, [&](int, float (&z)[4]) {
      if (by_count) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int bin = step_of(z[e], origin, steps);
          if (bin < kBins - 1) atomicAdd(&s.count[bin], 1u);  // no mass past the last step: a cut there cuts nothing
        }
      } else {
        add_masses(z, low);
      }
      return false;
    });
    merge_histograms(s, C, rank, !by_count);
    find_bin(s, !by_count, k, limit);
    int bin = s.bin;
    uint32_t count_before = s.count_before;
    u64 mass_before = s.mass_before;
    const uint32_t n = count_before + s.found;
    if (by_count && n <= kCap) {
      gather(std::false_type(), 0, bin < kBins ? bin : kBins - 2, low);  // after it no CTA touches another's memory
      if (rank == 0) {
        sort_candidates(s, n);
        finish_candidates(a, s, reinterpret_cast<ulonglong2*>(store), m, n, k, p, whole, floor_w, top, rate, u);
      }
      return;
    }

    // ---- too many: the cut itself, for top-k and then for top-p
    u64 total = whole;
#pragma unroll 1
    for (int turn = by_count ? 0 : 1; turn < 2; ++turn) {
      if (turn == 1) {
        if (p >= 1.0f) break;
        if (by_count) {  // masses of the steps, which top-k did not need
          limit = top_p_limit(p, total);
          clear_histogram(s);
          __syncthreads();
          z_of.each4(seg_from, seg_to, [&](int, float (&z)[4]) {
            add_masses(z, -INFINITY);
            return false;
          });
          merge_histograms(s, C, rank, true);
          find_bin(s, true, 0, limit);
          bin = s.bin, count_before = s.count_before, mass_before = s.mass_before;
        }
      }
      if (bin == kBins) {  // fewer than k tokens have mass: top-k cuts nothing
        __syncthreads();
        if (turn == 0 && !(p >= 1.0f)) {
          segment(Whole(), seg_from, seg_to, 0, 0.0f);
          total = cluster_mass();
        }
        continue;
      }
      u64 one = 0;  // mass of one token at the cut
      const uint32_t here = gather(std::false_type(), bin, bin, turn == 1 ? low : -INFINITY);
      if (here <= kCap) {
        if (rank == 0) {
          sort_candidates(s, here);
          // a thread takes four places in a row; masses count only for top-p
          constexpr int kOwn = kCap / kThreads;
          u64 q[kOwn], sum = 0;
#pragma unroll
          for (int e = 0; e < kOwn; ++e) {
            const uint32_t i = tid * kOwn + e;
            q[e] = i < here ? mass_of(weight_of(key_logit((uint32_t)(s.cand[i] >> 32)), top, rate)) : 0;
            sum += q[e];
          }
          const u64 incl = warp_incl(sum, lane);
          if (lane == 31) s.warp_mass[warp] = incl;
          __syncthreads();
          u64 before = mass_before + incl - sum;
          for (int w = 0; w < warp; ++w) before += s.warp_mass[w];
#pragma unroll
          for (int e = 0; e < kOwn; ++e) {
            const uint32_t i = tid * kOwn + e;
            // the last token that stays
            const bool ends = turn == 1 ? before < limit && before + q[e] >= limit : i + 1 == k - count_before;
            if (i < here && ends) {
              const uint32_t key = (uint32_t)(s.cand[i] >> 32);
              uint32_t lo = 0, hi = i;  // the first of its equals
              while (lo < hi) {
                const uint32_t mid = (lo + hi) / 2;
                if ((uint32_t)(s.cand[mid] >> 32) < key) lo = mid + 1;
                else hi = mid;
              }
              s.cut = key, s.stay = i - lo + 1, s.one = q[e];
            }
            before += q[e];
          }
          __syncthreads();
          if (tid < C) {
            st_dsmem_u32(map_to_rank(smem_addr(&s.cut), tid), s.cut);
            st_dsmem_u32(map_to_rank(smem_addr(&s.stay), tid), s.stay);
            st_dsmem_u64(map_to_rank(smem_addr(&s.one), tid), s.one);
          }
        }
        cluster_sync();
        cut = s.cut, r_keep = s.stay, one = s.one;
      } else {
        // digits of 10, 10, 10 and 2 bits
        uint32_t prefix = 0;
#pragma unroll 1
        for (int level = 0; level < 4; ++level) {
          const int shift = level < 3 ? 22 - 10 * level : 0, bits = level < 3 ? 10 : 2;
          __syncthreads();
          clear_histogram(s);
          __syncthreads();
          z_of.each4(seg_from, seg_to, [&](int, float (&z)[4]) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if (step_of(z[e], origin, steps) != bin) continue;
              const uint32_t key = down_key(z[e]);
              if (level && (key >> (shift + bits)) != prefix) continue;
              const int d = (int)((key >> shift) & ((1u << bits) - 1));
              atomicAdd(&s.count[d], 1u);
              add_mass(s, d, mass_of(weight_of(z[e], top, rate)));
            }
            return false;
          });
          merge_histograms(s, C, rank, true);
          find_bin(s, turn == 1, k > count_before ? k - count_before : 0, limit - mass_before);
          const int d = s.bin;
          count_before += s.count_before;
          if (turn == 1) mass_before += s.mass_before;
          if (level == 3) one = s.all_mass[d] / s.all_count[d];  // equal keys, equal masses
          prefix = (prefix << bits) | (uint32_t)d;
        }
        cut = prefix;
        r_keep = turn == 0 ? k - count_before : (uint32_t)((limit - mass_before + one - 1) / one);
      }
      if (turn == 0 && !(p >= 1.0f)) {  // S of what top-k leaves
        segment(WithCut(), seg_from, seg_to, cut, 0.0f);
        total = cluster_mass() + (u64)r_keep * one;
      }
    }
  }

  // ---- kept mass of every warp's segment, over the cluster; then, in the CTA whose slice holds the
  // aim, of the sixteenths of the segment that holds it; then the walk to the token
  u64 total = 0, before = 0, one = 0, aim = 0;
  uint32_t kept = 0, ties_before = 0;
  int from = seg_from, to = seg_to;
  auto staying = [&](uint32_t ties, uint32_t passed) {  // of `ties` tokens at the cut after `passed` others
    const uint32_t left = r_keep > passed ? r_keep - passed : 0;
    return ties < left ? ties : left;
  };
#pragma unroll 1
  for (int level = 0; level < 2; ++level) {
    if (cut == 0xFFFFFFFFu) segment(Plain(), from, to, 0, floor_w);
    else segment(WithCut(), from, to, cut, floor_w);
    __syncthreads();
    if (lane == 0) {
      s.warp_mass[warp] = seg_mass;
      s.warp_count[warp] = seg_count;
      s.warp_ties[warp] = seg_ties;
      s.warp_tie[warp] = seg_tie;
    }
    __syncthreads();
    if (level == 0) {
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
      uint32_t seen = 0;
      for (int r = 0; r < C; ++r) one = s.rank_tie[r] > one ? s.rank_tie[r] : one;
      for (int r = 0; r < C; ++r) {
        if (r == rank) before = total, ties_before = seen;
        const uint32_t stay = staying(s.rank_ties[r], seen);
        total += s.rank_mass[r] + stay * one;
        kept += s.rank_count[r] + (one ? stay : 0);
        seen += s.rank_ties[r];
      }
      aim = aim_of(u, total);
      if (aim < before) return;
    }
    int owner = 0;
    for (; owner < kWarps; ++owner) {
      const u64 share = s.warp_mass[owner] + staying(s.warp_ties[owner], ties_before) * one;
      if (aim < before + share) break;
      before += share;
      ties_before += s.warp_ties[owner];
    }
    if (owner == kWarps || (level == 1 && owner != warp)) return;
    if (level == 0) {
      const int each = ((a.per_warp / 128 + kWarps - 1) / kWarps) * 128;
      to = (owner + 1) * a.per_warp;
      from = min(owner * a.per_warp + warp * each, to);
      to = min(from + each, to);
    }
  }
  z_of.each4(from, to, [&](int i, float (&z)[4]) {
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
      return true;
    }
    before += __shfl_sync(~0u, incl, 31);
    ties_before += __shfl_sync(~0u, ties_incl, 31);
    return false;
  });
}

template <bool BF16, bool HELD>
cudaError_t launch(SampleArgs a, int C, cudaStream_t s) {
  a.cluster = C;
  const int step = HELD ? 128 : 512;
  a.per_warp = ((a.V + C * kWarps - 1) / (C * kWarps) + step - 1) / step * step;
  a.aligned = ((uintptr_t)a.logits & 15) == 0 && (a.row_stride * (BF16 ? 2 : 4)) % 16 == 0;
  const size_t slice = HELD ? (size_t)kWarps * a.per_warp * (BF16 ? 2 : 4) : 0;
  const size_t bytes = (sizeof(Shared) + 15) / 16 * 16 + std::max(slice, (size_t)kCap * 16);
  static std::atomic<int> ready[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!ready[dev].load(std::memory_order_relaxed)) {
    e = cudaFuncSetAttribute(sample_kernel<BF16, HELD>, cudaFuncAttributeMaxDynamicSharedMemorySize, 220 * 1024);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(sample_kernel<BF16, HELD>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
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
  return cudaLaunchKernelEx(&cfg, sample_kernel<BF16, HELD>, a);
}

template <bool BF16>
cudaError_t launch_rows(const SampleArgs& a, cudaStream_t s) {
  // The more CTAs the sooner a row is done, down to slices of 16,384 elements; but few clusters of 16
  // find room at once, and rows that wait for room are done soonest by fours.  V = 248,320, fp32,
  // top-k 20 and top-p / no truncation, us: six rows on 16 CTAs 15.7 / 10.9, on eight 16.6 / 13.3; eight
  // rows 19.4 / 15.2 and 16.8 / 13.1; 32 rows on eight 22.8 / 22.6, on four 23.0 / 23.1; 48 rows 35.7 / 33.4
  // and 27.4 / 33.2, on two 31.3 / 36.4; 192 rows 101 / 105, 73 / 89 and 89 / 91.
  int C = 1;
  while (C < kMaxCluster && (long long)C * 16384 < a.V) C *= 2;
  if (C == 16 && a.M * 16 > 96) C = 8;
  if (C == 8 && a.M * 8 > 256) C = 4;
  // A slice is held in shared memory where two CTAs still share an SM (fp32, one row on 16: 14.7 / 9.4 us,
  // 15.0 / 10.4 read from L2), and a larger one where every CTA has an SM of its own (12 rows on eight:
  // 17.0 / 13.9 and 17.9 / 15.4; 16 rows: 27.0 / 23.9 and 19.9 / 20.6).
  const long long slice = (long long)((a.V + C * kWarps - 1) / (C * kWarps) + 127) / 128 * 128 * kWarps * (BF16 ? 2 : 4);
  return slice <= (a.M * C <= 96 ? 163840 : 65536) ? launch<BF16, true>(a, C, s) : launch<BF16, false>(a, C, s);
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
  const cudaError_t e = dtype == LOWBIT_LOGITS_BF16 ? launch_rows<true>(a, s) : launch_rows<false>(a, s);
  return e == cudaSuccess ? LOWBIT_OK : LOWBIT_ERR_CUDA;
}
