// Attention of new tokens over a paged key/value cache, one pass over the keys:
//   per query row   s_j = scale * q . k_j;  m = max_j s_j;  l = sum_j exp(s_j - m);
//                   o = sum_j exp(s_j - m) v_j;   out = o / l,   lse = m + log l,
// with (m, l, o) of any two sets of keys joined by m = max(m1, m2), l = l1 e^(m1-m) + l2 e^(m2-m)
// and o likewise -- so a tile of keys is folded in at a time, and a long axis is split freely.
//
// attn_mma_kernel works on the warp-level MMA (m16n8k16, fp32 accumulation).  A CTA holds 16 * MT
// query rows (the rows of one key/value head that share its keys) and takes key tiles of 64 from a
// ring that a fifth warp fills by TMA, one box per page and 128-byte part of a row; with MT < 4 row
// groups the four compute warps take different keys of the tile and join at the item's end.  The
// copying warp walks the items on its own, so the next item's tiles arrive while one is finished.
// The grid is resident and the work is cut evenly over it (see paged.cuh); a second kernel joins
// items that were cut (attn_combine_kernel; for shared prefixes prefix_join_kernel).
//
// The weights exp(s_j - m) enter their product as bf16, or over an e4m3 cache as fp16: the MMA takes 16-bit
// operands, and of the two each goes with a type that holds the values exactly.  l sums the weights
// as they were in fp32, so the rounding (at most 2^-8, or 2^-11, of a weight) shows in the output alone: an error of
// 0.0023 of it over 32,765 bf16 keys, of which 0.0017 is the output's own rounding.
//
// Bound: few rows per key/value head read the cache once and are bound by HBM, plus what a call pays
// whatever its size (start, an empty pipeline, the combine step: 7.8 us for one row over 777 keys).
// 64 ragged requests of one token over an e4m3 cache: 39.2 us, 176 MB, 4.5 TB/s; 32 rows of one
// request over 30,000 bf16 keys: 38.7 us, 123 MB, 3.2 TB/s (the copy rate is 6.8).
#pragma once

#include "common.cuh"
#include "paged.cuh"
#include "paged_attn.cuh"
#include "ptx.cuh"

#include <cuda_fp16.h>

namespace lowbit {
namespace {

using namespace ptx;

constexpr int kThreads = 160;
constexpr int kComputeThreads = 128;
constexpr int kJoinThreads = 256;
constexpr int kBN = 64;  // keys per tile
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}
template <bool F16>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (F16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Four e4m3 codes as two pairs of fp16 values, low bytes first.
__device__ __forceinline__ void e4m3x4_f16x4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 x, y;\n\tmov.b32 {x, y}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, x;\n\tcvt.rn.f16x2.e4m3x2 %1, y;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// What a row's weights refer to when the largest of its scores so far (in powers of two) is `top`.  Over an
// e4m3 cache they enter their product as fp16, which has no values below 2^-24: there the largest
// weight is 2^15 instead of 1, so a weight loses bits only below 2^-29 of the largest and becomes zero
// below 2^-40.  (With 1 as the largest, a tail of keys 2^26 times below one leading key left the output
// although it counted in the sum.)  Scores past 2^20, whose own rounding approaches the shift, keep 1.
template <bool F16>
__device__ __forceinline__ float reference(float top) {
  return F16 && !far_score(top) ? top - 15.0f : top;
}
template <bool F16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t d;
  if (F16) asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

template <int D, int MT, bool FP8>
struct Cfg {
  static constexpr int kWarpsK = 4 / MT;               // warps that split a tile's keys
  static constexpr int kRows = 16 * MT;
  static constexpr int kRowBytes = D * (FP8 ? 1 : 2);  // one key's or value's row
  static constexpr int kPart = kRowBytes < 128 ? kRowBytes : 128;  // of it, what one box holds
  static constexpr int kParts = kRowBytes / kPart;
  static constexpr int kHalf = kBN * kRowBytes;        // one tile's keys (or values)
  static constexpr int kStage = 2 * kHalf;
  static constexpr int kSteps = D / 16;
  static constexpr bool kQShared = D > 128;            // query fragments in shared memory
  static constexpr int kQBytes = kQShared ? MT * kSteps * 512 : 0;
  // Two CTAs per SM where three stages of a CTA fit half of its shared memory (all but heads of 256
  // in bf16), and as many stages as then fit, up to six.
  static constexpr int kCtas = 3 * kStage + kQBytes + 2048 <= 113 * 1024 ? 2 : 1;
  static constexpr int kFit = ((kCtas == 2 ? 113 : 226) * 1024 - 2048 - kQBytes) / kStage;
  static constexpr int kStages = kFit > 6 ? 6 : kFit;
  static constexpr int kSmem = 1024 + kStages * kStage + kQBytes;
  static_assert(2 * 64 * D <= kStage, "two warps' outputs pass through one stage");
};

// Byte offset of 16-byte chunk c of row r of a tile, as the tensor copy swizzles it: parts of 128
// bytes (chunk index XOR row mod 8) one after another, or rows of 64 bytes (XOR row / 2 mod 4).
template <int RB>
__device__ __forceinline__ uint32_t chunk_off(int r, int c) {
  if (RB == 64) return (uint32_t)(r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
  return (uint32_t)((c >> 3) * (kBN * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}
// Key (inside a group of eight) that the score matrix's column i stands for.  Over an e4m3 cache a
// lane reads 16 bytes of a key's row; taking rows 0, 4, 1, 5, ... puts the two rows that eight
// lanes read at once into different halves of the banks.  Values use the same order.
template <int RB, bool FP8>
__device__ __forceinline__ int key_of(int i) {
  return FP8 && RB >= 128 ? ((i >> 1) | ((i & 1) << 2)) : i;
}

struct RingBars {
  uint64_t full[8], empty[8];
  volatile int failed;  // some lane of the compute warps has given up a wait
};
__device__ __forceinline__ void init_bars(RingBars& bars, int stages) {
  for (int i = 0; i < stages; ++i) mbar_init(smem_addr(&bars.full[i]), 1), mbar_init(smem_addr(&bars.empty[i]), 4);
  bars.failed = 0;
  fence_mbar_init();
}
// A compute warp's wait; after the first one that gives up the warp takes no data and releases no stage, so
// that the copying warp finds none free and gives up too, and its rows are not stored.
__device__ __forceinline__ void take_or_fail(const AttnArgs& a, RingBars& bars, uint64_t& bar, uint32_t phase, bool& ok) {
  if (ok && !mbar_wait(smem_addr(&bar), phase)) {
    record_error(a.p.err, LOWBIT_ERR_TIMEOUT);
    bars.failed = 1;
    ok = false;
  }
}

// The copying warp: every key tile of the CTA's share, into the ring as stages come free.
template <class C, bool FP8, class A>
__device__ __forceinline__ void copy_tiles(const A& a, const CUtensorMap& kmap, const CUtensorMap& vmap,
                                           RingBars& bars, uint32_t ring, Walk it, int left) {
  constexpr int S = C::kStages, RB = C::kRowBytes;
  const PagedArgs& p = a.p;
  const int lane = threadIdx.x & 31;
  int stage = 0;
  uint32_t phase = 0;
  const int box = min(p.page_mask + 1, kBN), boxes = kBN / box;  // keys per box
  int filled = 0;
  bool ok = true;
  for (;;) {
    const int kt0 = it.tile, kt1 = kt0 + walk_take(it, left);
    if (kt1 == kt0) break;
    const int first = (it.span.lo & ~(kBN - 1)) + lane * box;
    const int32_t* row = table_of(a, it.b, it.q);
    // Page of this lane's box of tile kt (-2: no key of it is seen), looked up one tile ahead.
    auto page_of = [&](int kt, int extra) {
      const int key = first + kt * kBN + extra * box;
      if (lane + extra >= boxes || key >= it.span.hi || key + box <= it.span.lo) return -2;
      const int page = __ldg(row + (key >> p.page_shift));
      if (page >= 0 && page < p.pages) return page;
      record_error(p.err, LOWBIT_ERR_INVALID_ARG);
      return -1;  // outside the tensor map: the copy fills zeros
    };
    int next = page_of(kt0, 0);
    for (int kt = kt0; kt < kt1; ++kt) {
      const int page = next;
      if (kt + 1 < kt1) next = page_of(kt + 1, 0);
      if (!mbar_wait(smem_addr(&bars.empty[stage]), phase ^ 1)) {
        record_error(p.err, LOWBIT_ERR_TIMEOUT);
        ok = false;
        break;
      }
      if (a.stall) {  // nothing is copied
        if (++stage == S) stage = 0, phase ^= 1;
        continue;
      }
      const uint32_t bar = smem_addr(&bars.full[stage]);
      const int page2 = boxes > 32 ? page_of(kt, 32) : -2;  // pages of one slot: 64 boxes
      const int n = __popc(__ballot_sync(~0u, page != -2)) + __popc(__ballot_sync(~0u, page2 != -2));
      if (lane == 0) mbar_arrive_expect_tx(bar, (uint32_t)(n * box * RB * 2));
      __syncwarp();
      const int slot = (first + kt * kBN) & p.page_mask;
      auto copy = [&](int pg, int i) {
        const uint32_t dst = ring + stage * C::kStage + i * box * C::kPart;
#pragma unroll
        for (int part = 0; part < C::kParts; ++part) {
          constexpr int kElems = C::kPart / (FP8 ? 1 : 2);
          tma_load_4d(dst + part * (kBN * C::kPart), &kmap, part * kElems, slot, it.h, pg, bar);
          tma_load_4d(dst + C::kHalf + part * (kBN * C::kPart), &vmap, part * kElems, slot, it.h, pg, bar);
        }
      };
      if (page != -2) copy(page, lane);
      if (page2 != -2) copy(page2, lane + 32);
      if (++stage == S) stage = 0, phase ^= 1;
      if (filled < S) ++filled;
    }
    if (!ok || left <= 0 || !walk_next(a, it)) break;
  }
  // leave only when no copy is in flight
  for (int i = 0; i < filled; ++i) {
    if (--stage < 0) stage = S - 1, phase ^= 1;
    mbar_wait(smem_addr(&bars.full[stage]), phase);
  }
}

template <int D, int MT, bool FP8, class A>
__global__ void __launch_bounds__(kThreads, Cfg<D, MT, FP8>::kCtas)
attn_mma_kernel(const __grid_constant__ A a, const __grid_constant__ CUtensorMap kmap,
                const __grid_constant__ CUtensorMap vmap) {
  using C = Cfg<D, MT, FP8>;
  constexpr int RB = C::kRowBytes, S = C::kStages;
  constexpr int kNT = 2 * MT;       // 8-key tiles per warp
  constexpr int kDT = D / 8;        // 8-dim tiles
  extern __shared__ uint8_t raw[];
  __shared__ RingBars bars;
  __shared__ float2 s_ml[4][16];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t ring = (smem_addr(raw) + 1023u) & ~1023u;
  uint8_t* const smem = raw + (ring - smem_addr(raw));
  const PagedArgs& p = a.p;

  if (tid == 0) {
    init_bars(bars, S);
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __syncthreads();  // the barriers are initialised
  Walk it;
  Share share;
  const bool busy = start_walk<kThreads>(a, blockIdx.x, it, share);
  if (!kPrefix<A> && tid == 0) say_cut(a, blockIdx.x, nullptr, 0, 1, 0);
  if (!busy) return;
  int left = share.left;
  int stage = 0;
  uint32_t phase = 0;

  if (warp == 4) {
    copy_tiles<C, FP8>(a, kmap, vmap, bars, ring, it, left);
    return;
  }

  const int g = lane >> 2, t = lane & 3;
  const int wr = warp / C::kWarpsK, wk = warp % C::kWarpsK;  // row group, key group
  const int wkey = wk * kNT * 8;                              // this warp's keys inside a tile
  bool first = true, ok = true;
  for (;;) {
    const Request q = it.q;
    const int kt0 = it.tile, kt1 = kt0 + walk_take(it, left);
    if (kt1 == kt0) return;
    const Span span = it.span;
    const int base_key = span.lo & ~(kBN - 1);
    const int r0 = it.qt * C::kRows;
    const int rows = q.n * a.shape.G;  // query rows of the request for this head

    // ---- this warp's two row slots per lane: g and g + 8 of its 16 rows
    int jlo[2], jhi[2];
    long long qrow[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = r0 + wr * 16 + g + 8 * i;
      const int tok = token_of(a.shape, r);
      const bool in = r < rows;
      const int pos = q.kv - q.n + tok;
      jhi[i] = in ? (a.shape.causal && !q.all ? min(q.kv, pos + 1) : q.kv) : 0;
      jlo[i] = first_key(a.shape, pos);
      qrow[i] = in ? (long long)(q.row0 + tok) * a.Hq + it.h * a.shape.G + (r - tok * a.shape.G) : -1;
    }
    // keys that every row of the CTA's tile sees need no mask
    const int last_row = min(r0 + C::kRows, rows) - 1;
    const int all_lo = first_key(a.shape, q.kv - q.n + token_of(a.shape, last_row));
    const int all_hi = a.shape.causal && !q.all ? min(q.kv, q.kv - q.n + token_of(a.shape, r0) + 1) : q.kv;

    // ---- query fragments; with an e4m3 cache the row is scaled by a power of two into fp16
    uint32_t qf[C::kQShared ? 1 : C::kSteps][4];
    float coef[2];  // exponent per unit of the raw product, in powers of two
    uint4* const qs = reinterpret_cast<uint4*>(smem + S * C::kStage) + (size_t)wr * C::kSteps * 32;
    {
      const float ks = FP8 && p.k_scale ? __ldg(p.k_scale + it.h) : 1.0f;
      uint32_t f[C::kSteps][4];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = r0 + wr * 16 + g + 8 * i;
        const int tok = token_of(a.shape, r);
        const uint16_t* src = a.q + (long long)(q.row0 + tok) * a.q_stride + (long long)(it.h * a.shape.G + r - tok * a.shape.G) * D;
#pragma unroll
        for (int st = 0; st < C::kSteps; ++st)
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            // bf16: columns 16 st + 2t (+8); e4m3: the order in which a 16-byte load of a key's
            // row hands them out, 64 (st/4) + 16 t + 4 (st%4) (+2)
            const int col = FP8 ? 64 * (st / 4) + 16 * t + 4 * (st % 4) + half * 2 : 16 * st + 2 * t + half * 8;
            f[st][2 * half + i] = qrow[i] >= 0 ? *reinterpret_cast<const uint32_t*>(src + col) : 0u;
          }
      }
      coef[0] = coef[1] = a.scale * ks * kLog2e;
      if (FP8) {
        // the four lanes of a row hold all of it
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float top = 0.0f;
#pragma unroll
          for (int st = 0; st < C::kSteps; ++st)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              const uint32_t v = f[st][2 * half + i];
              top = fmaxf(top, fmaxf(fabsf(__uint_as_float(v << 16)), fabsf(__uint_as_float(v & 0xFFFF0000u))));
            }
          top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
          top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
          // 2^-e with 2^e <= top < 2^(e+1): the row's largest becomes 1..2.  A row of zeros, or one
          // with an Inf or a NaN, stays as it is.
          const int e = (int)(__float_as_uint(top) >> 23) - 127;
          const int ee = (top > 0.0f && e < 128) ? max(-100, min(100, e)) : 0;
          const float up = __uint_as_float((uint32_t)(127 - ee) << 23);
          coef[i] *= __uint_as_float((uint32_t)(127 + ee) << 23);
#pragma unroll
          for (int st = 0; st < C::kSteps; ++st)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              const uint32_t v = f[st][2 * half + i];
              f[st][2 * half + i] = pack2<true>(__uint_as_float(v << 16) * up, __uint_as_float(v & 0xFFFF0000u) * up);
            }
        }
      }
#pragma unroll
      for (int st = 0; st < C::kSteps; ++st) {
        if (C::kQShared) {
          if (wk == 0) qs[st * 32 + lane] = make_uint4(f[st][0], f[st][1], f[st][2], f[st][3]);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) qf[C::kQShared ? 0 : st][i] = f[st][i];
        }
      }
      if (C::kQShared) named_barrier(1, kComputeThreads);
    }

    float o[kDT][4];
#pragma unroll
    for (int i = 0; i < kDT; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[i][e] = 0.0f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
    int last = 0;  // stage of the item's last tile, released after the join

    for (int kt = kt0; kt < kt1; ++kt) {
      take_or_fail(a, bars, bars.full[stage], phase, ok);
      const uint32_t ks = ring + stage * C::kStage, vs = ks + C::kHalf;
      const int key0 = base_key + kt * kBN;

      // Values outside the span (unwritten slots, what an earlier tile left) become zeros, since
      // 0 * NaN would reach the sums.  Every warp clears all rows that it reads.
      if (key0 < span.lo || key0 + kBN > span.hi) {
        constexpr int kChunks = RB / 16;
        for (int i = lane; i < kNT * 8 * kChunks; i += 32) {
          const int r = wkey + i / kChunks;
          if (key0 + r < span.lo || key0 + r >= span.hi)
            asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(vs + chunk_off<RB>(r, i % kChunks)), "r"(0) : "memory");
        }
        fence_proxy_async_smem();
        __syncwarp();
      }

      // scores of 16 rows and kNT * 8 keys
      float sc[kNT][4];
#pragma unroll
      for (int i = 0; i < kNT; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[i][e] = 0.0f;
      if (FP8) {
#pragma unroll
        for (int j = 0; j < D / 64; ++j) {
          uint32_t qa[4][4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if (C::kQShared) {
              const uint4 v = qs[(4 * j + e) * 32 + lane];
              qa[e][0] = v.x, qa[e][1] = v.y, qa[e][2] = v.z, qa[e][3] = v.w;
            } else {
#pragma unroll
              for (int i = 0; i < 4; ++i) qa[e][i] = qf[C::kQShared ? 0 : 4 * j + e][i];
            }
          }
#pragma unroll
          for (int n = 0; n < kNT; ++n) {
            const uint4 kw = lds128(ks + chunk_off<RB>(wkey + n * 8 + key_of<RB, FP8>(g), 4 * j + t));
            const uint32_t ww[4] = {kw.x, kw.y, kw.z, kw.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              uint32_t b0, b1;
              e4m3x4_f16x4(ww[e], b0, b1);
              mma16816<true>(sc[n], qa[e], b0, b1);
            }
          }
        }
      } else {
#pragma unroll
        for (int st = 0; st < C::kSteps; ++st) {
          uint32_t qa[4];
          if (C::kQShared) {
            const uint4 v = qs[st * 32 + lane];
            qa[0] = v.x, qa[1] = v.y, qa[2] = v.z, qa[3] = v.w;
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) qa[i] = qf[C::kQShared ? 0 : st][i];
          }
#pragma unroll
          for (int n = 0; n < kNT; n += 2) {
            uint32_t kb[4];
            const int r = wkey + n * 8 + ((lane >> 4) << 3) + (lane & 7);
            ldsm4(kb, ks + chunk_off<RB>(r, 2 * st + ((lane >> 3) & 1)));
            mma16816<false>(sc[n], qa, kb[0], kb[1]);
            mma16816<false>(sc[n + 1], qa, kb[2], kb[3]);
          }
        }
      }

      // scaled (in powers of two) and, where the tile is not seen whole by every row, masked
      const bool masked = key0 < all_lo || key0 + kBN > all_hi;
      float tm[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int n = 0; n < kNT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          sc[n][e] *= coef[e >> 1];
          const int key = key0 + wkey + n * 8 + key_of<RB, FP8>(2 * t + (e & 1));
          if (masked && (key < jlo[e >> 1] || key >= jhi[e >> 1])) sc[n][e] = -INFINITY;
          tm[e >> 1] = fmaxf(tm[e >> 1], sc[n][e]);
        }
      // fold the tile in
      float keep[2], base[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        tm[i] = fmaxf(tm[i], __shfl_xor_sync(~0u, tm[i], 1));
        tm[i] = fmaxf(tm[i], __shfl_xor_sync(~0u, tm[i], 2));
        const float mn = fmaxf(m[i], reference<FP8>(tm[i]));
        base[i] = mn == -INFINITY ? 0.0f : mn;  // nothing seen yet: every weight is 2^-inf = 0
        keep[i] = ex2(m[i] - base[i]);
        m[i] = mn;
        l[i] *= keep[i];
      }
      uint32_t pa[kNT / 2][4];
#pragma unroll
      for (int n = 0; n < kNT; ++n) {
        float w4[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          w4[e] = ex2(sc[n][e] - base[e >> 1]);
          l[e >> 1] += w4[e];
        }
        pa[n / 2][(n & 1) * 2] = pack2<FP8>(w4[0], w4[1]);
        pa[n / 2][(n & 1) * 2 + 1] = pack2<FP8>(w4[2], w4[3]);
      }
      if (__any_sync(~0u, keep[0] != 1.0f || keep[1] != 1.0f)) {
#pragma unroll
        for (int i = 0; i < kDT; ++i) {
          o[i][0] *= keep[0], o[i][1] *= keep[0];
          o[i][2] *= keep[1], o[i][3] *= keep[1];
        }
      }
      // o += weights x values
#pragma unroll
      for (int k2 = 0; k2 < kNT / 2; ++k2) {
        const int r = wkey + k2 * 16 + ((lane >> 3) & 1) * 8 + key_of<RB, FP8>(lane & 7);
        if (FP8) {
#pragma unroll
          for (int d = 0; d < D / 32; ++d) {
            uint32_t vb[4];
            ldsm4t(vb, vs + chunk_off<RB>(r, 2 * d + (lane >> 4)));
            // a word holds two keys' bytes of an even and an odd dim: [k0 d0, k0 d1, k1 d0, k1 d1]
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
              uint32_t even[2], odd[2];
              e4m3x4_f16x4(__byte_perm(vb[2 * hh], 0, 0x3120), even[0], odd[0]);
              e4m3x4_f16x4(__byte_perm(vb[2 * hh + 1], 0, 0x3120), even[1], odd[1]);
              mma16816<true>(o[4 * d + 2 * hh], pa[k2], even[0], even[1]);
              mma16816<true>(o[4 * d + 2 * hh + 1], pa[k2], odd[0], odd[1]);
            }
          }
        } else {
#pragma unroll
          for (int d = 0; d < D / 16; ++d) {
            uint32_t vb[4];
            ldsm4t(vb, vs + chunk_off<RB>(r, 2 * d + (lane >> 4)));
            mma16816<false>(o[2 * d], pa[k2], vb[0], vb[1]);
            mma16816<false>(o[2 * d + 1], pa[k2], vb[2], vb[3]);
          }
        }
      }
      last = stage;
      if (kt + 1 < kt1 || MT == 4) {
        __syncwarp();
        if (lane == 0 && ok) mbar_arrive(smem_addr(&bars.empty[stage]));
      }
      if (++stage == S) stage = 0, phase ^= 1;
    }

#pragma unroll
    for (int i = 0; i < 2; ++i) {
      l[i] += __shfl_xor_sync(~0u, l[i], 1);
      l[i] += __shfl_xor_sync(~0u, l[i], 2);
    }
    // ---- join the warps of a row group, through the last tile's stage: two warps' fragments fit
    if (MT < 4) {
      if (t == 0) {
        s_ml[warp][g] = make_float2(m[0], l[0]);
        s_ml[warp][g + 8] = make_float2(m[1], l[1]);
      }
      named_barrier(1, kComputeThreads);  // also: every warp is done with the last tile
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float mm = -INFINITY, ll = 0.0f;
#pragma unroll
        for (int k = 0; k < C::kWarpsK; ++k) mm = fmaxf(mm, s_ml[wr * C::kWarpsK + k][g + 8 * i].x);
        const float f = mm == -INFINITY ? 0.0f : ex2(m[i] - mm);
#pragma unroll
        for (int k = 0; k < C::kWarpsK; ++k) {
          const float2 x = s_ml[wr * C::kWarpsK + k][g + 8 * i];
          ll += (mm == -INFINITY ? 0.0f : ex2(x.x - mm)) * x.y;
        }
        m[i] = mm;
        l[i] = ll;
#pragma unroll
        for (int d = 0; d < kDT; ++d) o[d][2 * i] *= f, o[d][2 * i + 1] *= f;
      }
      float4* const buf = reinterpret_cast<float4*>(smem + last * C::kStage) + lane;
      auto give = [&](int place) {
#pragma unroll
        for (int d = 0; d < kDT; ++d) buf[(place * kDT + d) * 32] = make_float4(o[d][0], o[d][1], o[d][2], o[d][3]);
      };
      auto take = [&](int place) {
#pragma unroll
        for (int d = 0; d < kDT; ++d) {
          const float4 v = buf[(place * kDT + d) * 32];
          o[d][0] += v.x, o[d][1] += v.y, o[d][2] += v.z, o[d][3] += v.w;
        }
      };
      if (MT == 1) {
        if (wk >= 2) give(wk - 2);
        named_barrier(1, kComputeThreads);
        if (wk < 2) take(wk);
        if (wk == 1) give(1);  // over what it has just read
        named_barrier(1, kComputeThreads);
        if (wk == 0) take(1);
      } else {
        if (wk == 1) give(wr);
        named_barrier(1, kComputeThreads);
        if (wk == 0) take(wr);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0 && ok) mbar_arrive(smem_addr(&bars.empty[last]));
    }

    // ---- store: the row group's first warp holds its rows
    if (wk == 0) {
      // what other warps added: their failures came before the join's barriers
      const bool good = MT < 4 ? !bars.failed : __all_sync(~0u, ok);
      const bool whole = kt0 == 0 && kt1 == it.tiles, final = whole && !kPrefix<A>;
      const float vscale = FP8 && p.v_scale ? __ldg(p.v_scale + it.h) : 1.0f;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (qrow[i] < 0) continue;
        const long long piece = (2LL * blockIdx.x + (first ? 0 : 1)) * C::kRows + wr * 16 + g + 8 * i;
        const Part to = part_of<D>(a, it, whole, qrow[i], piece);
        float* const part = to.o;
        if (t == 0 && kt0 == 0) say_found(a, it, qrow[i], good, kt1, wr * 16 + g + 8 * i, share.chunk, piece);
        if (!good) {
          if (t == 0 && !final) *to.ml = make_float2(0.0f, kNoPiece);
          continue;
        }
        const float f = final ? (l[i] > 0.0f ? vscale / l[i] : (l[i] == 0.0f ? 0.0f : l[i])) : 1.0f;
        uint16_t* const dst = a.out + qrow[i] * D;
#pragma unroll
        for (int d = 0; d < kDT; d += 2) {
          const float x0 = o[d][2 * i] * f, x1 = o[d][2 * i + 1] * f, y0 = o[d + 1][2 * i] * f, y1 = o[d + 1][2 * i + 1] * f;
          if (FP8) {  // dims 8 d + 4 t ..: even ones in tile d, odd ones in tile d + 1
            if (final) *reinterpret_cast<uint2*>(dst + 8 * d + 4 * t) = make_uint2(pack2<false>(x0, y0), pack2<false>(x1, y1));
            else *reinterpret_cast<float4*>(part + 8 * d + 4 * t) = make_float4(x0, y0, x1, y1);
          } else if (final) {
            *reinterpret_cast<uint32_t*>(dst + 8 * d + 2 * t) = pack2<false>(x0, x1);
            *reinterpret_cast<uint32_t*>(dst + 8 * d + 8 + 2 * t) = pack2<false>(y0, y1);
          } else {
            *reinterpret_cast<float2*>(part + 8 * d + 2 * t) = make_float2(x0, x1);
            *reinterpret_cast<float2*>(part + 8 * d + 8 + 2 * t) = make_float2(y0, y1);
          }
        }
        if (t == 0) {
          if (!final) *to.ml = make_float2(m[i], l[i]);
          else if (a.lse) a.lse[qrow[i]] = l[i] == 0.0f ? -INFINITY : m[i] * 0.6931471805599453f + logf(l[i]);
        }
      }
    }
    if (!kPrefix<A> && tid == 0 && kt0 == 0 && kt1 < it.tiles)
      say_cut(a, blockIdx.x, &it, kt1, share.chunk, 2 * blockIdx.x + (first ? 0 : 1));
    if (C::kQShared || MT < 4) named_barrier(1, kComputeThreads);  // s_ml and qs are free again
    first = false;
    if (left <= 0 || !walk_next(a, it)) return;
  }
}

// Eight rows and fewer (a decode step: one token, up to eight heads a group).  The products change
// sides, so that the keys, not the rows, fill the MMA's 16: S^T = K Q^T and O^T = V^T P^T, half the MMAs and half
// the exponentials of the 16-row kernel.  A lane holds two keys' scores of rows 2t and 2t + 1; P^T
// becomes the other operand by an 8 x 8 transpose of its 16-bit pairs.  64 requests of 1 to 16,384 keys
// over an e4m3 cache: 47.4 us on the 16-row kernel, whose issue slots were the limit, 39.2 us here.
template <int D, bool FP8>
struct Cfg8 {
  static constexpr int kRowBytes = D * (FP8 ? 1 : 2);
  static constexpr int kPart = kRowBytes < 128 ? kRowBytes : 128;
  static constexpr int kParts = kRowBytes / kPart;
  static constexpr int kHalf = kBN * kRowBytes;
  static constexpr int kStage = 2 * kHalf;
  static constexpr int kSteps = D / 16;
  static constexpr int kCtas = kStage <= 8192 ? 4 : (kStage <= 16384 ? 3 : (kStage <= 32768 ? 2 : 1));
  static constexpr int kFit = (227 * 1024 / kCtas - 3 * 1024) / kStage;
  static constexpr int kStages = kFit > 6 ? 6 : kFit;
  static constexpr int kSmem = 1024 + kStages * kStage;
  static_assert(64 * D <= kStage, "two warps' outputs pass through one stage");
};

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

template <int D, bool FP8, class A>
__global__ void __launch_bounds__(kThreads, Cfg8<D, FP8>::kCtas)
attn_row8_kernel(const __grid_constant__ A a, const __grid_constant__ CUtensorMap kmap,
                 const __grid_constant__ CUtensorMap vmap) {
  using C = Cfg8<D, FP8>;
  constexpr int RB = C::kRowBytes, S = C::kStages, kDT = D / 16;
  extern __shared__ uint8_t raw[];
  __shared__ RingBars bars;
  __shared__ float2 s_ml[4][8];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t ring = (smem_addr(raw) + 1023u) & ~1023u;
  uint8_t* const smem = raw + (ring - smem_addr(raw));
  const PagedArgs& p = a.p;

  if (tid == 0) {
    init_bars(bars, S);
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __syncthreads();  // the barriers are initialised
  Walk it;
  Share share;
  const bool busy = start_walk<kThreads>(a, blockIdx.x, it, share);
  if (!kPrefix<A> && tid == 0) say_cut(a, blockIdx.x, nullptr, 0, 1, 0);
  if (!busy) return;
  int left = share.left;
  if (warp == 4) {
    copy_tiles<C, FP8>(a, kmap, vmap, bars, ring, it, left);
    return;
  }

  int stage = 0;
  uint32_t phase = 0;
  const int g = lane >> 2, t = lane & 3;
  const int wkey = warp * 16;  // this warp's keys inside a tile
  bool first = true, ok = true;
  for (;;) {
    const Request q = it.q;
    const int kt0 = it.tile, kt1 = kt0 + walk_take(it, left);
    if (kt1 == kt0) return;
    const Span span = it.span;
    const int base_key = span.lo & ~(kBN - 1);
    const int r0 = it.qt * 8, rows = q.n * a.shape.G;

    // the query operand: row g's elements; over an e4m3 cache scaled by a power of two into fp16
    uint32_t qf[C::kSteps][2];
    float row_coef = a.scale * (FP8 && p.k_scale ? __ldg(p.k_scale + it.h) : 1.0f) * kLog2e;
    {
      const int r = r0 + g, tok = token_of(a.shape, r);
      const uint16_t* src = a.q + (long long)(q.row0 + tok) * a.q_stride + (long long)(it.h * a.shape.G + r - tok * a.shape.G) * D;
#pragma unroll
      for (int st = 0; st < C::kSteps; ++st)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int col = FP8 ? 64 * (st / 4) + 16 * t + 4 * (st % 4) + i * 2 : 16 * st + 2 * t + i * 8;
          qf[st][i] = r < rows ? *reinterpret_cast<const uint32_t*>(src + col) : 0u;
        }
      if (FP8) {  // as in attn_mma_kernel
        float top = 0.0f;
#pragma unroll
        for (int st = 0; st < C::kSteps; ++st)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            top = fmaxf(top, fmaxf(fabsf(__uint_as_float(qf[st][i] << 16)), fabsf(__uint_as_float(qf[st][i] & 0xFFFF0000u))));
        top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
        top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
        const int e = (int)(__float_as_uint(top) >> 23) - 127;
        const int ee = (top > 0.0f && e < 128) ? max(-100, min(100, e)) : 0;
        const float up = __uint_as_float((uint32_t)(127 - ee) << 23);
        row_coef *= __uint_as_float((uint32_t)(127 + ee) << 23);
#pragma unroll
        for (int st = 0; st < C::kSteps; ++st)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            qf[st][i] = pack2<true>(__uint_as_float(qf[st][i] << 16) * up, __uint_as_float(qf[st][i] & 0xFFFF0000u) * up);
      }
    }
    // the two rows whose scores this lane holds
    int jlo[2], jhi[2];
    long long qrow[2];
    float coef[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = r0 + 2 * t + i, tok = token_of(a.shape, r), pos = q.kv - q.n + tok;
      const bool in = r < rows;
      jhi[i] = in ? (a.shape.causal && !q.all ? min(q.kv, pos + 1) : q.kv) : 0;
      jlo[i] = first_key(a.shape, pos);
      qrow[i] = in ? (long long)(q.row0 + tok) * a.Hq + it.h * a.shape.G + (r - tok * a.shape.G) : -1;
      coef[i] = __shfl_sync(~0u, row_coef, (2 * t + i) * 4);
    }
    const int last_row = min(r0 + 8, rows) - 1;
    const int all_lo = first_key(a.shape, q.kv - q.n + token_of(a.shape, last_row));
    const int all_hi = a.shape.causal && !q.all ? min(q.kv, q.kv - q.n + token_of(a.shape, r0) + 1) : q.kv;

    float o[kDT][4];
#pragma unroll
    for (int i = 0; i < kDT; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[i][e] = 0.0f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
    int last = 0;

    for (int kt = kt0; kt < kt1; ++kt) {
      take_or_fail(a, bars, bars.full[stage], phase, ok);
      const uint32_t ks = ring + stage * C::kStage, vs = ks + C::kHalf;
      const int key0 = base_key + kt * kBN;
      if (key0 < span.lo || key0 + kBN > span.hi) {  // values outside the span: as in attn_mma_kernel
        constexpr int kChunks = RB / 16;
        for (int i = lane; i < 16 * kChunks; i += 32) {
          const int r = wkey + i / kChunks;
          if (key0 + r < span.lo || key0 + r >= span.hi)
            asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(vs + chunk_off<RB>(r, i % kChunks)), "r"(0) : "memory");
        }
        fence_proxy_async_smem();
        __syncwarp();
      }

      // scores of keys g and g + 8, rows 2t and 2t + 1; two chains, joined
      float sc[4] = {0.f, 0.f, 0.f, 0.f}, sd[4] = {0.f, 0.f, 0.f, 0.f};
      if (FP8) {
#pragma unroll
        for (int j = 0; j < D / 64; ++j) {
          const uint4 x = lds128(ks + chunk_off<RB>(wkey + key_of<RB, FP8>(g), 4 * j + t));
          const uint4 y = lds128(ks + chunk_off<RB>(wkey + 8 + key_of<RB, FP8>(g), 4 * j + t));
          const uint32_t xw[4] = {x.x, x.y, x.z, x.w}, yw[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint32_t f[4];
            e4m3x4_f16x4(xw[e], f[0], f[2]);
            e4m3x4_f16x4(yw[e], f[1], f[3]);
            mma16816<true>(e & 1 ? sd : sc, f, qf[4 * j + e][0], qf[4 * j + e][1]);
          }
        }
      } else {
#pragma unroll
        for (int st = 0; st < C::kSteps; ++st) {
          uint32_t f[4];  // keys 0-7 and 8-15 of dims 0-7, then of dims 8-15
          ldsm4(f, ks + chunk_off<RB>(wkey + (lane & 15), 2 * st + (lane >> 4)));
          mma16816<false>(st & 1 ? sd : sc, f, qf[st][0], qf[st][1]);
        }
      }

      const bool masked = key0 < all_lo || key0 + kBN > all_hi;
      float tm[2];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        sc[e] = (sc[e] + sd[e]) * coef[e & 1];
        const int key = key0 + wkey + key_of<RB, FP8>(g) + 8 * (e >> 1);
        if (masked && (key < jlo[e & 1] || key >= jhi[e & 1])) sc[e] = -INFINITY;
      }
      float keep[2], base[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        tm[i] = fmaxf(sc[i], sc[2 + i]);
#pragma unroll
        for (int x = 4; x < 32; x *= 2) tm[i] = fmaxf(tm[i], __shfl_xor_sync(~0u, tm[i], x));
        const float mn = fmaxf(m[i], reference<FP8>(tm[i]));
        base[i] = mn == -INFINITY ? 0.0f : mn;
        keep[i] = ex2(m[i] - base[i]);
        m[i] = mn;
        l[i] *= keep[i];
      }
      uint32_t pb[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {  // keys g, then keys g + 8
        const float x = ex2(sc[2 * i] - base[0]), y = ex2(sc[2 * i + 1] - base[1]);
        l[0] += x;
        l[1] += y;
        pb[i] = transpose8x8(pack2<FP8>(x, y));
      }
      if (__any_sync(~0u, keep[0] != 1.0f || keep[1] != 1.0f)) {
#pragma unroll
        for (int i = 0; i < kDT; ++i) {
          o[i][0] *= keep[0], o[i][1] *= keep[1];
          o[i][2] *= keep[0], o[i][3] *= keep[1];
        }
      }
      const int r = wkey + ((lane >> 3) & 1) * 8 + key_of<RB, FP8>(lane & 7);
      if (FP8) {
#pragma unroll
        for (int d = 0; d < D / 32; ++d) {
          uint32_t vb[4];
          ldsm4t(vb, vs + chunk_off<RB>(r, 2 * d + (lane >> 4)));
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            // rows g: even dims, rows g + 8: odd dims, of this group of 16
            uint32_t f[4];
            e4m3x4_f16x4(__byte_perm(vb[2 * hh], 0, 0x3120), f[0], f[1]);
            e4m3x4_f16x4(__byte_perm(vb[2 * hh + 1], 0, 0x3120), f[2], f[3]);
            mma16816<true>(o[2 * d + hh], f, pb[0], pb[1]);
          }
        }
      } else {
#pragma unroll
        for (int d = 0; d < kDT; ++d) {
          uint32_t vb[4];
          ldsm4t(vb, vs + chunk_off<RB>(r, 2 * d + (lane >> 4)));
          const uint32_t f[4] = {vb[0], vb[2], vb[1], vb[3]};
          mma16816<false>(o[d], f, pb[0], pb[1]);
        }
      }
      last = stage;
      if (kt + 1 < kt1) {
        __syncwarp();
        if (lane == 0 && ok) mbar_arrive(smem_addr(&bars.empty[stage]));
      }
      if (++stage == S) stage = 0, phase ^= 1;
    }

    // ---- join the four warps, through the last tile's stage
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
      for (int x = 4; x < 32; x *= 2) l[i] += __shfl_xor_sync(~0u, l[i], x);
      if (g == 0) s_ml[warp][2 * t + i] = make_float2(m[i], l[i]);
    }
    named_barrier(1, kComputeThreads);  // also: every warp is done with the last tile
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float mm = -INFINITY, ll = 0.0f;
#pragma unroll
      for (int k = 0; k < 4; ++k) mm = fmaxf(mm, s_ml[k][2 * t + i].x);
      const float f = mm == -INFINITY ? 0.0f : ex2(m[i] - mm);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 x = s_ml[k][2 * t + i];
        ll += (mm == -INFINITY ? 0.0f : ex2(x.x - mm)) * x.y;
      }
      m[i] = mm;
      l[i] = ll;
#pragma unroll
      for (int d = 0; d < kDT; ++d) o[d][i] *= f, o[d][2 + i] *= f;
    }
    float4* const buf = reinterpret_cast<float4*>(smem + last * C::kStage) + lane;
    auto give = [&](int place) {
#pragma unroll
      for (int d = 0; d < kDT; ++d) buf[(place * kDT + d) * 32] = make_float4(o[d][0], o[d][1], o[d][2], o[d][3]);
    };
    auto take = [&](int place) {
#pragma unroll
      for (int d = 0; d < kDT; ++d) {
        const float4 v = buf[(place * kDT + d) * 32];
        o[d][0] += v.x, o[d][1] += v.y, o[d][2] += v.z, o[d][3] += v.w;
      }
    };
    if (warp >= 2) give(warp - 2);
    named_barrier(1, kComputeThreads);
    if (warp < 2) take(warp);
    if (warp == 1) give(1);  // over what it has just read
    named_barrier(1, kComputeThreads);
    if (warp == 0) take(1);
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0 && ok) mbar_arrive(smem_addr(&bars.empty[last]));

    if (warp == 0) {
      const bool good = !bars.failed;  // as in attn_mma_kernel
      const bool whole = kt0 == 0 && kt1 == it.tiles, final = whole && !kPrefix<A>;
      const float vscale = FP8 && p.v_scale ? __ldg(p.v_scale + it.h) : 1.0f;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (qrow[i] < 0) continue;
        const long long piece = (2LL * blockIdx.x + (first ? 0 : 1)) * 8 + 2 * t + i;
        const Part to = part_of<D>(a, it, whole, qrow[i], piece);
        float* const part = to.o;
        if (g == 0 && kt0 == 0) say_found(a, it, qrow[i], good, kt1, 2 * t + i, share.chunk, piece);
        if (!good) {
          if (g == 0 && !final) *to.ml = make_float2(0.0f, kNoPiece);
          continue;
        }
        const float f = final ? (l[i] > 0.0f ? vscale / l[i] : (l[i] == 0.0f ? 0.0f : l[i])) : 1.0f;
        uint16_t* const dst = a.out + qrow[i] * D;
#pragma unroll
        for (int d = 0; d < kDT; ++d) {
          const float x = o[d][i] * f, y = o[d][2 + i] * f;
          if (FP8) {  // dims 16 d + 2 g and the next
            if (final) *reinterpret_cast<uint32_t*>(dst + 16 * d + 2 * g) = pack2<false>(x, y);
            else *reinterpret_cast<float2*>(part + 16 * d + 2 * g) = make_float2(x, y);
          } else if (final) {  // dims 16 d + g and + 8
            dst[16 * d + g] = float_to_bf16_bits(x);
            dst[16 * d + g + 8] = float_to_bf16_bits(y);
          } else {
            part[16 * d + g] = x;
            part[16 * d + g + 8] = y;
          }
        }
        if (g == 0) {
          if (!final) *to.ml = make_float2(m[i], l[i]);
          else if (a.lse) a.lse[qrow[i]] = l[i] == 0.0f ? -INFINITY : m[i] * 0.6931471805599453f + logf(l[i]);
        }
      }
    }
    if (!kPrefix<A> && tid == 0 && kt0 == 0 && kt1 < it.tiles)
      say_cut(a, blockIdx.x, &it, kt1, share.chunk, 2 * blockIdx.x + (first ? 0 : 1));
    named_barrier(1, kComputeThreads);  // s_ml is free again
    first = false;
    if (left <= 0 || !walk_next(a, it)) return;
  }
}

// `kernel` with 1 << r_shift rows per item on a resident grid, and the combine step behind it.
template <class C, class A>
cudaError_t launch_ring(void (*kernel)(const A, const CUtensorMap, const CUtensorMap), std::atomic<int>* ready,
                        A a, int D, bool fp8, int r_shift, cudaStream_t s) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  int ctas = ready[dev].load(std::memory_order_relaxed);
  if (!ctas) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    int sms = 0, per = 0;
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kernel, kThreads, C::kSmem);
    if (e != cudaSuccess) return e;
    ctas = std::max(1, std::min(std::min(sms * per, kMaxCtas), kMaxPieceRows / 2 >> r_shift));
    ready[dev].store(ctas, std::memory_order_relaxed);
  }
  CUtensorMap kmap, vmap;
  if (!encode_cache(&kmap, a.p, a.p.k, D, fp8, kBN) || !encode_cache(&vmap, a.p, a.p.v, D, fp8, kBN))
    return cudaErrorNotSupported;
  a.ctas = ctas;
  a.shape.r_shift = r_shift;
  a.shape.bn_shift = 6;
  a.shape.lead = 3;  // 64 ragged requests over e4m3: 42.6 us with 2 tiles' worth, 38.4 with 3, 39.6 with 6
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr;
  attention_config(&cfg, &attr, ctas, kThreads, C::kSmem, s);
  e = cudaLaunchKernelEx(&cfg, kernel, a, kmap, vmap);
  if constexpr (kPrefix<A>) return e;
  else return e != cudaSuccess ? e : launch_combine(a, D, s);
}
template <int D, int MT, bool FP8, class A>
cudaError_t launch_mma(const A& a, cudaStream_t s) {
  static std::atomic<int> ready[kMaxDevices];
  return launch_ring<Cfg<D, MT, FP8>>(attn_mma_kernel<D, MT, FP8, A>, ready, a, D, FP8, MT == 1 ? 4 : (MT == 2 ? 5 : 6), s);
}
template <int D, bool FP8, class A>
cudaError_t launch_row8(const A& a, cudaStream_t s) {
  static std::atomic<int> ready[kMaxDevices];
  return launch_ring<Cfg8<D, FP8>>(attn_row8_kernel<D, FP8, A>, ready, a, D, FP8, 3, s);
}

}  // namespace
}  // namespace lowbit
