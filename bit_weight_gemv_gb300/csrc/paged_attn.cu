// Attention of new tokens over a paged key/value cache, one pass over the keys:
//   per query row   s_j = scale * q . k_j;  m = max_j s_j;  l = sum_j exp(s_j - m);
//                   o = sum_j exp(s_j - m) v_j;   out = o / l,   lse = m + log l,
// with (m, l, o) of any two sets of keys joined by m = max(m1, m2), l = l1 e^(m1-m) + l2 e^(m2-m)
// and o likewise -- so a tile of keys is folded in at a time, and a long axis is split freely.
//
// attn_mma_kernel works on the warp-level MMA (m16n8k16, fp32 accumulation).  A CTA of four
// warps holds 16 * MT query rows (the rows of one key/value head that share its keys) and takes
// key tiles of 64 through a ring of cp.async stages; with MT < 4 row groups the other warps
// take different keys of the tile and the CTA joins them at the end.  The grid is resident and
// the work is cut evenly over it (see paged.cuh); attn_combine_kernel joins items that were cut.
#include "common.cuh"
#include "paged.cuh"
#include "paged_attn.cuh"
#include "ptx.cuh"

#include <cuda_fp16.h>

namespace lowbit {
namespace {

using namespace ptx;

constexpr int kThreads = 128;
constexpr int kJoinThreads = 512;
constexpr int kBN = 64;  // keys per tile
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool real) {
  const int n = real ? 16 : 0;  // the rest of the 16 bytes is written as zeros
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
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
// Two e4m3 codes (the low 16 bits) as two fp16 values: exact.
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t w) {
  uint32_t d;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(d) : "r"(w));
  return d;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
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
  static constexpr int kHalf = kBN * kRowBytes;        // one tile's keys (or values)
  static constexpr int kStage = 2 * kHalf;
  static constexpr int kStages = kStage >= 65536 ? 3 : (kStage >= 32768 ? 3 : 4);
  static constexpr int kSteps = D / 16;
  static constexpr bool kQShared = D > 128;            // query fragments in shared memory
  static constexpr int kQBytes = kQShared ? MT * kSteps * 512 : 0;
  static constexpr int kSmem = kStages * kStage + kQBytes;
  static constexpr int kOut = kWarpsK * 16 * MT * (D + 4) * 4;  // joining buffer (reuses the ring)
  static_assert(kOut <= kStages * kStage, "joining buffer");
};

// Byte offset of 16-byte chunk c of row r of a tile: the chunk index is XORed with a function of
// the row that takes 8 different values over 8 rows (128-byte rows and longer), so ldmatrix's
// 8 rows and the 16-byte loads of two rows' halves both meet every bank once.
template <int RB>
__device__ __forceinline__ uint32_t chunk_off(int r, int c) {
  const int x = RB >= 128 ? (((r & 1) << 2) | ((r >> 1) & 3)) : ((r >> 1) & 3);
  return (uint32_t)(r * RB + ((c ^ x) << 4));
}

template <int D, int MT, bool FP8>
__global__ void __launch_bounds__(kThreads, (Cfg<D, MT, FP8>::kSmem <= 110 * 1024 ? 2 : 1))
attn_mma_kernel(const AttnArgs a) {
  using C = Cfg<D, MT, FP8>;
  constexpr int RB = C::kRowBytes, S = C::kStages;
  constexpr int kNT = 2 * MT;       // 8-key tiles per warp
  constexpr int kDT = D / 8;        // 8-dim tiles
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ Plan plan;
  __shared__ float s_ml[4][16][2];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  const int wr = warp / C::kWarpsK, wk = warp % C::kWarpsK;  // row group, key group
  const uint32_t ring = smem_addr(smem);
  const PagedArgs& p = a.p;

  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  make_plan<kThreads>(a, plan, blockIdx.x);
  __syncthreads();

  if (plan.begin >= plan.end) return;
  Walk it = walk_start(a, plan);
  int left = (int)(plan.end - plan.begin);
  bool first = true;
  for (;;) {
    const Request q = it.q;
    const int b = it.b;
    const int kt0 = it.tile, kt1 = kt0 + walk_take(it, left);
    if (kt1 == kt0) return;
    const Span span = it.span;
    const int base_key = span.lo / kBN * kBN;
    const int r0 = it.qt * C::kRows;
    const int rows = q.n * a.shape.G;  // query rows of the request for this head

    // ---- this warp's two row slots per lane: g and g + 8 of its 16 rows
    int jlo[2], jhi[2];
    long long qrow[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = r0 + wr * 16 + g + 8 * i;
      const int tok = r / a.shape.G;
      const bool in = r < rows;
      const int pos = q.kv - q.n + tok;
      jhi[i] = in ? (a.shape.causal ? min(q.kv, pos + 1) : q.kv) : 0;
      jlo[i] = a.shape.window ? max(0, pos - a.shape.window + 1) : 0;
      qrow[i] = in ? (long long)(q.row0 + tok) * a.Hq + it.h * a.shape.G + (r - tok * a.shape.G) : -1;
    }
    // keys that every row of the CTA's tile sees need no mask
    const int last_row = min(r0 + C::kRows, rows) - 1;
    const int all_lo = a.shape.window ? max(0, q.kv - q.n + last_row / a.shape.G - a.shape.window + 1) : 0;
    const int all_hi = a.shape.causal ? min(q.kv, q.kv - q.n + r0 / a.shape.G + 1) : q.kv;

    // ---- query fragments; with an e4m3 cache the row is scaled by a power of two into fp16
    uint32_t qf[C::kQShared ? 1 : C::kSteps][4];
    float coef[2];  // exponent per unit of the raw product, in powers of two
    {
      const float ks = FP8 && p.k_scale ? __ldg(p.k_scale + it.h) : 1.0f;
      float scale2 = a.scale * ks * kLog2e;
      const uint16_t* src[2];
      float up[2] = {1.0f, 1.0f};
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = r0 + wr * 16 + g + 8 * i;
        const int tok = r / a.shape.G;
        src[i] = a.q + (long long)(q.row0 + tok) * a.q_stride + (long long)(it.h * a.shape.G + r - tok * a.shape.G) * D;
        coef[i] = scale2;
        if (FP8) {
          float m = 0.0f;
          if (qrow[i] >= 0)
            for (int d = t * 8; d < D; d += 32) {
              const uint4 v = *reinterpret_cast<const uint4*>(src[i] + d);
              const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
              for (int e = 0; e < 4; ++e)
                m = fmaxf(m, fmaxf(fabsf(__uint_as_float(u[e] << 16)), fabsf(__uint_as_float(u[e] & 0xFFFF0000u))));
            }
          m = fmaxf(m, __shfl_xor_sync(~0u, m, 1));
          m = fmaxf(m, __shfl_xor_sync(~0u, m, 2));
          // 2^-e with 2^e <= m < 2^(e+1): the row's largest becomes 1..2.  A row of zeros, or one
          // with an Inf or a NaN, stays as it is.
          const int e = (int)(__float_as_uint(m) >> 23) - 127;
          const int ee = (m > 0.0f && e < 128) ? max(-100, min(100, e)) : 0;
          up[i] = __uint_as_float((uint32_t)(127 - ee) << 23);
          coef[i] = scale2 * __uint_as_float((uint32_t)(127 + ee) << 23);
        }
      }
      uint4* qs = reinterpret_cast<uint4*>(smem + S * C::kStage) + (size_t)wr * C::kSteps * 32;
#pragma unroll
      for (int st = 0; st < C::kSteps; ++st) {
        uint32_t f[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int row = i & 1;
          // bf16: columns 16 st + 2t (+8); e4m3: the order in which a 16-byte load of a key's
          // row hands them out, 64 (st/4) + 16 t + 4 (st%4) (+2)
          const int col = FP8 ? 64 * (st / 4) + 16 * t + 4 * (st % 4) + (i >> 1) * 2 : 16 * st + 2 * t + (i >> 1) * 8;
          uint32_t v = qrow[row] >= 0 ? *reinterpret_cast<const uint32_t*>(src[row] + col) : 0u;
          if (FP8) v = pack2<true>(__uint_as_float(v << 16) * up[row], __uint_as_float(v & 0xFFFF0000u) * up[row]);
          f[i] = v;
        }
        if (C::kQShared) {
          if (wk == 0) qs[st * 32 + lane] = make_uint4(f[0], f[1], f[2], f[3]);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) qf[st][i] = f[i];
        }
      }
      if (C::kQShared) __syncthreads();
    }

    // ---- copy of key tile kt into stage st: rows outside the span become zeros
    auto load_tile = [&](int kt, int st) {
      constexpr int kChunks = RB / 16;
      constexpr int kIter = kBN * kChunks / kThreads;
      const uint32_t dst = ring + st * C::kStage;
      const long long head = (long long)it.h * p.head_stride;
#pragma unroll
      for (int i = 0; i < kIter; ++i) {
        const int idx = tid + i * kThreads;
        const int r = idx / kChunks, c = idx % kChunks;
        const int key = base_key + kt * kBN + r;
        bool real = key >= span.lo && key < span.hi;
        long long at = 0;
        if (real) {
          const int page = __ldg(p.table + (long long)b * p.table_stride + (key >> p.page_shift));
          real = page >= 0 && page < p.pages;
          if (!real) record_error(p.err, LOWBIT_ERR_INVALID_ARG);
          else at = (long long)page * p.page_stride + (long long)(key & p.page_mask) * p.token_stride + head + c * 16;
        }
        cp_async16(dst + chunk_off<RB>(r, c), p.k + at, real);
        cp_async16(dst + C::kHalf + chunk_off<RB>(r, c), p.v + at, real);
      }
    };

    float o[kDT][4];
#pragma unroll
    for (int i = 0; i < kDT; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[i][e] = 0.0f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};

#pragma unroll
    for (int s = 0; s < S - 1; ++s) {
      if (kt0 + s < kt1) load_tile(kt0 + s, s);
      cp_async_commit();
    }
    int stage = 0;
    for (int kt = kt0; kt < kt1; ++kt) {
      cp_async_wait<S - 2>();
      __syncthreads();
      {
        const int ns = stage == 0 ? S - 1 : stage - 1;  // the stage that tile kt - 1 has left
        if (kt + S - 1 < kt1) load_tile(kt + S - 1, ns);
        cp_async_commit();
      }
      const uint32_t ks = ring + stage * C::kStage, vs = ks + C::kHalf;
      const int key0 = base_key + kt * kBN;
      const int wkey = wk * kNT * 8;  // this warp's keys inside the tile

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
              const uint4 v = reinterpret_cast<const uint4*>(smem + S * C::kStage)[((size_t)wr * C::kSteps + 4 * j + e) * 32 + lane];
              qa[e][0] = v.x, qa[e][1] = v.y, qa[e][2] = v.z, qa[e][3] = v.w;
            } else {
#pragma unroll
              for (int i = 0; i < 4; ++i) qa[e][i] = qf[C::kQShared ? 0 : 4 * j + e][i];
            }
          }
#pragma unroll
          for (int n = 0; n < kNT; ++n) {
            const uint4 kw = lds128(ks + chunk_off<RB>(wkey + n * 8 + g, 4 * j + t));
            const uint32_t ww[4] = {kw.x, kw.y, kw.z, kw.w};
#pragma unroll
            for (int e = 0; e < 4; ++e)
              mma16816<true>(sc[n], qa[e], e4m3x2_f16x2(ww[e]), e4m3x2_f16x2(ww[e] >> 16));
          }
        }
      } else {
#pragma unroll
        for (int st = 0; st < C::kSteps; ++st) {
          uint32_t qa[4];
          if (C::kQShared) {
            const uint4 v = reinterpret_cast<const uint4*>(smem + S * C::kStage)[((size_t)wr * C::kSteps + st) * 32 + lane];
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
          const int key = key0 + wkey + n * 8 + 2 * t + (e & 1);
          if (masked && (key < jlo[e >> 1] || key >= jhi[e >> 1])) sc[n][e] = -INFINITY;
          tm[e >> 1] = fmaxf(tm[e >> 1], sc[n][e]);
        }
      // fold the tile in
      float keep[2], base[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        tm[i] = fmaxf(tm[i], __shfl_xor_sync(~0u, tm[i], 1));
        tm[i] = fmaxf(tm[i], __shfl_xor_sync(~0u, tm[i], 2));
        const float mn = fmaxf(m[i], tm[i]);
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
        const int r = wkey + k2 * 16 + ((lane >> 3) & 1) * 8 + (lane & 7);
        if (FP8) {
#pragma unroll
          for (int d = 0; d < D / 32; ++d) {
            uint32_t vb[4];
            ldsm4t(vb, vs + chunk_off<RB>(r, 2 * d + (lane >> 4)));
            // a word holds two keys' bytes of an even and an odd dim: [k0 d0, k0 d1, k1 d0, k1 d1]
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
              const uint32_t x0 = __byte_perm(vb[2 * hh], 0, 0x3120), x1 = __byte_perm(vb[2 * hh + 1], 0, 0x3120);
              mma16816<true>(o[4 * d + 2 * hh], pa[k2], e4m3x2_f16x2(x0), e4m3x2_f16x2(x1));
              mma16816<true>(o[4 * d + 2 * hh + 1], pa[k2], e4m3x2_f16x2(x0 >> 16), e4m3x2_f16x2(x1 >> 16));
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
      stage = stage + 1 == S ? 0 : stage + 1;
    }
    cp_async_wait<0>();
    __syncthreads();  // every warp is done with the ring, which now takes the outputs

    // ---- join the warps of a row group and store
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      l[i] += __shfl_xor_sync(~0u, l[i], 1);
      l[i] += __shfl_xor_sync(~0u, l[i], 2);
      if (t == 0) {
        s_ml[warp][g + 8 * i][0] = m[i];
        s_ml[warp][g + 8 * i][1] = l[i];
      }
    }
    float* so = reinterpret_cast<float*>(smem) + (size_t)warp * 16 * (D + 4);
#pragma unroll
    for (int d = 0; d < kDT; ++d)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int row = g + 8 * (e >> 1);
        const int col = FP8 ? 16 * (d / 2) + 4 * t + 2 * (e & 1) + (d & 1) : 8 * d + 2 * t + (e & 1);
        so[row * (D + 4) + col] = o[d][e];
      }
    __syncthreads();
    const bool whole = kt0 == 0 && kt1 == it.tiles;
    const long long slot = 2LL * blockIdx.x + (first ? 0 : 1);
    const float vscale = FP8 && p.v_scale ? __ldg(p.v_scale + it.h) : 1.0f;
    constexpr int kQuads = D / 4;
    for (int idx = tid; idx < C::kRows * kQuads; idx += kThreads) {
      const int row = idx / kQuads, c = (idx % kQuads) * 4;
      const int r = r0 + row;
      if (r >= rows) break;
      const int wbase = (row >> 4) * C::kWarpsK, lr = row & 15;
      float mm = -INFINITY;
#pragma unroll
      for (int k = 0; k < C::kWarpsK; ++k) mm = fmaxf(mm, s_ml[wbase + k][lr][0]);
      float ll = 0.0f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int k = 0; k < C::kWarpsK; ++k) {
        const float f = mm == -INFINITY ? 0.0f : ex2(s_ml[wbase + k][lr][0] - mm);
        ll += f * s_ml[wbase + k][lr][1];
        const float4 v = *reinterpret_cast<const float4*>(reinterpret_cast<float*>(smem) + (size_t)((wbase + k) * 16 + lr) * (D + 4) + c);
        acc.x += f * v.x, acc.y += f * v.y, acc.z += f * v.z, acc.w += f * v.w;
      }
      if (whole) {
        const int tok = r / a.shape.G;
        store_row(a, (long long)(q.row0 + tok) * a.Hq + it.h * a.shape.G + (r - tok * a.shape.G), D, c, acc, mm, ll, vscale);
      } else {
        store_piece(a, slot, C::kRows, D, row, c, acc, mm, ll);
      }
    }
    __syncthreads();  // the ring and s_ml are free again
    first = false;
    if (left <= 0 || !walk_next(a, it)) return;
  }
}

// Items that the cuts went through: blocks (j, *) look at cut j.  The blocks of one item's cuts
// share its rows, so the work of joining spreads over as many blocks as there are pieces, times
// gridDim.y.  A warp takes
// a row: its lanes hold the pieces' (maximum, sum) 32 at a time, so the weights cost one round
// trip, and then one part of the row each, whose loads do not wait for one another.
template <int D>
__global__ void __launch_bounds__(kJoinThreads) attn_combine_kernel(const AttnArgs a) {
  __shared__ Plan plan;
  // the schedule reads the batch alone, which no kernel since the attention's start has written
  make_plan<kJoinThreads>(a, plan, blockIdx.x + 1);
  __syncthreads();
  Walk it;
  bool cut = plan.begin < plan.end;
  if (cut) {
    it = walk_start(a, plan);
    cut = it.tile > 0;  // else the cut fell between two items, or inside a lead
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (!cut) return;
  const long long tiles_at = plan.begin - it.tile;           // where the item's tiles begin
  const long long from = tiles_at - a.shape.lead;            // and its lead
  const long long c0 = quotient(tiles_at, plan.chunk);       // CTAs with a piece: c0..c0 + n
  const int n = (int)(quotient(tiles_at + it.tiles - 1, plan.chunk) - c0);
  const int shares = n * gridDim.y, mine = (int)(blockIdx.x + 1 - (c0 + 1)) * gridDim.y + blockIdx.y;
  const long long slot0 = 2 * c0 + (from > c0 * plan.chunk ? 1 : 0);
  const int G = a.shape.G, R = 1 << a.shape.r_shift, r0 = it.qt << a.shape.r_shift;
  const int rows = min(R, it.q.n * G - r0);
  const int ra = (int)((long long)rows * mine / shares), rb = (int)((long long)rows * (mine + 1) / shares);
  const float vscale = a.p.v_scale ? __ldg(a.p.v_scale + it.h) : 1.0f;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kPart = D >= 128 ? 4 : 2, kParts = D / (32 * kPart);
  for (int row = ra + warp; row < rb; row += kJoinThreads / 32) {
    float m = -INFINITY;
    for (int i = lane; i <= n; i += 32) m = fmaxf(m, a.piece_ml[(i ? 2 * (c0 + i) : slot0) * R + row].x);
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
    float l = 0.0f, acc[kParts][kPart] = {};
    for (int i0 = 0; i0 <= n; i0 += 32) {
      float f = 0.0f;
      if (i0 + lane <= n) {
        const int i = i0 + lane;
        const float2 ml = a.piece_ml[(i ? 2 * (c0 + i) : slot0) * R + row];
        f = m == -INFINITY ? 0.0f : ex2(ml.x - m);
        l += f * ml.y;
      }
      const int k1 = min(32, n + 1 - i0);
#pragma unroll 8
      for (int k = 0; k < k1; ++k) {
        const float fk = __shfl_sync(~0u, f, k);
        const long long slot = i0 + k ? 2 * (c0 + i0 + k) : slot0;
        const float* src = a.piece_o + (slot * R + row) * D + lane * kPart;
#pragma unroll
        for (int q = 0; q < kParts; ++q) {
          float v[kPart];
          if (kPart == 4) *reinterpret_cast<float4*>(v) = *reinterpret_cast<const float4*>(src + q * 128);
          else *reinterpret_cast<float2*>(v) = *reinterpret_cast<const float2*>(src);
#pragma unroll
          for (int e = 0; e < kPart; ++e) acc[q][e] += fk * v[e];
        }
      }
    }
    for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(~0u, l, o);
    const int r = r0 + row, tok = r / G;
    const long long orow = (long long)(it.q.row0 + tok) * a.Hq + it.h * G + (r - tok * G);
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
}

template <int D, int MT, bool FP8>
cudaError_t launch_mma(AttnArgs a, cudaStream_t s) {
  using C = Cfg<D, MT, FP8>;
  static std::atomic<int> ready[kMaxDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  int ctas = ready[dev].load(std::memory_order_relaxed);
  if (!ctas) {
    e = cudaFuncSetAttribute(attn_mma_kernel<D, MT, FP8>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    int sms = 0, per = 0;
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, attn_mma_kernel<D, MT, FP8>, kThreads, C::kSmem);
    if (e != cudaSuccess) return e;
    ctas = std::max(1, std::min(sms * per, kMaxPieceRows / 2 / C::kRows));
    ready[dev].store(ctas, std::memory_order_relaxed);
  }
  a.ctas = ctas;
  a.shape.r_shift = MT == 1 ? 4 : (MT == 2 ? 5 : 6);
  a.shape.bn_shift = 6;
  a.shape.lead = tune("LEAD", 4);
  a.min_chunk = tune("MINC", 1);
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr;
  attention_config(&cfg, &attr, ctas, kThreads, C::kSmem, s);
  e = cudaLaunchKernelEx(&cfg, attn_mma_kernel<D, MT, FP8>, a);
  return e != cudaSuccess ? e : launch_combine(a, D, s);
}

template <int D, bool FP8>
cudaError_t launch_rows(const AttnArgs& a, cudaStream_t s) {
  // Rows that share a request's keys, on average: the host knows the totals only.
  const long long rows = ((long long)a.p.T * a.shape.G + a.p.B - 1) / a.p.B;
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

cudaError_t launch_combine(const AttnArgs& a, int D, cudaStream_t s) {
  if (a.ctas < 2) return cudaSuccess;
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr;
  attention_config(&cfg, &attr, a.ctas - 1, kJoinThreads, 0, s);
  cfg.gridDim.y = a.shape.r_shift > 6 ? 1u << (a.shape.r_shift - 6) : 1;  // 64 rows of an item each
  if (D == 64) return cudaLaunchKernelEx(&cfg, attn_combine_kernel<64>, a);
  if (D == 128) return cudaLaunchKernelEx(&cfg, attn_combine_kernel<128>, a);
  return cudaLaunchKernelEx(&cfg, attn_combine_kernel<256>, a);
}

cudaError_t launch_attention_mma(const AttnArgs& a, int D, bool fp8, cudaStream_t s) {
  if (D == 64) return fp8 ? launch_rows<64, true>(a, s) : launch_rows<64, false>(a, s);
  if (D == 128) return fp8 ? launch_rows<128, true>(a, s) : launch_rows<128, false>(a, s);
  return fp8 ? launch_rows<256, true>(a, s) : launch_rows<256, false>(a, s);
}

}  // namespace lowbit

using namespace lowbit;

extern "C" {

size_t lowbit_paged_attention_workspace_bytes(int T, int B, int Hq, int Hk, int D) {
  if (T < 0 || T > kMaxTokens || B < 1 || B > kMaxBatch || Hk < 1 || Hk > 4096 || Hq < 1 || Hq > 65536 ||
      Hq % Hk || (D != 64 && D != 128 && D != 256))
    return 0;
  return (size_t)kMaxPieceRows * (size_t)(D + 2) * sizeof(float);
}

lowbit_status lowbit_paged_attention(const uint16_t* q, int64_t q_stride, int Hq,
                                     const lowbit_paged_batch* batch, const lowbit_paged_cache* cache,
                                     float scale, int causal, int window, uint16_t* out, float* lse,
                                     void* workspace, size_t ws_bytes, void* stream) {
  AttnArgs a = {};
  const lowbit_status st = make_paged_args(batch, cache, &a.p);
  if (st != LOWBIT_OK) return st;
  if (a.p.T == 0) return LOWBIT_OK;  // the token arrays may then be null
  if (!q || !out || !(scale == scale)) return LOWBIT_ERR_INVALID_ARG;
  const int D = cache->head_dim;
  if (Hq < 1 || Hq > 65536 || Hq % cache->heads || window < 0 || q_stride < (int64_t)Hq * D ||
      (long long)a.p.T * (Hq / cache->heads) > 0x7FFFFF00LL ||
      ((long long)a.p.width << a.p.page_shift) > 0x7FFFFF00LL)
    return LOWBIT_ERR_SHAPE;
  if (!workspace || ws_bytes < lowbit_paged_attention_workspace_bytes(a.p.T, a.p.B, Hq, cache->heads, D))
    return LOWBIT_ERR_WORKSPACE;
  if (((uintptr_t)q | (uintptr_t)out | (uintptr_t)workspace) & 15 || q_stride % 8 || ((uintptr_t)lse & 3))
    return LOWBIT_ERR_ALIGN;
  a.p.err = device_error_word();
  if (!a.p.err) return LOWBIT_ERR_CUDA;
  a.shape = ItemShape{Hq / cache->heads, 0, 0, 0, causal != 0, window};
  a.q = q;
  a.q_stride = q_stride;
  a.Hq = Hq;
  a.scale = scale;
  a.out = out;
  a.lse = lse;
  a.piece_o = static_cast<float*>(workspace);
  a.piece_ml = reinterpret_cast<float2*>(a.piece_o + (size_t)kMaxPieceRows * D);
  const bool fp8 = cache->dtype == LOWBIT_CACHE_E4M3;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  // Rows that share a request's keys, on average: the host knows the totals only.
  const long long rows = ((long long)a.p.T * a.shape.G + a.p.B - 1) / a.p.B;
  const cudaError_t e = rows > 32 && attention_tc_fits(a, D, fp8) ? launch_attention_tc(a, D, rows > 128, s)
                                                                 : launch_attention_mma(a, D, fp8, s);
  return e == cudaSuccess ? LOWBIT_OK : LOWBIT_ERR_CUDA;
}

}  // extern "C"
