// Attention over a paged cache on the fifth-generation tensor cores, for many query rows per
// key/value head (prompt chunks, verify blocks of grouped heads).  Same mathematics and schedule
// as attn_mma_kernel (see paged_attn.cu and paged.cuh).
//
// One CTA per SM, two "slots" of 128 query rows that keep the tensor pipe busy in turn:
//   warps 0-3, 4-7 -- softmax of slot 0 and 1, one thread per row: read the row's 128 scores from
//       tensor memory, fold them into (m, l) and write the weights back as bf16 over the scores,
//       where they are the A operand of the product with V;
//   warp 8 -- copies: K and V tiles of 128 keys by TMA, one box per page and 64-element half;
//   warp 9 -- issues the MMAs: S = Q K^T (both in shared memory) and O += P V (P in tensor memory,
//       V as it lies in the cache, keys along the reduction);
//   warps 10 and 11 -- the queries of the next item;
//   warps 12-15, over an e4m3 cache only -- tiles into 16 bits on their way from the copies to the MMAs:
//       keys as bf16, which the queries are, values as fp16, which the weights then are; both exact.
// PAIR: the slots hold different rows and share every tile (256 rows per item).  Otherwise both
// slots hold the same 128 rows and take alternate tiles; their (m, l, O) are joined at the end.
// O stays in tensor memory; it is rescaled only when a row's maximum has grown by more than 2^8
// since the value the weights refer to, so most tiles never touch it (weights up to 2^8 round to
// bf16 with the same relative error, and sums are fp32).  Over an e4m3 cache the weights are fp16, which ends
// at 2^16 and has no values below 2^-24: they refer to 2^-7 of the maximum, so the largest is 2^7 to 2^15, and
// a weight becomes zero only below 2^-32 of it (24 draft blocks 54.0 us; with rescaling from a growth of 2^3 on
// and 2^-12 of the maximum 56.9).  Scores past 2^20 are rounded to fp32 before the reference
// is taken off (the difference of a fused product and a rounded one would be an eighth and more), and
// refer to the largest itself.
//
// Bound: the tensor pipe, shared memory and the issuing thread together.  A prompt chunk of 4,001
// tokens over 16,331 keys (32 heads on 8 of 128, causal, 939 GFLOP): 664 to 675 us call after call under
// the power limit, 1,400 TFLOP/s, 81% of a large library product there; 638 us in bursts, 1,472 TFLOP/s,
// 77%.  S = Q K^T reads both operands from shared memory, and an MMA comes every 81 cycles for 64 of
// work.  Few rows are bound by the chain of a tile (scores, softmax, product, 3 us on two slots in turn):
// one request's 64 rows over 32,765 keys 34.6 us, 134 MB, 3.9 TB/s; 24 ragged requests of 64 rows 51.8 us,
// 246 MB, 4.7 TB/s.  Over e4m3 caches the conversion takes issue slots from the softmax: 1,200 tokens over
// 4,000 keys 91 us (80 in bf16, 250 on the warp-level MMA); 64 rows over 32,765 keys 34.0 us (54 on the
// warp-level MMA).
#include <cuda_fp16.h>

#include <type_traits>

#include "common.cuh"
#include "paged.cuh"
#include "paged_attn.cuh"
#include "ptx.cuh"

namespace lowbit {
namespace {

using namespace ptx;

constexpr int kTcBN = 128;
constexpr int kLoadWarp = 8, kMmaWarp = 9, kConvertWarp = 12;
constexpr float kGrow = 8.0f;

template <int D, bool PAIR, bool FP8>
struct Tc {
  static constexpr int kThreads = FP8 ? 512 : 384;
  static constexpr int kTile = 128 * D * 2;   // 128 rows of Q, K or V
  static constexpr int kHalves = D / 64;      // 64-element (128-byte) halves of a row
  // e4m3: tiles arrive in a ring of their own
  static constexpr int kRaw = 128 * D, kRawStages = !FP8 ? 0 : (D == 64 ? 6 : (PAIR ? 2 : 3));
  static constexpr int kStages = D == 64 ? (FP8 ? 6 : 8) : (FP8 ? 4 : 5);
  static constexpr int kQ = PAIR ? 2 * kTile : kTile + 2048;  // queries; or one tile and the slots' statistics
  static constexpr int kSmem = 1024 + kQ + kStages * kTile + kRawStages * kRaw;
  static constexpr uint32_t kS = 0, kO = 256;  // tensor memory columns: S (and P) of slot s at 128 s,
};                                             // O at 256 + D s

struct TcShared {
  uint64_t kv_full[8], kv_empty[8], raw_full[8], raw_empty[8];
  uint64_t q_full, q_free, s_full[2], p_full[2], o_full[2];
  uint64_t joined, left;  // both slots' statistics are written; both slots have read both O
  uint32_t tmem;
};

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float* r) {
  uint32_t* u = reinterpret_cast<uint32_t*>(r);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]),
        "=r"(u[8]), "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15]),
        "=r"(u[16]), "=r"(u[17]), "=r"(u[18]), "=r"(u[19]), "=r"(u[20]), "=r"(u[21]), "=r"(u[22]), "=r"(u[23]),
        "=r"(u[24]), "=r"(u[25]), "=r"(u[26]), "=r"(u[27]), "=r"(u[28]), "=r"(u[29]), "=r"(u[30]), "=r"(u[31])
      : "r"(taddr)
      : "memory");
}
// D[tmem] (+)= A x B^T with A in shared memory, or in tensor memory, issued by one thread.  Matrix
// descriptors are passed as their low words beside constant high words: the thread that issues has
// 64 cycles per MMA (128 x 128 x 16), and building 64-bit descriptors for each took it 90 to 110.
__device__ __forceinline__ void umma_ss(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t hi, uint32_t idesc,
                                        uint32_t accumulate, uint32_t issue) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 a, b;\n\t"
      "setp.ne.b32 p, %5, 0;\n\tsetp.ne.b32 q, %6, 0;\n\tmov.b64 a, {%1, %3};\n\tmov.b64 b, {%2, %3};\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n\t}" ::"r"(d_tmem),
      "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "r"(accumulate), "r"(issue)
      : "memory");
}
__device__ __forceinline__ void umma_ts_lo(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo, uint32_t hi, uint32_t idesc,
                                           uint32_t accumulate, uint32_t issue) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 b;\n\t"
      "setp.ne.b32 p, %5, 0;\n\tsetp.ne.b32 q, %6, 0;\n\tmov.b64 b, {%2, %3};\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "r"(b_lo), "r"(hi), "r"(idesc), "r"(accumulate), "r"(issue)
      : "memory");
}
// Both kinds of descriptor have 128-byte rows under the 128-byte swizzle, in 8-row groups 1024
// bytes apart.  The low word holds the address and, where the reduction runs over rows (V), the
// distance to the next 64 elements of the other dimension.
constexpr uint32_t kDescHi = (1024 >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t half_bytes) {
  return ((saddr & 0x3FFFFu) >> 4) | ((half_bytes >> 4) << 16);
}
__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
// Two e4m3 codes as fp16, and two fp16 values as bf16: both exact, since e4m3 has four bits of
// significand and an exponent that either type holds.
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t two) {
  uint32_t d;
  asm("{\n\t.reg .b16 x;\n\tcvt.u16.u32 x, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, x;\n\t}" : "=r"(d) : "r"(two));
  return d;
}
__device__ __forceinline__ uint32_t f16x2_bf16x2(uint32_t h) {
  const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&h));
  return pack_bf16x2(x.x, x.y);
}
// 32 bytes: at once where addresses allow (`wide`), since each thread has a row of its own and a
// whole sector per store halves their cost; else as two stores of 16.
__device__ __forceinline__ void st_global_32(void* at, const uint32_t* w, bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(at), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    reinterpret_cast<uint4*>(at)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    reinterpret_cast<uint4*>(at)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}
// Two fp32 operations at once, each rounded as the single one.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)), "l"(reinterpret_cast<uint64_t&>(c)));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
  return d;
}

// A wait that remembers failure: once one has given up, the role leaves its loops.
#define WAIT_OR(bar, parity, what)                 \
  if (!mbar_wait(smem_addr(&(bar)), (parity))) {   \
    record_error(p.err, LOWBIT_ERR_TIMEOUT);       \
    what;                                          \
  }

template <int D, bool PAIR, bool FP8>
__global__ void __launch_bounds__(FP8 ? 512 : 384, 1)
attn_tc_kernel(const __grid_constant__ AttnArgs a, const __grid_constant__ CUtensorMap kmap,
               const __grid_constant__ CUtensorMap vmap) {
  using C = Tc<D, PAIR, FP8>;
  constexpr int S = C::kStages;
  constexpr int kRows = PAIR ? 256 : 128;
  extern __shared__ uint8_t raw[];
  __shared__ TcShared sh;
  const uint32_t base = (smem_addr(raw) + 1023u) & ~1023u;
  const uint32_t q_at = base, ring = base + C::kQ;
  float2* const ml = reinterpret_cast<float2*>(raw + (base - smem_addr(raw)) + C::kTile);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const PagedArgs& p = a.p;

  if (tid == 0) {
    for (int i = 0; i < S; ++i) mbar_init(smem_addr(&sh.kv_full[i]), FP8 ? 128 : 1), mbar_init(smem_addr(&sh.kv_empty[i]), 1);
    for (int i = 0; i < C::kRawStages; ++i) mbar_init(smem_addr(&sh.raw_full[i]), 1), mbar_init(smem_addr(&sh.raw_empty[i]), 128);
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_addr(&sh.s_full[i]), 1);
      mbar_init(smem_addr(&sh.p_full[i]), 128);
      mbar_init(smem_addr(&sh.o_full[i]), 1);
    }
    mbar_init(smem_addr(&sh.q_full), 64);
    mbar_init(smem_addr(&sh.q_free), 1);
    mbar_init(smem_addr(&sh.joined), 256);
    mbar_init(smem_addr(&sh.left), 256);
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_addr(&sh.tmem), 512);
    tmem_relinquish();
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  Walk it;
  Share share;
  const bool busy = start_walk<C::kThreads>(a, blockIdx.x, it, share);
  if (tid == 0) say_cut(a, blockIdx.x, nullptr, 0, 1, 0);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;  // an allocation of all 512 columns starts at 0, which the MMA warp builds on
  const int G = a.shape.G;

  if (busy) {
    int left = share.left;

    // Registers: 384 threads launch with 168 each (64,512); 256 softmax threads take 208 and the
    // other 128 keep 80 (63,488).  512 threads launch with 128 each (65,536): 200 and 56, or 168 and 88,
    // are as many.
    constexpr int kSide = !FP8 ? 80 : (PAIR ? 56 : 88), kSoftmax = !FP8 ? 208 : (PAIR ? 200 : 168);
    // The tiles of the share, in the order in which the MMA warp takes them: tile(key tile, is V).
    auto in_order = [&](const bool& ok, auto&& tile) {
      for (;;) {
        const int kt0 = it.tile, n = walk_take(it, left);
        if (n == 0) break;
        tile(kt0, false);
        if (!PAIR && ok && n > 1) tile(kt0 + 1, false);
        for (int j = 0; j < n && ok; ++j) {
          tile(kt0 + j, true);
          const int next = j + (PAIR ? 1 : 2);
          if (next < n && ok) tile(kt0 + next, false);
        }
        if (!ok || left <= 0 || !walk_next(a, it)) break;
      }
    };
    if (warp == kLoadWarp) {
      // ------------------------------------------------------------------ copies
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kSide));
      constexpr int kDepth = FP8 ? C::kRawStages : S, kBytes = FP8 ? C::kRaw : C::kTile;
      uint64_t* const full = FP8 ? sh.raw_full : sh.kv_full;
      uint64_t* const empty = FP8 ? sh.raw_empty : sh.kv_empty;
      const uint32_t dst = FP8 ? ring + S * C::kTile : ring;
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      int filled = 0;  // loads issued, up to kDepth
      const int box = min(p.page_mask + 1, kTcBN), boxes = kTcBN / box;  // keys per box
      in_order(ok, [&](int kt, bool value) {
        const CUtensorMap* map = value ? &vmap : &kmap;
        WAIT_OR(empty[stage], phase ^ 1, { ok = false; return; });
        const int key0 = it.span.lo / kTcBN * kTcBN + kt * kTcBN + lane * box;
        const bool mine = lane < boxes && key0 < it.span.hi && key0 + box > it.span.lo;
        int page = 0;
        if (mine) {
          page = __ldg(p.table + (long long)it.b * p.table_stride + (key0 >> p.page_shift));
          // a page outside the cache is outside the tensor map: the copy fills zeros
          if (page < 0 || page >= p.pages) record_error(p.err, LOWBIT_ERR_INVALID_ARG), page = -1;
        }
        const int n = __popc(__ballot_sync(~0u, mine));
        const uint32_t bar = smem_addr(&full[stage]);
        if (lane == 0) mbar_arrive_expect_tx(bar, (uint32_t)(n * box * (kBytes / 128)));
        __syncwarp();
        if (mine) {
          if (FP8) {
            tma_load_4d(dst + stage * kBytes + lane * box * D, map, 0, key0 & p.page_mask, it.h, page, bar);
          } else {
#pragma unroll
            for (int h = 0; h < C::kHalves; ++h)
              tma_load_4d(dst + stage * kBytes + h * (kTcBN * 128) + lane * box * 128, map, 64 * h,
                          key0 & p.page_mask, it.h, page, bar);
          }
        }
        if (++stage == kDepth) stage = 0, phase ^= 1;
        if (filled < kDepth) ++filled;
      });
      // Leave only when no copy is in flight and every release has arrived.
      for (int i = 0; i < filled; ++i) {
        if (--stage < 0) stage = kDepth - 1, phase ^= 1;
        mbar_wait(smem_addr(&full[stage]), phase);
        if (ok) WAIT_OR(empty[stage], phase, ok = false);
      }
    } else if (FP8 && warp >= kConvertWarp) {
      // ------------------------------------------------------------------ e4m3 to 16 bits
      // A thread takes a row: K becomes bf16, as the queries are, and V fp16, as the weights are over
      // such a cache, in the layout that TMA gives a 16-bit tile.
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kSide));
      const int row = tid - 32 * kConvertWarp;
      int stage = 0, raw_stage = 0, filled = 0;
      uint32_t phase = 0, raw_phase = 0;
      bool ok = true;
      in_order(ok, [&](int, bool value) {
        WAIT_OR(sh.raw_full[raw_stage], raw_phase, { ok = false; return; });
        WAIT_OR(sh.kv_empty[stage], phase ^ 1, { ok = false; return; });
        const uint32_t from = ring + S * C::kTile + raw_stage * C::kRaw + row * D;
        const uint32_t to = ring + stage * C::kTile + row * 128;
        const int from_turn = D == 128 ? row & 7 : (row >> 1) & 3;
        // 3,000 tokens (PAIR): 118 us with one, 120 with two, 127 with four; 24 draft blocks 53.1 with
        // four, 57.1 with eight
#pragma unroll(PAIR ? 1 : 4)
        for (int c = 0; c < D / 16; ++c) {
          uint32_t w[4], x[8];
          asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                       : "r"(from + ((c ^ from_turn) << 4)));
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] = e4m3x2_f16x2(i & 1 ? w[i / 2] >> 16 : w[i / 2]);
          if (!value) {
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = f16x2_bf16x2(x[i]);
          }
#pragma unroll
          for (int h = 0; h < 2; ++h)
            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(
                             to + (c / 4) * (128 * 128) + (((((c & 3) * 2 + h)) ^ (row & 7)) << 4)),
                         "r"(x[4 * h]), "r"(x[4 * h + 1]), "r"(x[4 * h + 2]), "r"(x[4 * h + 3])
                         : "memory");
        }
        fence_proxy_async_smem();
        mbar_arrive(smem_addr(&sh.kv_full[stage]));
        mbar_arrive(smem_addr(&sh.raw_empty[raw_stage]));
        if (++stage == S) stage = 0, phase ^= 1;
        if (++raw_stage == C::kRawStages) raw_stage = 0, raw_phase ^= 1;
        if (filled < S) ++filled;
      });
      for (int i = 0; i < filled; ++i) {  // every release has arrived
        if (--stage < 0) stage = S - 1, phase ^= 1;
        if (ok) WAIT_OR(sh.kv_empty[stage], phase, ok = false);
      }
    } else if (warp == kMmaWarp) {
      // ------------------------------------------------------------------ MMA issue
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kSide));
      constexpr uint32_t kIdQK = umma_idesc_bf16(128, 128);
      // B with rows along the reduction; operand formats bf16 (1), or f16 (0)
      constexpr uint32_t kIdPV = (umma_idesc_bf16(128, D) & (FP8 ? ~((1u << 7) | (1u << 10)) : ~0u)) | (1u << 16);
      int stage = 0;
      uint32_t phase = 0;
      uint32_t q_phase = 0, p_phase[2] = {0, 0};
      // low descriptor words of the queries, and of ring stage 0 as K and as V
      const uint32_t q_lo = desc_lo(q_at, 16), k_lo = desc_lo(ring, 16), v_lo = desc_lo(ring, kTcBN * 128);
      const uint32_t one = lane == 0;
      auto qk = [&](int slot, int st) {
        st = __shfl_sync(~0u, st, 0);  // uniform for the compiler too
        const uint32_t qa = q_lo + (PAIR ? slot * (C::kTile >> 4) : 0), kb = k_lo + st * (C::kTile >> 4);
        const uint32_t d = C::kS + 128 * slot;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t off = ((k / 4) * (128 * 128) + (k % 4) * 32) >> 4;
          umma_ss(d, qa + off, kb + off, kDescHi, kIdQK, k > 0, one);
        }
        if (one) umma_commit(smem_addr(&sh.s_full[slot]));
        __syncwarp();
      };
      auto pv = [&](int slot, int st, bool add) {
        st = __shfl_sync(~0u, st, 0);
        const uint32_t vb = v_lo + st * (C::kTile >> 4);
        const uint32_t d = C::kO + D * slot, pa = C::kS + 128 * slot;
        umma_ts_lo(d, pa, vb, kDescHi, kIdPV, add, one);
#pragma unroll
        for (int k = 1; k < kTcBN / 16; ++k) umma_ts_lo(d, pa + 8 * k, vb + k * (2048 >> 4), kDescHi, kIdPV, 1, one);
        __syncwarp();
      };
      auto commit = [&](uint64_t& bar) {
        if (lane == 0) umma_commit(smem_addr(&bar));
        __syncwarp();
      };
      auto advance = [&]() {
        const int st = stage;
        if (++stage == S) stage = 0, phase ^= 1;
        return st;
      };
      bool ok = true;
      for (;;) {
        const int kt0 = it.tile, n = walk_take(it, left);
        if (n == 0) break;
        const int key_first = it.span.lo / kTcBN * kTcBN + kt0 * kTcBN;
        const int slots = PAIR && it.q.n * G - it.qt * kRows <= 128 ? 1 : 2;
        // Waits for the next K tile; returns its stage.
        auto next_tile = [&]() {
          WAIT_OR(sh.kv_full[stage], phase, ok = false);
          return advance();
        };
        // The V tile of keys key0..: rows outside the span (unwritten slots, stale buffers) become
        // zeros, since 0 * NaN would reach the sums.
        auto next_v = [&](int key0) {
          WAIT_OR(sh.kv_full[stage], phase, ok = false);
          if (ok && (key0 < it.span.lo || key0 + kTcBN > it.span.hi)) {
            const uint32_t vb = ring + stage * C::kTile;
            for (int i = lane; i < kTcBN * C::kHalves * 8; i += 32) {
              const int row = (i >> 3) & (kTcBN - 1), key = key0 + row;
              if (key < it.span.lo || key >= it.span.hi)
                asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(vb + i * 16), "r"(0) : "memory");
            }
            fence_proxy_async_smem();
            __syncwarp();
          }
          return advance();
        };
        WAIT_OR(sh.q_full, q_phase, ok = false);
        q_phase ^= 1;
        tc_fence_after();
        if (!ok) break;
        if constexpr (PAIR) {
          int sk = next_tile();
          if (!ok) break;
#pragma unroll
          for (int s = 0; s < 2; ++s)
            if (s < slots) qk(s, sk);
          if (n == 1) commit(sh.q_free);
          // Step j multiplies tile j's weights with its V and asks for the scores of tile j + 1.
          for (int j = 0; j < n && ok; ++j) {
            const int sv = next_v(key_first + j * kTcBN);
            const bool more = j + 1 < n;
            const bool k_ready = more && mbar_try_wait(smem_addr(&sh.kv_full[stage]), phase);
#pragma unroll
            for (int s = 0; s < 2; ++s) {
              if (s >= slots || !ok) break;
              WAIT_OR(sh.p_full[s], p_phase[s], { ok = false; break; });
              p_phase[s] ^= 1;
              tc_fence_after();
              pv(s, sv, j > 0);
              if (!more) {
                commit(sh.o_full[s]);
              } else {
                if (s == 0) {
                  if (!k_ready) WAIT_OR(sh.kv_full[stage], phase, { ok = false; break; });
                  sk = advance();
                }
                qk(s, sk);
                if (j + 2 == n && s + 1 == slots) commit(sh.q_free);
              }
            }
          }
        } else {
          for (int s = 0; s < min(n, 2) && ok; ++s) {
            const int st = next_tile();
            if (!ok) break;
            qk(s, st);
            commit(sh.kv_empty[st]);
          }
          if (ok && n <= 2) commit(sh.q_free);
          for (int j = 0; j < n && ok; ++j) {
            const int s = j & 1;
            const int sv = next_v(key_first + j * kTcBN);
            if (!ok) break;
            WAIT_OR(sh.p_full[s], p_phase[s], { ok = false; break; });
            p_phase[s] ^= 1;
            tc_fence_after();
            pv(s, sv, j > 1);
            commit(sh.kv_empty[sv]);
            if (j + 2 < n) {
              const int st = next_tile();
              if (!ok) break;
              qk(s, st);
              commit(sh.kv_empty[st]);
              if (j + 3 == n) commit(sh.q_free);
            } else {
              commit(sh.o_full[s]);
            }
          }
          if (ok && n == 1) commit(sh.o_full[1]);
        }
        if (!ok) break;
        if (left <= 0 || !walk_next(a, it)) break;
      }
      if (!ok) {  // nothing of this CTA may still be in flight when it leaves
        commit(sh.s_full[0]);
        const long long t0 = clock64();
        while (clock64() - t0 < 20000000LL) {}
      }
    } else if (warp > kMmaWarp) {
      // ------------------------------------------------------------------ queries
      // The item's rows into shared memory, swizzled as TMA would leave them, as soon as the last
      // scores of the item before are there: the copy then hides behind its last weights and its
      // way out (loaded at the item's start by the softmax warps, the rows took 10,000 cycles).
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kSide));
      uint32_t free_phase = 1;  // the place is free to begin with
      for (;;) {
        if (a.stall || walk_take(it, left) == 0) break;
        WAIT_OR(sh.q_free, free_phase, break);
        free_phase ^= 1;
        constexpr int kChunks = D / 8;
        const int r0 = it.qt * kRows, rows = min(kRows, it.q.n * G - r0);
        for (int i = tid - 32 * (kMmaWarp + 1); i < rows * kChunks; i += 64) {
          const int rr = i / kChunks, c = i % kChunks, r = r0 + rr, tok = token_of(a.shape, r);
          const uint16_t* src = a.q + (long long)(it.q.row0 + tok) * a.q_stride + (long long)(it.h * G + r - tok * G) * D + c * 8;
          const uint32_t dst = q_at + (rr >> 7) * C::kTile + (c / 8) * (128 * 128) + (rr & 127) * 128 + (((c & 7) ^ (rr & 7)) << 4);
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        fence_proxy_async_smem();
        mbar_arrive(smem_addr(&sh.q_full));
        if (left <= 0 || !walk_next(a, it)) break;
      }
    } else {
      // ------------------------------------------------------------------ softmax
      asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmax));
      const int slot = warp >> 2, row = (warp & 3) * 32 + lane, t128 = tid & 127;
      const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
      const uint32_t s_at = tmem + C::kS + 128 * slot + lanes;
      uint32_t s_phase = 0, o_phase = 0, j_phase = 0;
      int rel = 0;  // PAIR: ring stage that is released next
      bool first = true, ok = true;
      for (;;) {
        const int kt0 = it.tile, n = walk_take(it, left);
        if (n == 0) break;
        const float scale = FP8 && p.k_scale ? a.scale * __ldg(p.k_scale + it.h) : a.scale;
        const float vscale = FP8 && p.v_scale ? __ldg(p.v_scale + it.h) : 1.0f;
        // a scale of zero keeps masked scores at -inf
        const float coef = fmaxf(fabsf(scale) * 1.4426950408889634f, 1e-37f);
        const float signed_coef = copysignf(coef, scale);
        const int rows = it.q.n * G, r0 = it.qt * kRows;
        const int r_tile = r0 + (PAIR ? slot * 128 : 0);
        const bool active = r_tile < rows;
        // PAIR: a commit of the MMA thread costs the tensor pipe about 120 cycles, so the tiles are
        // not released by commits of their own: when the last active slot's scores of tile j have
        // come, K of tile j and V of tile j - 1 have been read.
        const bool frees = PAIR && t128 == 0 && (slot == 1 || rows - r0 <= 128);
        auto release = [&]() {
          if (frees) mbar_arrive(smem_addr(&sh.kv_empty[rel]));
          if (++rel == S) rel = 0;
        };
        const int key_first = it.span.lo / kTcBN * kTcBN + kt0 * kTcBN;

        // the keys this row sees
        const int r = r_tile + row, tok = token_of(a.shape, r);
        const bool in = r < rows;
        const int pos = it.q.kv - it.q.n + tok;
        const int jhi = in ? (a.shape.causal ? min(it.q.kv, pos + 1) : it.q.kv) : 0;
        const int jlo = first_key(a.shape, pos);
        const bool work = __any_sync(~0u, in);  // a warp without rows only keeps the pace

        constexpr float kLift = FP8 ? 7.0f : 0.0f;
        float m = -INFINITY, l = 0.0f;  // m: what the weights so far refer to
        float slack = kGrow + kLift;    // a maximum this far above m moves it
        // The scores in powers of two are s * sign * unit, the first product rounded and the second fused with
        // the subtraction of m: sign is 1 or -1, so that the largest stays the largest under a negative
        // scale, and unit is coef, until m of some row of the warp is past 2^20: then sign takes coef.
        float sign = copysignf(1.0f, scale), unit = coef;
        bool turned = scale < 0.0f;
        int steps = 0;
        if (active && ok) {
          for (int j = PAIR ? 0 : slot; j < n; j += PAIR ? 1 : 2, ++steps) {
            WAIT_OR(sh.s_full[slot], s_phase, { ok = false; break; });
            s_phase ^= 1;
            tc_fence_after();
            if (PAIR) {
              release();
              if (j > 0) release();
            }
            const int key0 = key_first + j * kTcBN;
            // the maximum grew: l and (past the slot's first tile) O follow the new reference
            auto refer = [&](float top, float* s) {
              const bool grow = top > m + slack;  // from -inf: any finite maximum
              if (__any_sync(~0u, grow)) {
                const bool far = __any_sync(~0u, in && far_score(fmaxf(m, top)));
                if (far != (slack == 0.0f)) {
                  if (PAIR) {
                    const float turn = far ? coef : 1.0f / coef;
#pragma unroll
                    for (int i = 0; i < 128; ++i) s[i] *= turn;
                  }
                  slack = far ? 0.0f : kGrow + kLift;
                  unit = far ? 1.0f : coef;
                  sign = far ? signed_coef : copysignf(1.0f, signed_coef);
                  turned = far || scale < 0.0f;
                }
                const float ref = far ? top : top - kLift;
                const float f = grow ? exp2_approx(m - ref) : 1.0f;
                if (grow) m = ref;
                l *= f;
                // the product before this one is complete: its tensor work came before these scores'
                if (steps > 0) {
                  const uint32_t o_at = tmem + C::kO + D * slot + lanes;
#pragma unroll 1
                  for (int c = 0; c < D; c += 16) {
                    uint32_t o[16];
                    tmem_ld16(o_at + c, o);
                    tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                    tmem_st16(o_at + c, o);
                  }
                }
              }
            };
            // weights of 32 scores (times `unit`), as 16-bit pairs, and their sum into l
            auto weigh = [&](const float* s, int c) {
              const float ref = m == -INFINITY ? 0.0f : -m;
              float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
              uint32_t w[16];
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                float2 x = fma2(make_float2(s[2 * i], s[2 * i + 1]), make_float2(unit, unit), make_float2(ref, ref));
                x.x = exp2_approx(x.x);
                x.y = exp2_approx(x.y);
                sum[i & 1] = add2(sum[i & 1], x);
                w[i] = FP8 ? pack_f16x2(x.x, x.y) : pack_bf16x2(x.x, x.y);
              }
              tmem_st16(s_at + 16 * c, w);
              l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
            };
            if (PAIR && work) {
              // all 128 scores at once, straight through: the prompt kernels run long enough
              float s[128];
#pragma unroll
              for (int c = 0; c < 4; ++c) tmem_ld32(s_at + 32 * c, s + 32 * c);
              tmem_ld_wait();
              if (turned) {
#pragma unroll
                for (int i = 0; i < 128; ++i) s[i] *= sign;
              }
              if (__any_sync(~0u, in && (key0 < jlo || key0 + kTcBN > jhi))) {
#pragma unroll
                for (int i = 0; i < 128; ++i)
                  if (key0 + i < jlo || key0 + i >= jhi) s[i] = -INFINITY;
              }
              float t8[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) t8[e] = max3(s[e], s[8 + e], s[16 + e]);
#pragma unroll
              for (int i = 24; i < 120; i += 16)
#pragma unroll
                for (int e = 0; e < 8; ++e) t8[e] = max3(t8[e], s[i + e], s[i + 8 + e]);
              const float t_a = max3(max3(t8[0], s[120], s[121]), max3(t8[1], s[122], s[123]), t8[2]);
              const float t_b = max3(max3(t8[3], s[124], s[125]), max3(t8[4], s[126], s[127]), t8[5]);
              refer(max3(max3(t_a, t_b, t8[6]), t8[7], t8[7]) * unit, s);
#pragma unroll
              for (int c = 0; c < 4; ++c) weigh(s + 32 * c, c);
              tmem_st_wait();
            } else if (work && !PAIR) {
              // 32 scores at a time, read once for the maximum and once for the weights, in a loop
              // that stays rolled: unrolled, a call's first tile waited 5 us for its instructions
              const bool masked = __any_sync(~0u, in && (key0 < jlo || key0 + kTcBN > jhi));
              float top = -INFINITY;
#pragma unroll 1
              for (int i = 0; i < 8; ++i) {
                const int c = i & 3;
                float s[32];
                tmem_ld32(s_at + 32 * c, s);
                tmem_ld_wait();
                if (turned) {
#pragma unroll
                  for (int k = 0; k < 32; ++k) s[k] *= sign;
                }
                if (masked) {
                  const int from = jlo - key0 - 32 * c, to = jhi - key0 - 32 * c;
#pragma unroll
                  for (int k = 0; k < 32; ++k)
                    if (k < from || k >= to) s[k] = -INFINITY;
                }
                if (i < 4) {
#pragma unroll
                  for (int k = 0; k < 32; k += 2) top = fmaxf(top, fmaxf(s[k], s[k + 1]));
                  if (i == 3) refer(top * unit, nullptr);  // the scores are read again
                } else {
                  weigh(s, c);
                }
              }
              tmem_st_wait();
            }
            tc_fence_before();
            mbar_arrive(smem_addr(&sh.p_full[slot]));
          }
        }

        // ---- the item's rows leave
        const bool whole = kt0 == 0 && n == it.tiles;
        if (tid == 0 && kt0 == 0 && !whole)
          say_cut(a, blockIdx.x, &it, n, share.chunk, 2 * blockIdx.x + (first ? 0 : 1));
        const long long piece = (2LL * blockIdx.x + (first ? 0 : 1)) * kRows + (PAIR ? slot * 128 : 0) + row;
        if (PAIR) {
          if (active && ok) {
            WAIT_OR(sh.o_full[slot], o_phase, ok = false);
            o_phase ^= 1;
            release();
          } else {
            rel = (rel + 2 * n) % S;
          }
        } else if (ok) {
          ml[128 * slot + row] = make_float2(m, l);
          mbar_arrive(smem_addr(&sh.joined));
          WAIT_OR(sh.joined, j_phase, ok = false);
          if (ok) WAIT_OR(sh.o_full[0], o_phase, ok = false);
          if (ok) WAIT_OR(sh.o_full[1], o_phase, ok = false);
          o_phase ^= 1;
        }
        if (!ok) break;
        tc_fence_after();
        if (active && work) {
          // PAIR: this slot's row.  Else both slots' parts of the row; each slot stores half of it.
          float f0 = 1.0f, f1 = 0.0f;
          if (!PAIR) {
            const float2 x = ml[row], y = ml[128 + row];
            m = fmaxf(x.x, y.x);
            f0 = m == -INFINITY ? 0.0f : exp2_approx(x.x - m);
            f1 = m == -INFINITY ? 0.0f : exp2_approx(y.x - m);
            l = f0 * x.y + f1 * y.y;
          }
          const bool two = !PAIR && n > 1;
          const float inv = whole ? (l > 0.0f ? vscale / l : (l == 0.0f ? 0.0f : l)) : 1.0f;
          const long long orow = (long long)(it.q.row0 + tok) * a.Hq + it.h * G + (r - tok * G);
          constexpr int kCols = PAIR ? D : D / 2;
          const int c0 = PAIR ? 0 : slot * kCols;
#pragma unroll
          for (int c = 0; c < kCols; c += 16) {
            uint32_t x[16], y[16];
            tmem_ld16(tmem + C::kO + (PAIR ? D * slot : 0) + lanes + c0 + c, x);
            if (two) tmem_ld16(tmem + C::kO + D + lanes + c0 + c, y);
            tmem_ld_wait();
            float v[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              v[i] = __uint_as_float(x[i]);
              if (!PAIR) v[i] = two ? f0 * v[i] + f1 * __uint_as_float(y[i]) : f0 * v[i];
              v[i] *= inv;
            }
            if (in && whole) {
              uint32_t w[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) w[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
              st_global_32(a.out + orow * D + c0 + c, w, a.wide);
            } else if (in) {
              const uint32_t* w = reinterpret_cast<const uint32_t*>(v);
              st_global_32(a.piece_o + piece * D + c0 + c, w, a.wide);
              st_global_32(a.piece_o + piece * D + c0 + c + 8, w + 8, a.wide);
            }
          }
          if (in && (PAIR || slot == 0)) {
            if (!whole) a.piece_ml[piece] = make_float2(m, l);
            else if (a.lse) a.lse[orow] = l == 0.0f ? -INFINITY : m * 0.6931471805599453f + logf(l);
          }
        }
        tc_fence_before();
        if (!PAIR) {  // the next item's products overwrite what both slots read here
          mbar_arrive(smem_addr(&sh.left));
          WAIT_OR(sh.left, j_phase, { ok = false; break; });
          j_phase ^= 1;
        }
        first = false;
        if (left <= 0 || !walk_next(a, it)) break;
      }
      if (!ok) {  // neither piece of this row is to be joined
        for (int i = 0; i < 2; ++i)
          a.piece_ml[(2LL * blockIdx.x + i) * kRows + (PAIR ? slot * 128 : 0) + row] = make_float2(0.0f, kNoPiece);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
}

template <int D, bool PAIR, bool FP8>
cudaError_t launch_tc(AttnArgs a, cudaStream_t s) {
  using C = Tc<D, PAIR, FP8>;
  static std::atomic<int> ready[kMaxDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  int ctas = ready[dev].load(std::memory_order_relaxed);
  if (!ctas) {
    e = cudaFuncSetAttribute(attn_tc_kernel<D, PAIR, FP8>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    int sms = 0;
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    ctas = std::max(1, std::min(sms, kMaxPieceRows / 2 / (PAIR ? 256 : 128)));
    ready[dev].store(ctas, std::memory_order_relaxed);
  }
  CUtensorMap kmap, vmap;
  if (!encode_cache(&kmap, a.p, a.p.k, D, FP8, kTcBN) || !encode_cache(&vmap, a.p, a.p.v, D, FP8, kTcBN)) return cudaErrorNotSupported;
  a.ctas = ctas;
  a.shape.r_shift = PAIR ? 8 : 7;
  a.shape.bn_shift = 7;
  // what an item costs beside its tiles, measured: 24 ragged draft blocks take 50.7 us with 3 tiles'
  // worth, 53 with 8 (and 190 with none, on an earlier form); 3,200 rows over 4,000 keys 154 us with
  // 2, 143 with 6
  a.shape.lead = PAIR ? 6 : 3;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr = {};
  attention_config(&cfg, &attr, ctas, C::kThreads, C::kSmem, s);
  e = cudaLaunchKernelEx(&cfg, attn_tc_kernel<D, PAIR, FP8>, a, kmap, vmap);
  return e != cudaSuccess ? e : launch_combine(a, D, s);
}

}  // namespace

// True where the kernel can run: heads of 64 or 128, pages that TMA can box.
bool attention_tc_fits(const AttnArgs& a, int D) { return D <= 128 && a.p.page_mask + 1 >= 16; }

template <int D, bool PAIR>
cudaError_t launch_type(const AttnArgs& a, bool fp8, cudaStream_t s) {
  return fp8 ? launch_tc<D, PAIR, true>(a, s) : launch_tc<D, PAIR, false>(a, s);
}
cudaError_t launch_attention_tc(const AttnArgs& a, int D, bool fp8, bool pair, cudaStream_t s) {
  if (D == 64) return pair ? launch_type<64, true>(a, fp8, s) : launch_type<64, false>(a, fp8, s);
  return pair ? launch_type<128, true>(a, fp8, s) : launch_type<128, false>(a, fp8, s);
}

}  // namespace lowbit
