// What the attention kernels share: their arguments, the walk over a CTA's share of the work,
// the pieces of items that were cut, and the launch of a kernel with its combine step.
#pragma once

#include <algorithm>
#include <atomic>

#include "common.cuh"
#include "paged.cuh"
#include "ptx.cuh"

namespace lowbit {

constexpr int kMaxDevices = 64;
// Scores (in powers of two) past it are rounded to more than an eighth in fp32: their weights then refer to
// the largest itself.
constexpr float kFarScore = 1048576.0f;
__device__ __forceinline__ bool far_score(float x) { return fabsf(x) > kFarScore && fabsf(x) != INFINITY; }
// Query rows of all pieces together: every CTA may leave two (the item it starts inside of and
// the one it ends inside of).  The workspace holds D + 2 floats for each; a kernel's grid is
// limited so that 2 * CTAs * rows stays within it.
constexpr int kMaxPieceRows = 2 * 152 * 256;

// What a CTA says about the item that its share ends inside of, if it began that item: `more` other
// CTAs, the ones behind it, have a piece too (0: nothing to join).
// A piece whose CTA gave up a wait has a sum of -1 in its rows: the combine step leaves what it is part of
// unwritten.
constexpr float kNoPiece = -1.0f;
struct CutItem {
  int more, slot, rows, r0;  // its own piece's slot; the query tile's rows and first row
  int row0, h, pad0, pad1;   // the request's first row, the key/value head
};
constexpr int kMaxCtas = kMaxPieceRows / 2 / 16;

struct AttnArgs {
  PagedArgs p;
  ItemShape shape;
  const uint16_t* q;
  long long q_stride;
  int Hq;
  float scale;
  uint16_t* out;
  float* lse;
  float* piece_o;   // [slot][R][D], weights relative to the piece's reference, not divided by their sum
  float2* piece_ml; // [slot][R]: reference (of scale * score * log2 e; about the maximum) and sum
  CutItem* cuts;    // [CTA]
  int ctas;
  bool wide;        // out and the pieces start on 32-byte boundaries
  int stall;        // test-only stall setting (lowbit_debug_inject_stall), under which the first data (tiles,
                    // or queries on tcgen05) never come, so that every role's wait gives up; 0 in normal use
};

cudaError_t launch_attention_mma(const AttnArgs& a, int D, bool fp8, cudaStream_t s);

// a / b of nonnegative numbers: 32-bit where both fit (a 64-bit division is a hundred instructions).
__device__ __forceinline__ long long quotient(long long a, long long b) {
  if (((a | b) >> 32) == 0) return (uint32_t)a / (uint32_t)b;
  return a / b;
}
__device__ __forceinline__ long long warp_sum(long long c) {
  for (int o = 16; o; o >>= 1) c += __shfl_xor_sync(~0u, c, o);
  return c;
}
__device__ __forceinline__ long long warp_inclusive(long long c, int lane) {
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(~0u, c, o);
    if (lane >= o) c += v;
  }
  return c;
}

// Cost of one head of request b: by one thread, or (`lane` >= 0) by a whole warp.
__device__ __forceinline__ long long head_cost(const ItemShape& s, const Request& q, int lane) {
  const int nq = query_tiles(s, q);
  if (nq == 1) return tile_cost(s, tile_span(s, q, 0)) + s.lead;
  long long c = 0;
  for (int i = lane < 0 ? 0 : lane; i < nq; i += lane < 0 ? 1 : 32) c += tile_cost(s, tile_span(s, q, i)) + s.lead;
  return lane < 0 ? c : warp_sum(c);
}

// The walk over a CTA's share of the items: every warp keeps its own copy.
struct Walk {
  Request q;
  Span span;
  int b, h, qt, nq;
  int lead;         // of the item's lead, what is left
  int tile, tiles;  // next key tile of the item, and how many it has
};
__device__ __forceinline__ void walk_item(const AttnArgs& a, Walk& w, int off) {
  w.span = tile_span(a.shape, w.q, w.qt);
  w.tiles = tile_cost(a.shape, w.span);
  w.lead = max(0, a.shape.lead - off);
  w.tile = max(0, off - a.shape.lead);
}

// The share of CTA `cta`: its first unit, how many, and the walk to the first; false if it has
// none.  By all NT threads of the block.
struct Share {
  long long begin, chunk;
  int left;
};
// The short way, every warp on its own: up to 32 requests of one query tile each, one per lane, in
// 32 bits.  A decode or verify step is over in some microseconds, of which the instructions a
// CTA touches for the first time are a large part (about 6 cycles each when they come from
// memory), so this way is kept apart from the general one: 0 = not applicable, 1 = found,
// -1 = the CTA has no share.
__device__ __forceinline__ int start_walk_short(const AttnArgs& a, int cta, Walk& w, Share& sh) {
  const int lane = threadIdx.x & 31;
  if (a.p.B > 32) return 0;
  Request q = {0, 0, 0};
  if (lane < a.p.B) q = load_request(a.p, lane);
  // one tile holds every row: its keys end with the request's, whatever the mask
  const int lo = first_key(a.shape, q.kv - q.n);
  const bool none = lo >= q.kv;
  const int tiles = none ? 1 : ((q.kv - 1) >> a.shape.bn_shift) - (lo >> a.shape.bn_shift) + 1;
  const uint32_t cost = q.n ? (uint32_t)(tiles + a.shape.lead) : 0;
  const bool big = (long long)q.n * a.shape.G > (1 << a.shape.r_shift) || (unsigned long long)cost * a.p.Hk > (1u << 25);
  if (__any_sync(~0u, big)) return 0;
  uint32_t incl = cost * a.p.Hk;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t v = __shfl_up_sync(~0u, incl, o);
    if (lane >= o) incl += v;
  }
  const uint32_t total = __shfl_sync(~0u, incl, 31);
  const uint32_t chunk = (total + a.ctas - 1) / a.ctas;
  const uint32_t begin = cta * chunk;
  if (begin >= total) return -1;
  sh.begin = begin;
  sh.chunk = chunk;
  sh.left = (int)min(chunk, total - begin);
  const int src = __ffs(__ballot_sync(~0u, incl > begin)) - 1;
  uint32_t off = begin - __shfl_sync(~0u, incl - cost * a.p.Hk, src);
  const uint32_t each = __shfl_sync(~0u, cost, src);
  w.b = src;
  w.q.row0 = __shfl_sync(~0u, q.row0, src);
  w.q.n = __shfl_sync(~0u, q.n, src);
  w.q.kv = __shfl_sync(~0u, q.kv, src);
  w.span.lo = __shfl_sync(~0u, none ? 0 : lo, src);
  w.span.hi = __shfl_sync(~0u, none ? 0 : q.kv, src);
  w.h = (int)(off / each);
  off -= w.h * each;
  w.nq = 1;
  w.qt = 0;
  w.tiles = (int)each - a.shape.lead;
  w.lead = max(0, a.shape.lead - (int)off);
  w.tile = max(0, (int)off - a.shape.lead);
  return 1;
}
// Up to 32 requests every warp sums them on its own (one per lane, or one after another where each
// has many query tiles), so that nothing waits for a barrier; above, the block does.
template <int NT>
__device__ __forceinline__ bool start_walk(const AttnArgs& a, int cta, Walk& w, Share& sh) {
  __shared__ long long s_warp[NT / 32], s_off;
  __shared__ int s_b;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int brief = start_walk_short(a, cta, w, sh);
  if (brief) return brief > 0;
  const bool tall = (long long)a.p.T * a.shape.G > (4LL << a.shape.r_shift) * a.p.B;
  long long total, off = 0;
  auto share = [&]() {
    sh.chunk = quotient(total + a.ctas - 1, a.ctas);
    sh.begin = (long long)cta * sh.chunk;
    sh.left = (int)(min(sh.begin + sh.chunk, total) - sh.begin);
    return sh.left > 0;
  };
  w.b = 0;
  if (a.p.B <= 32) {
    long long sum = 0;
    if (tall) {
#pragma unroll 1
      for (int b = 0; b < a.p.B; ++b) {
        const long long c = head_cost(a.shape, load_request(a.p, b), lane) * a.p.Hk;
        if (lane == b) sum = c;
      }
    } else if (lane < a.p.B) {
      sum = head_cost(a.shape, load_request(a.p, lane), -1) * a.p.Hk;
    }
    const long long incl = warp_inclusive(sum, lane);
    total = __shfl_sync(~0u, incl, 31);
    if (!share()) return false;
    w.b = __ffs(__ballot_sync(~0u, incl > sh.begin)) - 1;
    off = sh.begin - __shfl_sync(~0u, incl - sum, w.b);
  } else {
    // One pass where every request has a thread (or a warp) of its own; else pass 0 sums and pass 1
    // finds the request that holds the share's begin.
    const int step = tall ? NT / 32 : NT;
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass) {
      long long carry = 0;
#pragma unroll 1
      for (int b0 = 0; b0 < a.p.B; b0 += step) {
        const int b = b0 + (tall ? warp : tid);
        long long c = 0;
        if (b < a.p.B) c = head_cost(a.shape, load_request(a.p, b), tall ? lane : -1) * a.p.Hk;
        const long long incl = tall ? c : warp_inclusive(c, lane);
        if (b0 || pass) __syncthreads();
        if (lane == 31) s_warp[warp] = incl;
        __syncthreads();
        long long before = carry;
#pragma unroll
        for (int i = 0; i < NT / 32; ++i) {
          const long long v = s_warp[i];
          if (i < warp) before += v;
          carry += v;
        }
        if (a.p.B <= step) {
          total = carry;
          if (!share()) return false;  // the whole block alike
        }
        const long long at = before + incl - c;
        if ((pass || a.p.B <= step) && sh.begin >= at && sh.begin < at + c && (!tall || lane == 0))
          s_b = b, s_off = sh.begin - at;
      }
      total = carry;
      if (a.p.B <= step) break;
      if (!pass && !share()) return false;
    }
    __syncthreads();
    w.b = s_b;
    off = s_off;
  }
  w.q = load_request(a.p, w.b);

  // the head, the query tile and the place inside the item
  w.nq = query_tiles(a.shape, w.q);
  const long long each = head_cost(a.shape, w.q, lane);
  w.h = (int)quotient(off, each);
  off -= w.h * each;
  w.qt = 0;
  if (w.nq > 1)
    for (int i0 = 0; i0 < w.nq; i0 += 32) {
      const int i = i0 + lane;
      const long long c = i < w.nq ? tile_cost(a.shape, tile_span(a.shape, w.q, i)) + a.shape.lead : 0;
      const long long incl = warp_inclusive(c, lane);
      const unsigned past = __ballot_sync(~0u, incl > off);
      if (past) {
        const int src = __ffs(past) - 1;
        w.qt = i0 + src;
        off -= __shfl_sync(~0u, incl - c, src);
        break;
      }
      off -= __shfl_sync(~0u, incl, 31);
    }
  walk_item(a, w, (int)off);
  return true;
}
// Key tiles of the current item that fall into what is left of the share, which they use up;
// 0 when the share ends before its tiles.
__device__ __forceinline__ int walk_take(Walk& w, int& left) {
  left -= w.lead;
  const int n = min(w.tiles - w.tile, left);
  left -= n;
  return max(0, n);
}
// To the next item; false past the last request.
__device__ __forceinline__ bool walk_next(const AttnArgs& a, Walk& w) {
  if (++w.qt == w.nq) {
    w.qt = 0;
    if (++w.h == a.p.Hk) {
      w.h = 0;
      do {
        if (++w.b >= a.p.B) return false;
        w.q = load_request(a.p, w.b);
        w.nq = query_tiles(a.shape, w.q);
      } while (w.nq == 0);
    }
  }
  walk_item(a, w, 0);
  return true;
}

// 4-D tiled tensor copy (TMA) global -> shared.
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w,
                                            uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
      : "memory");
}

// The cache as [page][head][slot][D], boxes of 128 bytes (64, where a row has no more) by one page's
// slots, at most `keys`, swizzled over the box's row length.
bool encode_cache(CUtensorMap* map, const PagedArgs& p, void* at, int D, bool fp8, int keys);

// By one thread: CTA `cta` leaves the walk's item after tile `done`, whose first piece it holds, or
// (w null) leaves nothing to join.
__device__ __forceinline__ void say_cut(const AttnArgs& a, int cta, const Walk* w, int done, long long chunk, int slot) {
  int4 lo = make_int4(0, 0, 0, 0), hi = lo;
  if (w) {
    const int R = 1 << a.shape.r_shift, r0 = w->qt << a.shape.r_shift;
    lo = make_int4((int)quotient(w->tiles - done + chunk - 1, chunk), slot, min(R, w->q.n * a.shape.G - r0), r0);
    hi = make_int4(w->q.row0, w->h, 0, 0);
  }
  reinterpret_cast<int4*>(a.cuts + cta)[0] = lo;
  reinterpret_cast<int4*>(a.cuts + cta)[1] = hi;
}

// Launch configuration of an attention kernel of `ctas` resident CTAs, and the combine step behind it.
void attention_config(cudaLaunchConfig_t* cfg, cudaLaunchAttribute* attr, int ctas, int threads, int smem,
                      cudaStream_t s);
cudaError_t launch_combine(const AttnArgs& a, int D, cudaStream_t s);

// The tensor-core kernel (paged_attn_tc.cu): whether it can take the call, and its launch with 256
// (`pair`) or 128 query rows per item.
bool attention_tc_fits(const AttnArgs& a, int D);
cudaError_t launch_attention_tc(const AttnArgs& a, int D, bool fp8, bool pair, cudaStream_t s);

}  // namespace lowbit
