// What the attention kernels share: their arguments, the walk over a CTA's share of the work,
// the pieces of items that were cut, and the launch of a kernel with its combine step.
#pragma once

#include <algorithm>
#include <atomic>
#include <type_traits>

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

// lowbit_prefix_attention runs the same kernels over a longer list of "requests": first its groups (all rows of a
// group over the keys that its requests share), then the requests over their own keys; a launch takes
// a part of that list.  Every row leaves as a piece does, from whichever of the two, and the join step
// (prefix_attn.cu) finds by `found` where its pieces are.
struct PrefixArgs : AttnArgs {
  int first;        // the launch's part of the list: p.B entries from here on
  int groups, requests;
  const int32_t* cu_groups;
  const int32_t* prefix_lens;
  long long rows;   // rows of out, T * Hq; of the arrays below first the shared part's, then the own part's
  float* base_o;    // [2][row][D]: rows that one CTA saw all keys of
  float2* base_ml;  // [2][row]
  int4* found;      // [2][row]: {kInBase or kLost}, or {more, first, next, apart}: places of the first piece and of
                    // the `more` that follow it, the second at `next` and the others `apart` behind one another
};
constexpr int kInBase = -1, kLost = -2;
template <class A>
constexpr bool kPrefix = std::is_same<A, PrefixArgs>::value;

__device__ __forceinline__ Request load_request(const AttnArgs& a, int b) {
  return check_request(a.p, a.p.cu_q[b], a.p.cu_q[b + 1], a.p.kv_lens[b]);
}
// The last group that begins at request b or before it, by bisection.  Every kernel of a call looks a request's group up
// with it, so that all agree where cu_groups is not ascending.
__device__ __forceinline__ int group_of(const PrefixArgs& a, int b) {
  int g = 0;
#pragma unroll 1
  for (int end = a.groups; end - g > 1;) {
    const int mid = (g + end) / 2;
    if (a.cu_groups[mid] <= b) g = mid;
    else end = mid;
  }
  return g;
}
// All rows of group g over the whole pages of its shared length; no rows where there are none.
__device__ __forceinline__ Request load_group(const PrefixArgs& a, int g) {
  const int from = a.cu_groups[g], to = a.cu_groups[g + 1], len = a.prefix_lens[g];
  if (from < 0 || to < from || to > a.requests || len < 0) {
    record_error(a.p.err, LOWBIT_ERR_INVALID_ARG);
    return Request{0, 0, 0, 0, 1};
  }
  Request r = check_request(a.p, a.p.cu_q[from], a.p.cu_q[to], len & ~a.p.page_mask);
  r.all = 1;
  if (r.kv == 0) r.n = 0;
  return r;
}
// Request b, of group g, without the keys that the group shares.  One that has new tokens among these counts as inconsistent;
// what else can be wrong with it the join step looks for, which keeps its loads out of the way here.
__device__ __forceinline__ Request load_own(const PrefixArgs& a, int b, int g) {
  const int skip = a.prefix_lens[g] & ~a.p.page_mask;
  Request r = check_request(a.p, a.p.cu_q[b], a.p.cu_q[b + 1], a.p.kv_lens[b]);
  if (r.n == 0) return r;
  if (skip < 0 || r.kv - r.n < skip) {
    record_error(a.p.err, LOWBIT_ERR_INVALID_ARG);
    return Request{0, 0, 0, 0, 0};
  }
  r.kv -= skip;
  r.skip = skip;
  return r;
}
__device__ __forceinline__ Request load_request(const PrefixArgs& a, int b) {
  b += a.first;
  return b < a.groups ? load_group(a, b) : load_own(a, b - a.groups, group_of(a, b - a.groups));
}
// The block table from the page of the request's first counted key on.
__device__ __forceinline__ const int32_t* table_of(const AttnArgs& a, int b, const Request&) {
  return a.p.table + (long long)b * a.p.table_stride;
}
__device__ __forceinline__ const int32_t* table_of(const PrefixArgs& a, int b, const Request& r) {
  b += a.first;
  b = b < a.groups ? a.cu_groups[b] : b - a.groups;
  return a.p.table + (long long)b * a.p.table_stride + (r.skip >> a.p.page_shift);
}

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
template <class A>
__device__ __forceinline__ int start_walk_short(const A& a, int cta, Walk& w, Share& sh) {
  const int lane = threadIdx.x & 31;
  if (a.p.B > 32) return 0;
  Request q = {0, 0, 0, 0, 0};
  if (lane < a.p.B) q = load_request(a, lane);
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
  w.q.skip = kPrefix<A> ? __shfl_sync(~0u, q.skip, src) : 0;  // the constant leaves no trace in the plain kernels
  w.q.all = kPrefix<A> ? __shfl_sync(~0u, q.all, src) : 0;
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
template <int NT, class A>
__device__ __forceinline__ bool start_walk(const A& a, int cta, Walk& w, Share& sh) {
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
        const long long c = head_cost(a.shape, load_request(a, b), lane) * a.p.Hk;
        if (lane == b) sum = c;
      }
    } else if (lane < a.p.B) {
      sum = head_cost(a.shape, load_request(a, lane), -1) * a.p.Hk;
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
        if (b < a.p.B) c = head_cost(a.shape, load_request(a, b), tall ? lane : -1) * a.p.Hk;
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
  w.q = load_request(a, w.b);

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
template <class A>
__device__ __forceinline__ bool walk_next(const A& a, Walk& w) {
  if (++w.qt == w.nq) {
    w.qt = 0;
    if (++w.h == a.p.Hk) {
      w.h = 0;
      do {
        if (++w.b >= a.p.B) return false;
        w.q = load_request(a, w.b);
        w.nq = query_tiles(a.shape, w.q);
      } while (w.nq == 0);
    }
  }
  walk_item(a, w, 0);
  return true;
}

// Where a row's (reference, sum) and output go that do not go to out: to its piece, or to its base.
struct Part {
  float2* ml;
  float* o;
};
template <int D>
__device__ __forceinline__ Part part_of(const AttnArgs& a, const Walk&, bool, long long, long long piece) {
  return Part{a.piece_ml + piece, a.piece_o + piece * D};
}
template <int D>
__device__ __forceinline__ Part part_of(const PrefixArgs& a, const Walk& w, bool whole, long long row, long long piece) {
  if (!whole) return Part{a.piece_ml + piece, a.piece_o + piece * D};
  if (a.first + w.b >= a.groups) row += a.rows;
  return Part{a.base_ml + row, a.base_o + row * D};
}
// By the CTA that holds the first piece of a row, place `in_tile` of its item, done up to key tile `done`.
__device__ __forceinline__ void say_found(const AttnArgs&, const Walk&, long long, bool, int, int, long long, long long) {}
__device__ __forceinline__ void say_found(const PrefixArgs& a, const Walk& w, long long row, bool good, int done, int in_tile,
                                          long long chunk, long long piece) {
  if (a.first + w.b >= a.groups) row += a.rows;
  int4 f = make_int4(good ? kInBase : kLost, 0, 0, 0);
  if (good && done < w.tiles)
    f = make_int4((int)quotient(w.tiles - done + chunk - 1, chunk), (int)piece,
                  (2 * ((int)blockIdx.x + 1) << a.shape.r_shift) + in_tile, 2 << a.shape.r_shift);
  a.found[row] = f;
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

// Launch configuration of an attention kernel of `ctas` resident CTAs.
void attention_config(cudaLaunchConfig_t* cfg, cudaLaunchAttribute* attr, int ctas, int threads, int smem,
                      cudaStream_t s);

// The tensor-core kernel (paged_attn_tc.cu): whether it can take the call, and its launch with 256
// (`pair`) or 128 query rows per item.
bool attention_tc_fits(const AttnArgs& a, int D);
cudaError_t launch_attention_tc(const AttnArgs& a, int D, bool fp8, bool pair, cudaStream_t s);
cudaError_t launch_attention_tc(const PrefixArgs& a, int D, bool fp8, bool pair, cudaStream_t s);
// The combine step behind lowbit_paged_attention's.
cudaError_t launch_combine(const AttnArgs& a, int D, cudaStream_t s);


// Checks of the arguments that both attention calls take; fills `a` all but the workspace and the error word.
// LOWBIT_OK with T = 0: nothing to do.
lowbit_status make_attn_args(const uint16_t* q, int64_t q_stride, int Hq, const lowbit_paged_batch* batch,
                             const lowbit_paged_cache* cache, float scale, int causal, int window, uint16_t* out,
                             float* lse, AttnArgs* a);

// The pieces of a launch, and what its CTAs say about them, from `at` on (a multiple of 32 bytes in all).
inline size_t pieces_bytes(int D) {
  return (size_t)kMaxPieceRows * (size_t)(D + 2) * sizeof(float) + (size_t)kMaxCtas * sizeof(CutItem);
}
inline void use_pieces(AttnArgs* a, void* at, int D) {
  a->piece_o = static_cast<float*>(at);
  a->piece_ml = reinterpret_cast<float2*>(a->piece_o + (size_t)kMaxPieceRows * D);
  a->cuts = reinterpret_cast<CutItem*>(a->piece_ml + kMaxPieceRows);
}

// By the rows that share a request's keys, on average (the host knows the totals only; a request that
// differs from the average is computed right and slowly).  At 32 rows each side wins somewhere, the warp-level
// MMA on short contexts and where the start counts, tcgen05 on long ones; above, tcgen05 nearly always.  Heads of
// 128, one request of 30,000 keys, us on the warp-level MMA / tcgen05 with 128 rows an item / with
// 256: 32 rows 38.7 / 36.3 / 51.8, 64 rows 47.8 / 37.6 / 59.8, 400 rows 189 / 81 / 101; of 500 keys
// 9.6 / 11 / 13 with 32 rows.  Heads of 64: 48 rows 29.8 / 26.1, 32 requests of up to 16,000 keys 48.0 /
// 49.0.  256 rows an item pay when there are many: one request of 16,000 keys, 800 rows 71 with 128 and
// 69 with 256, 1,600 rows 116 and 103, 3,200 rows 200 and 171 (of 4,000 keys 33 and 37, 48 and 50, 69 and 69).
// Over e4m3 caches the same limits hold: heads of 128, 30,000 keys, warp-level MMA / tcgen05: 32 rows 35.3 /
// 29.5, 40 rows 48.2 / 32.2 (500 keys 10.4 / 10.8), 16 requests of up to 8,000 keys and 32 rows 28.7 / 29.8, 40
// rows 33.7 / 27.5; heads of 64, 48 rows 31.2 / 27.0 and 20.9 / 22.7; 256 rows an item: 16,000 keys, 1,600 rows
// 137 with 128 and 114 with 256 (of 4,000 keys 49 and 52).
inline cudaError_t launch_attention(const AttnArgs& a, int D, bool fp8, cudaStream_t s) {
  const long long rows = ((long long)a.p.T * a.shape.G + a.p.B - 1) / a.p.B;
  return rows > (D == 64 ? 48 : 32) && attention_tc_fits(a, D) ? launch_attention_tc(a, D, fp8, rows > 1024, s)
                                                               : launch_attention_mma(a, D, fp8, s);
}

}  // namespace lowbit
