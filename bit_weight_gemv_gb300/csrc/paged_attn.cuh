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
// Query rows of all pieces together: every CTA may leave two (the item it starts inside of and
// the one it ends inside of).  The workspace holds D + 2 floats for each; a kernel's grid is
// limited so that 2 * CTAs * rows stays within it.
constexpr int kMaxPieceRows = 2 * 152 * 256;

#include <cstdlib>
inline int tune(const char* n, int d) { const char* v = getenv(n); return v ? atoi(v) : d; }
struct AttnArgs {
  PagedArgs p;
  ItemShape shape;
  const uint16_t* q;
  long long q_stride;
  int Hq;
  float scale;
  uint16_t* out;
  float* lse;
  float* piece_o;   // [slot][R][D], relative to the piece's maximum, not divided by its sum
  float2* piece_ml; // [slot][R]: maximum (of scale * score * log2 e) and sum
  int ctas;
  int min_chunk;    // tiles a CTA takes at least
};

cudaError_t launch_attention_mma(const AttnArgs& a, int D, bool fp8, cudaStream_t s);

// A CTA's share [begin, end) of the work, in key tiles and leads, and where begin falls.
struct Plan {
  long long begin, end, chunk;
  long long off;  // of begin inside request b's work
  int b;
};

// a / b of nonnegative numbers: 32-bit where both fit (a 64-bit division is a hundred instructions).
__device__ __forceinline__ long long quotient(long long a, long long b) {
  if (((a | b) >> 32) == 0) return (uint32_t)a / (uint32_t)b;
  return a / b;
}

// Cost of one head of request b.  `lane` < 0: by one thread alone, else by a whole warp.
__device__ __forceinline__ long long head_cost(const ItemShape& s, const Request& q, int lane) {
  const int nq = query_tiles(s, q);
  if (nq == 1) return tile_cost(s, tile_span(s, q, 0)) + s.lead;
  long long c = 0;
  for (int i = lane < 0 ? 0 : lane; i < nq; i += lane < 0 ? 1 : 32) c += tile_cost(s, tile_span(s, q, i)) + s.lead;
  if (lane >= 0)
    for (int o = 16; o; o >>= 1) c += __shfl_xor_sync(~0u, c, o);
  return c;
}

// The CTA's share, by all NT threads of the block (a multiple of 32); `pl` is valid after the
// next __syncthreads.  Requests are summed one per thread, or one per warp where each has many
// query tiles.
template <int NT>
__device__ __forceinline__ void make_plan(const AttnArgs& a, Plan& pl, int cta) {
  __shared__ long long s_warp[NT / 32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const bool by_warp = (long long)a.p.T * a.shape.G > (4LL << a.shape.r_shift) * a.p.B;
  long long total = 0, chunk = 0, begin = 0, end = 0;
  if (tid == 0) pl.b = a.p.B, pl.off = 0, pl.begin = pl.end = 0;
  // pass 0 sums, pass 1 finds the request that holds `begin`; one pass serves when every request
  // has a thread (or a warp) of its own
  const int step = by_warp ? NT / 32 : NT;
  for (int pass = 0; pass < 2; ++pass) {
    long long carry = 0;
    for (int b0 = 0; b0 < a.p.B; b0 += step) {
      const int b = b0 + (by_warp ? warp : tid);
      long long c = 0;
      if (b < a.p.B) {
        const Request q = load_request(a.p, b);
        c = head_cost(a.shape, q, by_warp ? lane : -1) * a.p.Hk;
      }
      long long incl = c;  // inclusive sum over the requests of this warp
      if (!by_warp)
        for (int o = 1; o < 32; o <<= 1) {
          const long long v = __shfl_up_sync(~0u, incl, o);
          if (lane >= o) incl += v;
        }
      if (b0) __syncthreads();
      if (lane == 31) s_warp[warp] = incl;
      __syncthreads();
      long long before = carry;
#pragma unroll
      for (int i = 0; i < NT / 32; ++i) {
        const long long v = s_warp[i];
        if (i < warp) before += v;
        carry += v;
      }
      if (pass == 0 && a.p.B <= step) {
        total = carry;
        chunk = max((long long)a.min_chunk, quotient(total + a.ctas - 1, a.ctas));
        begin = (long long)cta * chunk;
        end = min(begin + chunk, total);
      }
      if (pass == 1 || a.p.B <= step) {
        const long long at = before + incl - c;
        if (begin < total && begin >= at && begin < at + c && (!by_warp || lane == 0)) {
          pl.b = b;
          pl.off = begin - at;
          pl.begin = begin;
          pl.end = end;
        }
      }
    }
    if (a.p.B <= step) break;
    total = carry;
    chunk = max((long long)a.min_chunk, quotient(total + a.ctas - 1, a.ctas));
    begin = (long long)cta * chunk;
    end = min(begin + chunk, total);
    __syncthreads();
  }
  if (tid == 0) pl.chunk = chunk;
}

// The walk over items from the plan's start: every warp keeps its own copy.
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
// By whole warps.
__device__ __forceinline__ Walk walk_start(const AttnArgs& a, const Plan& pl) {
  const int lane = threadIdx.x & 31;
  Walk w;
  w.b = pl.b;
  w.q = load_request(a.p, w.b);
  w.nq = query_tiles(a.shape, w.q);
  const long long each = head_cost(a.shape, w.q, lane);
  w.h = (int)quotient(pl.off, each);
  long long rest = pl.off - w.h * each;
  w.qt = 0;
  if (w.nq > 1)
    for (int i0 = 0; i0 < w.nq; i0 += 32) {
      const int i = i0 + lane;
      const long long c = i < w.nq ? tile_cost(a.shape, tile_span(a.shape, w.q, i)) + a.shape.lead : 0;
      long long incl = c;
      for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(~0u, incl, o);
        if (lane >= o) incl += v;
      }
      const unsigned past = __ballot_sync(~0u, incl > rest);
      if (past) {
        const int src = __ffs(past) - 1;
        w.qt = i0 + src;
        rest -= __shfl_sync(~0u, incl - c, src);
        break;
      }
      rest -= __shfl_sync(~0u, incl, 31);
    }
  walk_item(a, w, (int)rest);
  return w;
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

// Launch configuration of an attention kernel of `ctas` resident CTAs, and the combine step behind it.
void attention_config(cudaLaunchConfig_t* cfg, cudaLaunchAttribute* attr, int ctas, int threads, int smem,
                      cudaStream_t s);
cudaError_t launch_combine(const AttnArgs& a, int D, cudaStream_t s);

// The tensor-core kernel (paged_attn_tc.cu): whether it can take the call, and its launch with 256
// (`pair`) or 128 query rows per item.
bool attention_tc_fits(const AttnArgs& a, int D, bool fp8);
cudaError_t launch_attention_tc(const AttnArgs& a, int D, bool pair, cudaStream_t s);

}  // namespace lowbit
