// Definitions shared by the kernels that work on a paged key/value cache: the batch and cache as
// the kernels see them, host-side validation, and the schedule that splits attention work.
#pragma once

#include "common.cuh"

namespace lowbit {

constexpr int kMaxHeadDim = 256;
constexpr int kMaxPageSize = 1024;
constexpr int kMaxBatch = 1 << 16;
constexpr int kMaxTokens = 1 << 24;

// lowbit_paged_batch and lowbit_paged_cache with what the host has derived.
struct PagedArgs {
  const int32_t* cu_q;
  const int32_t* kv_lens;
  const int32_t* table;
  long long table_stride;
  int B, T, width;             // requests, rows of the token arrays, columns of the block table
  uint8_t* k;
  uint8_t* v;
  long long page_stride, token_stride, head_stride;  // bytes
  int pages, page_shift, page_mask;
  int Hk;
  const float* k_scale;
  const float* v_scale;
  int* err;
};

// Checks of the two descriptors; fills `a` (all but err).
lowbit_status make_paged_args(const lowbit_paged_batch* batch, const lowbit_paged_cache* cache,
                              PagedArgs* a);

// First row, new tokens and whole length of request b.  A request that the arrays describe
// inconsistently (decreasing offsets, rows past T, more keys than its pages hold) counts as one
// without tokens, and the device error word says so.
struct Request {
  int row0, n, kv;
};
__device__ __forceinline__ Request check_request(const PagedArgs& a, int from, int to, int kv) {
  Request r = {from, to - from, kv};
  if (r.row0 < 0 || r.n < 0 || r.row0 > a.T - r.n || r.kv < 0 ||
      (long long)r.kv > ((long long)a.width << a.page_shift)) {
    record_error(a.err, LOWBIT_ERR_INVALID_ARG);
    r.row0 = r.n = r.kv = 0;
  }
  return r;
}
__device__ __forceinline__ Request load_request(const PagedArgs& a, int b) {
  return check_request(a, a.cu_q[b], a.cu_q[b + 1], a.kv_lens[b]);
}

// ---------------------------------------------------------------------- attention schedule
// A work item is (request, key/value head, tile of R query rows); query row r of a request is
// token r / G, head r % G of the group, so the rows that share keys share a tile.  An item costs
// its number of key tiles of BN, counted from the tile that holds the first key any of its rows
// sees, and `lead` tiles more for what every item pays (queries in, outputs out, an empty
// pipeline).  Items are laid end to end (request, then head, then query tile), each with its lead
// first, and the whole length is cut into equal chunks, one per CTA: ragged batches balance by
// construction, and an item whose tiles a cut goes through is finished by the combine kernel from
// its pieces' (maximum, sum, output).  A batch of 64 requests of 1 to 16,384 keys, half of them
// below 128, took 160 us without the lead (some CTAs got 23 items of one tile).
struct Span {
  int lo, hi;  // keys [lo, hi) that some row of the tile sees; lo == hi: none
};
struct ItemShape {
  int G;
  uint32_t g_inv;         // floor(2^32 / G), at most 2^32 - 1
  int r_shift, bn_shift;  // R = 1 << r_shift rows, BN = 1 << bn_shift keys
  int lead;
  int causal, window;
};
// r / G: the product with floor(2^32 / G) is short of it by less than one.
__device__ __forceinline__ int token_of(const ItemShape& s, int r) {
  const uint32_t q = __umulhi((uint32_t)r, s.g_inv);
  return (int)(q + ((uint32_t)r - q * s.G >= (uint32_t)s.G ? 1u : 0u));
}
// First key that the window leaves a token at `pos`.  More new tokens than keys put the first ones at positions
// below zero, where window and position together may pass 32 bits: they lose no key to the window.
__device__ __forceinline__ int first_key(const ItemShape& s, int pos) {
  return s.window ? max(0, max(pos + 1, 0) - s.window) : 0;
}
__device__ __forceinline__ Span tile_span(const ItemShape& s, const Request& q, int qt) {
  const int r0 = qt << s.r_shift, r1 = min(r0 + (1 << s.r_shift), q.n * s.G) - 1;
  Span k;
  k.hi = s.causal ? max(0, min(q.kv, q.kv - q.n + token_of(s, r1) + 1)) : q.kv;
  k.lo = first_key(s, q.kv - q.n + token_of(s, r0));
  if (k.lo >= k.hi) k.lo = k.hi = 0;
  return k;
}
// Key tiles of the span; a tile without visible keys still costs one, which writes its zeros.
__device__ __forceinline__ int tile_cost(const ItemShape& s, const Span& k) {
  return max(1, ((k.hi - 1) >> s.bn_shift) - (k.lo >> s.bn_shift) + 1);
}
__device__ __forceinline__ int query_tiles(const ItemShape& s, const Request& q) {
  return (int)(((long long)q.n * s.G + (1 << s.r_shift) - 1) >> s.r_shift);
}

}  // namespace lowbit
