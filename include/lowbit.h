/*
 * lowbit.h -- C ABI of liblowbit.so: weight-only low-bit GEMV/GEMM for speculative decoding
 * on GB300 (sm_103a).
 *
 * The library multiplies bf16 activation rows X[M][K] (M = 1 for plain decoding, M = 16 for
 * verifying a 16-token draft block) by a weight matrix W[N][K] stored in one of two low-bit
 * formats, and can fuse the vocabulary argmax and greedy draft acceptance into the LM-head
 * multiply.  Y = X * W^T is bf16 [M][N], accumulated in fp32.
 *
 * Conventions shared by every entry point
 *   - Pointers are DEVICE pointers unless the comment says otherwise.  bf16 and fp16 arrays
 *     are passed as uint16_t bit patterns.  Arrays are dense and row-major.
 *   - `stream` is a cudaStream_t passed as void* (NULL = the legacy default stream).  Every
 *     call only enqueues work on `stream` and returns; results are ready when the stream is.
 *   - The caller owns and allocates all memory; the library never allocates device memory.
 *   - Arguments are validated on the host before anything is enqueued; on error nothing is
 *     enqueued and no output is touched.  A CUDA launch error returns LOWBIT_ERR_CUDA.
 *   - K must be a multiple of 128 (the quantisation group).  N >= 1 is arbitrary.
 *   - Packed weight buffers start with a 128-byte header (magic, format, N, K, P).  Kernels
 *     check it against the call's arguments; on a mismatch they write no output and record
 *     LOWBIT_ERR_INVALID_ARG in a per-device error word that lowbit_device_error() returns.
 *     The M = 1 kernels may start reading weights before the header has been checked, but
 *     only when the host has verified that the payload the arguments describe lies inside
 *     the device allocation that contains `packed`; otherwise nothing but the header is read
 *     on a mismatch.  lowbit_validate_packed() checks a header synchronously.
 *   - Multiplies are launched with programmatic dependent launch: they request their packed
 *     weights (header included) before waiting for the preceding kernel on the stream, and
 *     read activations / write outputs only after that wait.  So the kernel immediately
 *     before a multiply on the same stream must not write that multiply's packed buffer.
 *     lowbit_pack_int4, lowbit_pack_binplane and lowbit_pack_sa end with an empty kernel,
 *     which makes "pack, then multiply" on one stream safe.
 *   - No C++ exception crosses this interface.
 */
#ifndef LOWBIT_H
#define LOWBIT_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum lowbit_status {
  LOWBIT_OK = 0,
  LOWBIT_ERR_INVALID_ARG = 1, /* null pointer, negative size, wrong packed header */
  LOWBIT_ERR_SHAPE = 2,       /* K % 128 != 0, M outside 1..32, P outside 1..8, N < 1 */
  LOWBIT_ERR_ALIGN = 3,       /* a pointer is not 16-byte aligned */
  LOWBIT_ERR_WORKSPACE = 4,   /* workspace missing or smaller than lmhead_workspace_bytes() */
  LOWBIT_ERR_TIMEOUT = 5,     /* a bounded in-kernel wait gave up (recorded on the device) */
  LOWBIT_ERR_CUDA = 6         /* a CUDA runtime call or launch failed */
} lowbit_status;

/* Short English description of a status code (static string, never NULL). */
const char* lowbit_status_string(int status);

/* Library version as MAJOR*10000 + MINOR*100 + PATCH. */
int lowbit_version(void);

/* ------------------------------------------------------------------------------------------
 * Sizes (host-only, no CUDA call).  Return 0 for invalid shapes.
 */

/* Bytes of a packed INT4 buffer: 128-byte header + ceil(N/128)*128 rows of K/2 code bytes and
 * K/64 scale bytes.  For N a multiple of 128 the payload is exactly N*K/2 + N*K/64 bytes. */
size_t lowbit_int4_packed_bytes(int N, int K);

/* Bytes of a packed binary-plane buffer: header + ceil(N/128)*128 rows of P*K/8 sign bytes and
 * P*K/64 plane-scale bytes. */
size_t lowbit_binplane_packed_bytes(int P, int N, int K);

/* Bytes of a packed buffer of the deployed ShiftAdd format (lowbit_pack_sa): header +
 * ceil(N/128)*128 rows of P*K/8 sign bytes, P*K/G code bytes and K/128 bytes of d.  0 unless
 * K % 256 == 0, 1 <= P <= 8 and G is 64, 128 or 256. */
size_t lowbit_sa_packed_bytes(int P, int G, int N, int K);

/* Bytes of a packed NVFP4 buffer (lowbit_pack_nvfp4): header + ceil(N/128)*128 rows of K/2
 * code bytes and K/16 scale bytes. */
size_t lowbit_nvfp4_packed_bytes(int N, int K);

/* Bytes of a packed Q8 buffer (lowbit_pack_q8): header + ceil(N/128)*128 rows of K code bytes
 * and K/16 scale bytes (one fp16 per 32 inputs). */
size_t lowbit_q8_packed_bytes(int N, int K);

/* Bytes of the workspace lmhead_argmax_verify() needs (independent of N and K). */
size_t lmhead_workspace_bytes(int M, int N, int K);

/* ------------------------------------------------------------------------------------------
 * Offline repack (Efficient-Qwen report, section 2.1: codes rounded onto the INT4 grid under
 * frozen symmetric per-group scales, served as W4A16; ShiftAddQwen README, "Format" and
 * "Layout": binary planes with per-group scales and bit-exact packing).
 */

/* Repack canonical INT4 weights into the kernel layout.
 *   codes  : int8 [N][K], values in [-8, 7] (q of w = s*q); 16-byte aligned.  Values outside
 *            the range are out of contract: they are stored modulo 16.
 *   scales : fp16 [N][K/128], one symmetric scale per row and group of 128 inputs.
 *   packed : lowbit_int4_packed_bytes(N, K) bytes, 16-byte aligned; fully overwritten.
 * Layout of `packed` (little-endian): the header (magic 0x3242574C, format 1, version 2), then
 * rows in tiles of 128 (padding rows hold q = 0, scale 0).  Tile t and group g (inputs
 * 128g..128g+127) own one contiguous 8448-byte block at 128 + (t*(K/128) + g)*8448: for chunk
 * c = 0..3 and row r = n % 128 the 16 bytes at c*2048 + r*16 are four u32 words, word i
 * holding k = 128g + 32c + 8i + 2p + o (p = 0..3, o = 0..1) as the nibble q + 8 at bit
 * 4p + 16o; the fp16 scale s[n][g] sits at 8192 + r*2. */
lowbit_status lowbit_pack_int4(const int8_t* codes, const uint16_t* scales, int N, int K,
                               void* packed, void* stream);

/* Repack canonical binary planes (w = sum_p alpha_p * b_p, b in {-1,+1}).
 *   signbits : uint8 [P][N][K/8]; bit j (LSB first) of byte i is input k = 8i + j; 1 = +1.
 *   alpha    : fp16 [P][N][K/128], one scale per plane, row and group of 128 inputs.
 *   packed   : lowbit_binplane_packed_bytes(P, N, K) bytes, 16-byte aligned.
 * Layout: header (format 2), then tiles of 128 rows; tile t and group g own one contiguous
 * block of 2304*P bytes at 128 + (t*(K/128) + g)*2304*P: for plane p and row r = n % 128 the
 * 16 bytes at p*2048 + r*16 hold the 128 signs of k = 128g.. as four u32 words, word w
 * covering k0 = 128g + 32w with bit i = sign of k0 + 2i and bit 16 + i = sign of k0 + 2i + 1;
 * alpha[p][n][g] (fp16) sits at 2048*P + (p*128 + r)*2. */
lowbit_status lowbit_pack_binplane(const uint8_t* signbits, const uint16_t* alpha, int P, int N,
                                   int K, void* packed, void* stream);

/* Repack the deployed ShiftAdd format (ShiftAddQwen README, "Format": per super-block of 256
 * weights along the input dimension, Q sign planes, one u8 scale code per plane and group of G
 * weights, one fp16 scale d; alpha = d * a), so that
 *   w[n][k] = d[n][k/256] * sum_p a[p][n][k/G] * b[p][n][k],   b in {-1, +1}.
 *   signbits : uint8 [P][N][K/8], 16-byte aligned; bit j (LSB first) of byte i is input 8i + j;
 *              1 = +1.
 *   codes    : uint8 [P][N][K/G], the scale codes a (any alignment).
 *   d        : fp16 [N][K/256] (2-byte aligned).
 *   packed   : lowbit_sa_packed_bytes(P, G, N, K) bytes, 16-byte aligned; fully overwritten.
 *   1 <= P <= 8, G in {64, 128, 256}, K % 256 == 0 (else LOWBIT_ERR_SHAPE).
 * Layout: header (format 3, group field = G), then tiles of 128 rows; tile t and super-block
 * j (inputs 256j..256j+255) own one contiguous block of B = 4096P + 128P(256/G) + 256 bytes at
 * 128 + (t*(K/256) + j)*B: for plane p, half h and row r = n % 128 the 16 bytes at
 * p*4096 + h*2048 + r*16 hold the signs of k = 256j + 128h.. as four u32 words (word w covers
 * k0 = 256j + 128h + 32w: bit i = sign of k0 + 2i, bit 16 + i = sign of k0 + 2i + 1); the code
 * a[p][n][g] sits at 4096P + (p*(256/G) + g - j*(256/G))*128 + r, and d[n][j] (fp16) at
 * 4096P + 128P(256/G) + r*2.  Padding rows hold zero signs, codes and d. */
lowbit_status lowbit_pack_sa(const uint8_t* signbits, const uint8_t* codes, const uint16_t* d,
                             int P, int G, int N, int K, void* packed, void* stream);

/* Repack NVFP4 weights, the draft-head format of the small-vocabulary MTP study (section 3.3:
 * trim the head to the most used 32,768 tokens, quantise to NVFP4):
 *   w[n][k] = g * e4m3(scales[n][k/16]) * e2m1(code of k in row n).
 *   codes  : uint8 [N][K/2], 16-byte aligned; byte i holds inputs 2i (low nibble) and 2i + 1
 *            as 4-bit E2M1 codes (sign, two exponent bits with bias 1, one mantissa bit).
 *   scales : uint8 [N][K/16], E4M3 bytes (sign, four exponent bits with bias 7, three mantissa
 *            bits; 0x7F / 0xFF are NaN).       g : the fp32 tensor scale.
 *   packed : lowbit_nvfp4_packed_bytes(N, K) bytes, 16-byte aligned; fully overwritten.
 * Layout: header (format 4, the fp32 bits of g at byte 56), then per (tile t of 128 rows, group
 * j of 128 inputs) one block of 9216 bytes at 128 + (t*(K/128) + j)*9216: for chunk c = 0..3 and
 * row r the 16 code bytes of inputs 128j + 32c .. +31 at c*2048 + r*16, then the scale byte of
 * inputs 128j + 16i .. +15 at 8192 + i*128 + r (i = 0..7). */
lowbit_status lowbit_pack_nvfp4(const uint8_t* codes, const uint8_t* scales, float g, int N, int K,
                                void* packed, void* stream);

/* Repack Q8 weights, the 8-bit arm of the small-vocabulary MTP study's trimmed draft head
 * (section 3.3; read as the llama.cpp Q8_0 recipe the ShiftAddQwen README names):
 *   w[n][k] = d[n][k/32] * q[n][k].
 *   codes  : int8 [N][K] (two's complement, the full range -128..127), 16-byte aligned.
 *   scales : fp16 [N][K/32], 2-byte aligned.
 *   packed : lowbit_q8_packed_bytes(N, K) bytes, 16-byte aligned; fully overwritten.
 * Layout: header (format 5), then per (tile t of 128 rows, group g of 128 inputs) one block of
 * 17408 bytes at 128 + (t*(K/128) + g)*17408: for chunk c = 0..7 and row r the 16 code bytes of
 * inputs 128g + 16c .. +15 at c*2048 + r*16, then d[n][4g + j] (fp16) at 16384 + j*256 + r*2
 * (j = 0..3).  Padding rows hold code 0 and scale 0. */
lowbit_status lowbit_pack_q8(const int8_t* codes, const uint16_t* scales, int N, int K, void* packed,
                             void* stream);

/* Synchronous check (copies the 128-byte header to the host after synchronising `stream`)
 * that `packed` holds format `format` (1 = INT4, 2 = binary planes, 3 = sa, 4 = NVFP4, 5 = Q8)
 * with these N, K and, for formats 2 and 3, P (pass 0 for the others).  For the sa format the
 * header's code group G is only checked to be 64, 128 or 256.
 * Returns LOWBIT_OK or LOWBIT_ERR_INVALID_ARG. */
lowbit_status lowbit_validate_packed(const void* packed, int format, int P, int N, int K,
                                     void* stream);

/* ------------------------------------------------------------------------------------------
 * Multiplies.
 */

/* Y = X * W^T for symmetric per-group INT4 weights (Efficient-Qwen report, section 2.1):
 *   y[m][n] = sum_g s[n][g] * sum_{k in g} q[n][k] * x[m][k], fp32 accumulation across
 *   groups, each output rounded once to bf16 (nearest, ties to even).
 *   X : bf16 [M][K], 16-byte aligned.   packed : from lowbit_pack_int4(N, K).
 *   Y : bf16 [M][N], written in full.   1 <= M <= 32.
 * M <= 2 runs the streaming kernel (path 1 also at M = 3, 4): each run of 64 activations of a
 * row is held as int16 times one power of two (exact for every activation within a factor 2^7
 * of the run's largest, otherwise rounded to a multiple of 2^-15 of that largest) and the
 * products within a run are summed exactly in integers; a non-finite activation makes every
 * output of its row NaN.
 * M >= 3 runs the skinny GEMM on the warp-level tensor-core MMA (exact bf16 q times the bf16
 * activations, fp32 accumulation within a group, then s times the group's sum added in fp32). */
lowbit_status lowbit_gemm_int4(const uint16_t* X, const void* packed, int M, int N, int K,
                               uint16_t* Y, void* stream);

/* One multiply of a grouped call: the arguments of lowbit_gemm_int4 other than M. */
typedef struct lowbit_gemm_desc {
  const uint16_t* X;    /* bf16 [M][K], device, 16-byte aligned */
  const void* packed;   /* from lowbit_pack_int4(N, K), device, 16-byte aligned */
  uint16_t* Y;          /* bf16 [M][N], device */
  int N;
  int K;
} lowbit_gemm_desc;

/* Several independent INT4 multiplies with a common M (for example the q, k and v projections
 * of a decoder layer, which read the same activations), each with the contract and rounding
 * of lowbit_gemm_int4.  They share ONE launch (the streaming kernel at M <= 2, the warp-MMA
 * GEMM above), so the launch, pipeline fill and drain are paid once for the group instead of
 * once per matrix.
 *   descs : HOST array of `count` descriptors, 1 <= count <= 8; read during the call only.
 *   The multiplies must be independent: no Y may overlap any X, packed buffer or other Y of
 *   the group.  Every descriptor is validated before anything is enqueued. */
lowbit_status lowbit_gemm_int4_grouped(const lowbit_gemm_desc* descs, int count, int M,
                                       void* stream);
/* The same with the kernel family forced: `path` as lowbit_gemm_int4_path (1: the streaming
 * kernel, M <= 4, else LOWBIT_ERR_SHAPE). */
lowbit_status lowbit_gemm_int4_grouped_path(const lowbit_gemm_desc* descs, int count, int M,
                                            int path, void* stream);

/* Y = X * W^T for binary-plane weights (ShiftAddQwen README, "Method" and "Format"):
 *   y[m][n] = sum_p sum_g alpha[p][n][g] * sum_{k in g} b[p][n][k] * x[m][k].
 *   Shapes and rounding as lowbit_gemm_int4; packed from lowbit_pack_binplane(P, N, K).
 *   M = 1 runs the table-driven streaming kernel; M >= 2 the warp-level MMA on exact +-1
 *   bf16 fragments, one MMA set per plane, alpha applied per (plane, group) in fp32. */
lowbit_status lowbit_gemm_binplane(const uint16_t* X, const void* packed, int P, int M, int N,
                                   int K, uint16_t* Y, void* stream);

/* Y = X * W^T for the deployed ShiftAdd format (ShiftAddQwen README, "Format"):
 *   y[m][n] = sum_j d[n][j] * sum_p sum_{g in j} a[p][n][g] * sum_{k in g} b[p][n][k] * x[m][k],
 *   fp32 accumulation, each output rounded once to bf16.  X, Y as lowbit_gemm_int4,
 *   1 <= M <= 32; packed from lowbit_pack_sa(P, G, N, K); K % 256 == 0.  M = 1 runs the
 *   streaming mat-vec (per plane a table-driven sign-select-and-add, one scale per group);
 *   M >= 2 runs the warp-level MMA on exact +-1 fragments, each code group's sums scaled by
 *   d * a in fp32 (path 2: the tcgen05 GEMM, weights written as +-a in bf16).
 *   The header (format 3, P, N, K, G) is checked on the device as for the other formats. */
lowbit_status lowbit_gemm_sa(const uint16_t* X, const void* packed, int P, int G, int M, int N,
                             int K, uint16_t* Y, void* stream);

/* Y = X * W^T for NVFP4 weights (packed by lowbit_pack_nvfp4), 1 <= M <= 32, g applied in fp32
 * per output, each output rounded once to bf16.  M = 1 runs the streaming mat-vec (int16
 * activations, as the INT4 kernel); M >= 2 the tensor cores (each weight written to tensor
 * memory as the exact bf16 of e2m1 * e4m3).  (The draft step itself needs only the argmax:
 * lowbit_draft_argmax, which chooses its kernel the same way.) */
lowbit_status lowbit_gemm_nvfp4(const uint16_t* X, const void* packed, int M, int N, int K,
                                uint16_t* Y, void* stream);

/* Y = X * W^T for Q8 weights (lowbit_pack_q8), 1 <= M <= 32, fp32 accumulation, each output
 * rounded once to bf16.  M = 1 streams the weights (activations held as int16 per run of 64 as
 * in lowbit_gemm_int4; integer dot products against the signed codes, each run of 32 scaled
 * by its d in fp32); M >= 2 runs the warp-level MMA (each code written exactly as bf16, the
 * MMA sums of every 32 inputs scaled by d in fp32).  path: 0 the library's choice, 1 the
 * streaming kernel (M = 1 only, else LOWBIT_ERR_SHAPE), 3 the warp-level MMA. */
lowbit_status lowbit_gemm_q8(const uint16_t* X, const void* packed, int M, int N, int K, uint16_t* Y,
                             void* stream);
lowbit_status lowbit_gemm_q8_path(const uint16_t* X, const void* packed, int M, int N, int K,
                                  uint16_t* Y, int path, void* stream);

/* The draft step of a trimmed Q8 head: as lowbit_draft_argmax (ids[m] = id_map[argmax], fp32
 * logits never rounded, lowest row on ties, the same workspace rules), for a head packed by
 * lowbit_pack_q8.  M = 1 streams; M >= 2 runs the warp-level MMA. */
lowbit_status lowbit_draft_argmax_q8(const uint16_t* H, const void* packed_head, int M, int N, int K,
                                     const int32_t* id_map, int32_t* ids, void* workspace,
                                     size_t ws_bytes, void* stream);

/* Draft step of a trimmed NVFP4 head (small-vocabulary MTP study, section 3.3: the draft head
 * keeps the 32,768 most used rows of the vocabulary; its winners are mapped back to the full
 * vocabulary before verification):
 *   H      : bf16 [M][K] hidden rows, 1 <= M <= 32.   packed_head : from lowbit_pack_nvfp4.
 *   id_map : int32 [N], the full-vocabulary id of each head row, or NULL (ids are rows).
 *   ids    : int32 [M] out: id_map[argmax_n logit[m][n]], argmax over fp32 logits (never
 *            rounded), lowest row on ties.  Logits are not written anywhere.
 *   workspace : as lmhead_argmax_verify (lmhead_workspace_bytes, zero-filled once, left zero;
 *            calls sharing one must not overlap). */
lowbit_status lowbit_draft_argmax(const uint16_t* H, const void* packed_head, int M, int N, int K,
                                  const int32_t* id_map, int32_t* ids, void* workspace,
                                  size_t ws_bytes, void* stream);

/* LM-head verify step (small-vocabulary MTP study, section 3.3: full-vocabulary verification;
 * DFlash summary, section 4.1: tau in [1, gamma + 1]; Efficient-Qwen report, section 2.2).
 *   H        : bf16 [M][K] hidden rows of one verify block, 2 <= M <= 32 (M - 1 drafts).
 *   packed_head : INT4 head from lowbit_pack_int4(N, K), N = vocabulary rows.
 *   draft    : int32 [M-1] draft token ids for positions 1..M-1 of the block.
 *   argmax   : int32 [M] out: a[m] = argmax_n logit[m][n] over fp32 logits (never rounded),
 *              lowest index on ties.  Logits are not written anywhere.
 *   n_accept : int32 [1] out: n = largest j <= M-1 with draft[i] == a[i] for all i < j.
 *   bonus    : int32 [1] out: a[n], the target's token after the accepted prefix.
 *   workspace: lmhead_workspace_bytes(M, N, K) bytes, 16-byte aligned, ZERO-FILLED ONCE
 *              before first use; every call leaves it zero again.  Calls that share a
 *              workspace must not overlap on the GPU.  After a failed call, re-zero it. */
lowbit_status lmhead_argmax_verify(const uint16_t* H, const void* packed_head, int M, int N,
                                   int K, const int32_t* draft, int32_t* argmax,
                                   int32_t* n_accept, int32_t* bonus, void* workspace,
                                   size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------------------------------
 * Row-sharded LM head: verification with the vocabulary split across GPUs (small-vocabulary MTP
 * study, section 3.3: drafts are verified against the full vocabulary; DFlash summary, section
 * 4.1: greedy prefix acceptance).  Each GPU holds a contiguous slice of the head's rows, packed
 * on its own with lowbit_pack_int4; the only exchange is W * M 64-bit keys.
 *
 *   1. On every GPU: lmhead_argmax_partial on its slice -> keys_out[M].
 *   2. The caller all-gathers the keys of all W GPUs into keys[W][M] (shard order is free).
 *   3. On every GPU: lmhead_accept_keys(keys, W, ...) -> the same argmax, n_accept and bonus
 *      as lmhead_argmax_verify on the whole head (argmax over fp32 logits, lowest row on ties).
 *
 * Key of a token: (order-preserving bits of its best fp32 logit in the slice) << 32 |
 * (0xFFFFFFFF - global row), so that a larger key is a larger logit and, between equal logits,
 * the lower row; the maximum over slices is the full head's winner.
 */

/* Step 1.  packed_shard: lowbit_pack_int4 of rows row_offset .. row_offset + N - 1 of the head
 * (N rows, K inputs); H: bf16 [M][K], 1 <= M <= 32; row_offset >= 0 and row_offset + N < 2^31.
 *   keys_out : uint64 [M] out, 8-byte aligned (device).
 *   workspace: as lmhead_argmax_verify (lmhead_workspace_bytes(2, N, K), zero once, left zero).
 * Runs the default verify kernel (warp-level MMA); logits are never written. */
lowbit_status lmhead_argmax_partial(const uint16_t* H, const void* packed_shard, int M, int N, int K,
                                    int row_offset, uint64_t* keys_out, void* workspace,
                                    size_t ws_bytes, void* stream);

/* Step 3.  keys: uint64 [W][M] (device, 8-byte aligned), every shard's keys_out; draft: int32
 * [M-1]; argmax: int32 [M] out; n_accept, bonus: int32 [1] out, as lmhead_argmax_verify.
 * 2 <= M <= 32, W >= 1.  One small kernel. */
lowbit_status lmhead_accept_keys(const uint64_t* keys, int W, int M, const int32_t* draft,
                                 int32_t* argmax, int32_t* n_accept, int32_t* bonus, void* stream);

/* ------------------------------------------------------------------------------------------
 * Between the products: a paged key/value cache, attention over it, and sampling.
 *
 * A decoder layer's q, k and v products are followed by lowbit_kv_append (rotary positions, keys
 * and values into the cache) and lowbit_paged_attention (the new tokens over the cache), whose
 * output feeds the o product.  Both take the same description of the batch, on the device, so a
 * captured graph serves steps whose lengths differ.
 */

/* Which rows of the token arrays belong to which request.  Row cu_q[b] + i (0 <= i < n,
 * n = cu_q[b+1] - cu_q[b]) is new token i of request b; its position is kv_lens[b] - n + i,
 * where kv_lens[b] counts all keys of the request, the new ones included.  Position p is in
 * slot p % page_size of page block_table[b][p / page_size].  n = 0 is an idle request; rows past
 * cu_q[B] belong to nobody and are neither read nor written.
 * The kernels check what they read: a request whose cu_q decreases or passes T, or whose
 * kv_lens is negative or passes width * page_size, is skipped; a token whose page is outside
 * 0..num_pages-1 is not appended, and a key in such a page is read as zeros.  Each records
 * LOWBIT_ERR_INVALID_ARG in the device error word (lowbit_kv_append looks at the lengths of requests with
 * rows only).  Where offsets decrease, requests may claim the same row: it is appended for the first
 * of them, and attention writes it for each. */
typedef struct lowbit_paged_batch {
  const int32_t* cu_q;         /* device, [B + 1] */
  const int32_t* kv_lens;      /* device, [B] */
  const int32_t* block_table;  /* device, [B][table_stride], `width` entries used per row */
  int64_t table_stride;        /* elements, >= width */
  int B;                       /* requests, 1..65536 */
  int T;                       /* rows of the token arrays, 0..2^24 */
  int width;                   /* pages a request may have, >= 1 */
} lowbit_paged_batch;

#define LOWBIT_CACHE_BF16 0 /* keys and values as bf16 */
#define LOWBIT_CACHE_E4M3 1 /* as e4m3, times k_scale / v_scale of the head */

/* A cache of num_pages pages of page_size slots (a power of two, 1..1024; at least 2 with e4m3
 * heads of 64) for `heads` key/value heads of head_dim 64, 128 or 256.  Element (page, slot, head, d) of k (and v) is at
 * page * page_stride + slot * token_stride + head * head_stride + d: strides in elements,
 * positive multiples of 16 bytes below 2^39, so both orders of heads and slots fit.  The two arrays are
 * 16-byte aligned and share the strides. */
typedef struct lowbit_paged_cache {
  void* k;
  void* v;
  int64_t page_stride, token_stride, head_stride;
  int num_pages, page_size, heads, head_dim;
  int dtype;                   /* LOWBIT_CACHE_BF16 or LOWBIT_CACHE_E4M3 */
  const float* k_scale;        /* device, [heads], or NULL for 1 (e4m3 only; else NULL) */
  const float* v_scale;
} lowbit_paged_cache;

/* Rotary positions on the new tokens' queries and keys, and keys and values into the cache.
 *   q : bf16 [T][Hq][D] or NULL, k, v : bf16 [T][heads][D]; D = head_dim; the token strides
 *       q_stride, k_stride, v_stride are in elements (multiples of 8; heads are dense), so the
 *       three may be column ranges of one product's output.  16-byte aligned.
 *   rope : fp32 [rope_rows][rot], 16-byte aligned: row p holds cos then sin (rot/2 each) of
 *       position p.  rot is a multiple of 16, at most D; rot = 0 (rope NULL) rotates nothing.
 *       Element pair j is (x[j], x[j + rot/2]), or (x[2j], x[2j + 1]) when `interleaved`:
 *         a' = a cos - b sin,  b' = b cos + a sin   (fp32, every product and sum rounded).
 *       Elements from rot on, and values, are not rotated.
 *   q_out : bf16 [T][Hq][D], dense, 16-byte aligned (NULL with q).  It may be q itself where q is dense
 *       too; any other overlap with a row of q, k or v is refused (LOWBIT_ERR_INVALID_ARG).
 *   In the cache a bf16 element is rounded once; an e4m3 element is x / scale rounded to
 *   nearest-even and clipped to +-448 (NaN stays NaN).  Slots of other positions keep their
 *   contents.  A position at or past rope_rows is not appended and recorded in the device
 *   error word. */
lowbit_status lowbit_kv_append(const uint16_t* q, int64_t q_stride, const uint16_t* k,
                               int64_t k_stride, const uint16_t* v, int64_t v_stride, int Hq,
                               const float* rope, int rope_rows, int rot, int interleaved,
                               const lowbit_paged_batch* batch, const lowbit_paged_cache* cache,
                               uint16_t* q_out, void* stream);

/* lowbit_kv_append with a norm of each head of q and k before the rotation:
 *   y = x * w / sqrt(sum_d x_d^2 / D + eps)   over the head's D elements,
 * in fp32 from the bf16 elements up to the one rounding of what is stored (q_out, or the cache as there).
 *   q_weight, k_weight : fp32 [D], 16-byte aligned; NULL leaves q's, or k's, heads as they are (q_weight
 *       is NULL where q is).  Values are never normalised.
 *   eps : finite, >= 0; with 0, a head of zeros becomes NaN.
 *   The squares are summed in fp32, so a head whose sum of squares passes 3.4e38 (elements past 2^60) becomes
 *   zeros, or NaN where it holds an infinity.  Rows of nobody may be read here, whatever they hold, but reach nothing.
 *   All else is as in lowbit_kv_append. */
lowbit_status lowbit_kv_append_norm(const uint16_t* q, int64_t q_stride, const uint16_t* k,
                                    int64_t k_stride, const uint16_t* v, int64_t v_stride, int Hq,
                                    const float* q_weight, const float* k_weight, float eps,
                                    const float* rope, int rope_rows, int rot, int interleaved,
                                    const lowbit_paged_batch* batch,
                                    const lowbit_paged_cache* cache, uint16_t* q_out,
                                    void* stream);

/* Bytes of lowbit_paged_attention's workspace for up to T rows and B requests of Hq query and
 * Hk key/value heads of D (0 for invalid shapes): enough for the pieces of the largest grid, so it
 * depends on D alone (21, 40 or 80 MB for heads of 64, 128 or 256); one serves every call on a stream. */
size_t lowbit_paged_attention_workspace_bytes(int T, int B, int Hq, int Hk, int D);

/* Attention of every request's new tokens over its cached keys, grouped heads (query head h
 * reads key/value head h / (Hq / heads)):
 *   out[t][h] = sum_j softmax_j(scale * q[t][h] . k_j) v_j over the keys j the token sees:
 *   j < kv_lens[b]; j <= its position when `causal`; j > its position - window when window > 0.
 *   A token that sees no key gets zeros, and -inf as lse.
 *   Requests should be alike in new tokens: the kernel is chosen by their average (T / B).  width *
 *   page_size is at most 2^31 - 256 here.
 *   q   : bf16 [T][Hq][D], token stride q_stride (elements, a multiple of 8), 16-byte aligned.
 *   out : bf16 [T][Hq][D] dense, 16-byte aligned.    lse : fp32 [T][Hq] or NULL: the natural
 *   logarithm of the softmax's denominator (log sum_j exp(scale * q . k_j)).
 *   workspace : lowbit_paged_attention_workspace_bytes() bytes, 16-byte aligned, any contents.
 *   Scores, softmax statistics and outputs are held in fp32; the softmax weights enter their
 *   product with v rounded to bf16 (bf16 cache) or fp16 (e4m3 cache), 2^-8 or 2^-11 of themselves at
 *   most (over an e4m3 cache, weights under 2^-21 of the row's largest by 2^-32 of that one).  Slots
 *   outside a request's span are never used, whatever they hold.  A key that the mask hides from a
 *   token does not reach it, whatever it holds; a non-finite value v inside the span may (0 * inf is NaN), through the
 *   up to 256 rows of one request and head that are computed together.  The result does not depend
 *   on timing: the same call gives the same bits. */
lowbit_status lowbit_paged_attention(const uint16_t* q, int64_t q_stride, int Hq,
                                     const lowbit_paged_batch* batch,
                                     const lowbit_paged_cache* cache, float scale, int causal,
                                     int window, uint16_t* out, float* lse, void* workspace,
                                     size_t ws_bytes, void* stream);

/* Bytes of lowbit_prefix_attention's workspace for up to T rows and B requests of Hq query and Hk
 * key/value heads of D (0 for invalid shapes): twice lowbit_paged_attention's, and 8 D + 48 for each row
 * and query head, up to 96 (heads of 256: 48) for each request and key/value head. */
size_t lowbit_prefix_attention_workspace_bytes(int T, int B, int Hq, int Hk, int D);

/* lowbit_paged_attention (without a window) for requests whose first pages are the same ones: a long system
 * prompt, a document that many ask about, several answers to one prompt.  The shared pages are read once
 * for all rows of a group of requests, instead of once for each request.
 *   cu_groups   : int32 [groups + 1] on the device: group g is the requests cu_groups[g] ..
 *                 cu_groups[g + 1] - 1; 0 first, B last.  A group may be empty, or one request.
 *   prefix_lens : int32 [groups] on the device: the first prefix_lens[g] positions of the group's
 *                 requests hold the same keys and values.  The whole pages of it are taken from the
 *                 block table row of the group's first request (which may have no new tokens; its row is
 *                 read all the same); what lies behind the last whole page each request has on its
 *                 own.  0: nothing is shared.  New tokens come after the shared positions:
 *                 kv_lens[b] - new tokens >= the length of the whole pages.
 * kv_lens and block_table describe the whole requests, as for lowbit_kv_append and lowbit_paged_attention,
 * whose result over the same arguments is this one's but for rounding.  A group or request that the arrays
 * describe inconsistently is recorded in the device error word; its rows are not written, or (where only what
 * it shares is at fault) attend to the request's own block table.  Groups are looked up by bisection: where
 * cu_groups is not ascending, other groups may be left out with the one at fault.  What a row gets that
 * several requests claim (cu_q not ascending), or a request that several groups claim, is not defined.  Pages
 * are compared by nobody: where the table rows of a group differ in the shared pages, it is not defined which
 * of them a request sees.
 * Worth it where many requests with few rows each share much (16 requests of one token and more behind
 * thousands of keys).  From about 100 rows a request on (tokens times query heads per key/value head), and
 * under block tables of 1,024 slots (for small groups 2,048; not for very many requests over e4m3, or with
 * heads of 256), lowbit_paged_attention's kernels do the work, which are as fast there.  The kernels are
 * chosen by averages (T / groups, T / B) and by the length that the block table has room for: keep it about
 * as wide as the requests need.
 *   workspace : lowbit_prefix_attention_workspace_bytes() bytes, 16-byte aligned, any contents; calls that
 *   may run at the same time need one each.
 * All else (rounding, non-finite values, alignment) is as in lowbit_paged_attention; a non-finite v in
 * the shared pages reaches the rows of the whole group. */
lowbit_status lowbit_prefix_attention(const uint16_t* q, int64_t q_stride, int Hq,
                                      const lowbit_paged_batch* batch,
                                      const lowbit_paged_cache* cache, const int32_t* cu_groups,
                                      const int32_t* prefix_lens, int groups, float scale,
                                      int causal, uint16_t* out, float* lse, void* workspace,
                                      size_t ws_bytes, void* stream);

#define LOWBIT_LOGITS_FP32 0
#define LOWBIT_LOGITS_BF16 1

/* One token per row of logits, from given uniform numbers.
 *   logits : [M][V] fp32 or bf16 (dtype), row stride row_stride elements; M >= 1, 1 <= V <= 2^19.
 *   temperature, top_p, min_p : fp32 [M], top_k : int32 [M]; NULL = 1, 1, 0, 0 (no truncation).
 *   u : fp32 [M] in [0, 1) (others are clamped, NaN counts as 0).
 *   Per row, with z the logits (NaN counts as -inf, +inf as the largest finite value):
 *     w_i = exp((z_i - max z) * (1 / temperature)) in fp32, 0 where z_i = -inf, and its mass
 *     m_i = w_i * 2^40 rounded to a whole number: all sums below are exact in 64 bits and do
 *     not depend on their order.  Temperatures below 1e-6 (or NaN) are greedy (top_k = 1);
 *     above 1e6 they count as 1e6.
 *     Tokens are ordered by larger z, then lower index.  top_k keeps the first k (k <= 0 or
 *     > V: all); top_p then keeps, of the mass S of those, the tokens whose preceding mass is
 *     below max(1, ceil(top_p * S)) (top_p >= 1: all); min_p drops those with w < min(min_p, 1).
 *     With S the kept mass, the token is the first in index order whose inclusive kept mass
 *     exceeds floor(u * S).
 *   ids     : int32 [M] out: the token (id_map[token] when id_map, int32 [V], is not NULL), or
 *             -1 for a row without a finite logit.
 *   logprob : fp32 [M] out or NULL: log(m / S) of the token (-inf with id -1).
 *   kept    : int32 [M] out or NULL: tokens of nonzero mass that remain. */
lowbit_status lowbit_sample(const void* logits, int dtype, int64_t row_stride, int M, int V,
                            const float* temperature, const int32_t* top_k, const float* top_p,
                            const float* min_p, const float* u, const int32_t* id_map,
                            int32_t* ids, float* logprob, int32_t* kept, void* stream);

/* Rows of logits and the settings that say what of them may be drawn, as in lowbit_sample, but one setting
 * per request (NULL = 1, 0, 1, 0). */
typedef struct lowbit_row_settings {
  const void* logits;          /* [rows][V], row stride row_stride elements */
  int64_t row_stride;
  int dtype, rows, V;          /* LOWBIT_LOGITS_FP32 or LOWBIT_LOGITS_BF16; 1 <= V <= 2^19 */
  const float* temperature;    /* [B] */
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
} lowbit_row_settings;

/* Bytes of lowbit_verify_drafts's workspace for M rows of the target and N drafts: 2,080 and 32 each (0 for
 * invalid shapes). */
size_t lowbit_verify_drafts_workspace_bytes(int M, int N);

/* Drafted tokens accepted or rejected against the target's probabilities, and the token that follows, so
 * that the outcome is distributed as sampling from the target alone (lmhead_argmax_verify is the greedy
 * case).  Request b of B has the drafts cu_drafts[b] .. cu_drafts[b + 1] - 1, any number down to none,
 * and one row of the target more than drafts: rows cu_drafts[b] + b .. cu_drafts[b + 1] + b, of which row i
 * judges the request's draft i and the last one follows them all.
 *   target    : the target's rows; at least N + B of them where all are used.
 *   draft     : the drafter's rows, row r of the N that draft r was drawn from, or NULL: every draft was
 *               proposed with certainty (a greedy drafter, looked-up tokens).
 *   drafts    : int32 [N], tokens of the target's vocabulary.
 *   draft_index : int32 [target V]: the column of the drafter's rows that stands for a token, -1 for none (a
 *               trimmed vocabulary), or NULL: the token itself.  Needs draft.
 *   u : fp32 [N], v : fp32 [B], in [0, 1).  Smaller ones and NaN count as 0, larger ones as 1: a draft is then accepted
 *   where q(d) < p(d), and the next token is the last one that may be drawn.
 * With p and q the shares m / S of lowbit_sample's masses, under the request's settings, in the target's
 * and the drafter's row (q = 1 for the draft and 0 else where draft is NULL; a token without column has
 * q = 0, a row without a finite logit p = 0 or q = 0 throughout):
 *   draft i is accepted where u q(d) < p(d), both shares, product and comparison in 64-bit floating point;
 *   n is the number of accepted drafts before the first that is not; a draft outside the vocabulary
 *   is never accepted.
 *   The next token comes from row n with v.  Where n is all of them: as lowbit_sample draws it.  Else
 *   from the masses r_i * 2^40 rounded, r_i = max(0, w_i * f - w'_i * f') over the tokens that p keeps, with
 *   w, w' the weights (0 of a token dropped or without mass), f = 2^40 / S rounded to fp32, and each
 *   product and the difference rounded to fp32:
 *   the first token in index order whose inclusive mass exceeds floor(v * their sum).  Where that sum is
 *   zero, as lowbit_sample draws from p.
 *   n_accept : int32 [B] out: n.
 *   ids    : int32 [target rows] out: a request's tokens in its rows: the n accepted drafts, the next token (-1
 *            where its row has no finite logit), and -1 in the rows behind it.
 *   accept : fp32 [N] out or NULL: min(1, p(d) / q(d)) of every draft, whatever became of it.
 * A request that cu_drafts describes inconsistently (decreasing, or outside the arrays) gets n = 0, no ids and
 * is recorded in the device error word.  Rows of no request are neither read nor written.
 *   workspace : lowbit_verify_drafts_workspace_bytes() bytes, 16-byte aligned, any contents; calls that may
 *   run at the same time need one each.  The result does not depend on timing.
 * n_accept, ids, accept and workspace may lie over nothing else that the call is given
 * (LOWBIT_ERR_INVALID_ARG). */
lowbit_status lowbit_verify_drafts(const lowbit_row_settings* target, const lowbit_row_settings* draft,
                                   int B, int N, const int32_t* cu_drafts, const int32_t* drafts,
                                   const int32_t* draft_index, const float* u, const float* v,
                                   int32_t* n_accept, int32_t* ids, float* accept,
                                   void* workspace, size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------------------------------
 * For callers that cannot allocate device memory.
 */

/* lmhead_argmax_verify without the `workspace` argument.  The method has no counterpart to this
 * function: it is a library convenience for callers that own no device allocator and so cannot
 * provide the 512-byte workspace -- for example a plugin whose device memory is planned ahead
 * of time by its host engine, or a C caller that links only this library and the CUDA runtime
 * and must not allocate on its serving path.
 *   Arguments, shapes, results and rounding are those of lmhead_argmax_verify.
 *   Scratch: the library holds one 512-byte scratch per device in place of `workspace`.  The
 *     first call on a device looks up its address (cudaGetSymbolAddress); make that first call
 *     before any stream capture on that device.  Nothing is allocated or freed, ever.
 *   Zeroing: the scratch must be zero when the kernel starts; every call clears it on `stream`
 *     itself (cudaMemsetAsync) before the kernel, so the caller never has to.
 *   Limit: shapes whose workspace (lmhead_workspace_bytes) would exceed 512 bytes return
 *     LOWBIT_ERR_WORKSPACE; every shape lmhead_argmax_verify accepts fits today.
 *   Concurrency: all calls on one device share the one scratch, so two calls that may run at
 *     the same time (for example on two streams with no ordering between them) race and give
 *     wrong results.  Order such calls, or use lmhead_argmax_verify with one workspace each. */
lowbit_status lmhead_argmax_verify_noalloc(const uint16_t* H, const void* packed_head, int M,
                                           int N, int K, const int32_t* draft, int32_t* argmax,
                                           int32_t* n_accept, int32_t* bonus, void* stream);

/* ------------------------------------------------------------------------------------------
 * Kernel-family selection (diagnostics and testing).  Same contract as the functions above,
 * plus `path`: 0 = the library's choice; 1 = the CUDA-core kernels (INT4: the streaming
 * kernel up to M = 4, integer dot products on block-scaled int16 activations, and a
 * row-per-lane bf16 kernel above; planes: the table-driven streaming kernel at M = 1 and a
 * sign-XOR kernel above; LM head: the row-per-lane kernel); 2 = the tcgen05 kernels
 * (dequantisation into tensor memory, tcgen05 MMA with fp32 accumulation); 3 (INT4, binary planes,
 * the sa format and the LM head, any M) = the warp-level MMA kernels (mma.sync m16n8k16 on bf16 fragments
 * unpacked in registers; binary planes too).  The library's choice for M >= 3 INT4, for binary
 * planes and the sa format at M >= 2 and for the LM head is 3:
 * with 16 activation rows a 128-row tcgen05 MMA issues as slowly as with 64, and the
 * weight stream then outruns it.  Other values: INVALID_ARG.
 */
lowbit_status lowbit_gemm_int4_path(const uint16_t* X, const void* packed, int M, int N, int K,
                                    uint16_t* Y, int path, void* stream);
lowbit_status lowbit_gemm_binplane_path(const uint16_t* X, const void* packed, int P, int M,
                                        int N, int K, uint16_t* Y, int path, void* stream);
lowbit_status lmhead_argmax_verify_path(const uint16_t* H, const void* packed_head, int M, int N,
                                        int K, const int32_t* draft, int32_t* argmax,
                                        int32_t* n_accept, int32_t* bonus, void* workspace,
                                        size_t ws_bytes, int path, void* stream);
/* path 1 at M >= 2: CUDA-core kernel (sign select by XOR into the activation's sign bit). */
lowbit_status lowbit_gemm_sa_path(const uint16_t* X, const void* packed, int P, int G, int M,
                                  int N, int K, uint16_t* Y, int path, void* stream);
/* NVFP4: path 1 = the streaming mat-vec (M = 1 only; M > 1 returns LOWBIT_ERR_SHAPE), which
 * reads each code byte through a table of the two codes' 2 * e2m1 values and takes integer dot
 * products with block-scaled int16 activations, each run of 16 scaled by its e4m3 scale in
 * fp32; path 2 = the tensor-core kernel.  The library's choice is path 1 at M = 1. */
lowbit_status lowbit_gemm_nvfp4_path(const uint16_t* X, const void* packed, int M, int N, int K,
                                     uint16_t* Y, int path, void* stream);
lowbit_status lowbit_draft_argmax_path(const uint16_t* H, const void* packed_head, int M, int N,
                                       int K, const int32_t* id_map, int32_t* ids,
                                       void* workspace, size_t ws_bytes, int path, void* stream);

/* ------------------------------------------------------------------------------------------
 * Device-side error word.
 */

/* Testing only: with `on` nonzero, every later launch of the streaming and warp-MMA kernels
 * (the library's default kernels, path 1 at M = 1 and path 3) has its compute warps wait for
 * data on a barrier that nothing arrives on, so that its bounded waits give up: each data
 * wait then ends after about a millisecond instead of about a second.  Such a call writes no
 * output (Y, argmax, n_accept, bonus, ids keep their previous contents), leaves the LM-head
 * workspace zeroed, and records LOWBIT_ERR_TIMEOUT in the device error word.  A CTA still
 * waits for its own copies in flight before it exits.  The attention calls' kernels then get no data
 * (no key tiles, or on tcgen05 no queries): every role's wait runs out, after about a second, and
 * neither out nor lse is written.  The other tcgen05 kernels and the CUDA-core kernels are not
 * affected.  The setting is process-wide; pass 0 to restore normal operation. */
lowbit_status lowbit_debug_inject_stall(int on);

/* Synchronises `stream`, then returns (in *status_out) and clears the current device's
 * error word: LOWBIT_OK, LOWBIT_ERR_INVALID_ARG (a kernel found a packed header that did not
 * match its arguments) or LOWBIT_ERR_TIMEOUT (a bounded wait gave up).  The function's own
 * return value reports failures of the query itself. */
lowbit_status lowbit_device_error(void* stream, int* status_out);

#ifdef __cplusplus
}
#endif

#endif /* LOWBIT_H */
