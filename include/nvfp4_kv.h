/*
 * nvfp4_kv.h -- C ABI of the library's NVFP4 key/value cache: rotary
 * positions, appending to a paged cache, reading it back, and attention
 * over it.
 *
 * Conventions are those of nvfp4.h (device pointers owned by the caller,
 * asynchronous on `stream`, validation before any launch, NVFP4_* status
 * codes, nothing allocated). Tensors of heads are [tokens][heads][head_dim]
 * with head_dim contiguous; their token and head strides are given in
 * elements, so that a view of a fused projection's output is taken as it is.
 * Pointers must be 16-byte aligned and strides a multiple of 16 bytes.
 *
 * dtypes: NVFP4_F32, NVFP4_BF16, NVFP4_F16 (where a call lists them).
 *
 * Sizes that a grid does not hold are refused (NVFP4_ERR_SIZE): 2^28 tokens
 * of an append or a read, about 10^6 blocks of 16 elements in a token's heads,
 * 2^21 pieces of 128 rows (of all sequences and kv heads) of an attention.
 *
 * The cache. Keys and values are held as NVFP4: E2M1 codes, an E4M3 scale
 * per 16 elements along head_dim, and one binary32 scale per tensor,
 * S = amax / 2688, from the amax that the program gives for its keys and for
 * its values (calibrated, or any bound: larger values saturate as
 * nvfp4_quantize_1d's do). 16 consecutive tokens of one head are one record
 * of 18 * head_dim bytes; the cache is
 *     data [num_pages][kv_heads][page_size / 16][18 * head_dim].
 * With D = head_dim and t = 0..15 a record's token, a record holds
 *     8 D bytes  key codes    [g: 4][t: 16][D / 8]
 *                byte j of (g, t): elements g D/4 + 2j (low nibble), + 1
 *     8 D bytes  value codes  [t / 4: 4][c: 16][t % 4: 4][D / 32]
 *                byte j of (t, c): elements c D/16 + 2j (low nibble), + 1
 *       D bytes  key scales   [g: 4][t: 16][D / 64]
 *                byte j of (g, t): block g D/64 + j
 *       D bytes  value scales [block: D / 16][t: 16]
 * so that each 64-lane load of the attention's inner loop is one contiguous
 * span. head_dim is 64, 128 or 256; page_size a power of two from 16 to
 * 32768. Token p of sequence b is token p % page_size of page
 * page_table[b * table_stride + p / page_size].
 *
 * Indexes in device memory are checked by the kernels, not by the host: a
 * page outside [0, num_pages), or a position past the page table's row, is a
 * hole. Nothing is written to a hole, it reads as NaN, and attention takes
 * its tokens as masked.
 */
#ifndef NVFP4_KV_H
#define NVFP4_KV_H

#include "nvfp4.h"

#ifdef __cplusplus
extern "C" {
#endif

#define NVFP4_F16 2 /* a dtype beside NVFP4_F32 and NVFP4_BF16 */

/* flags */
#define NVFP4_ROPE_INTERLEAVED 0x1u /* pairs (2i, 2i + 1), not (i, i + rot_dim / 2) */
#define NVFP4_ROPE_ADJOINT 0x2u     /* rotate back: the gradient of the rotation    */
#define NVFP4_KV_CAUSAL 0x1u        /* a query sees the keys up to its own position */

/* scalings of nvfp4_rope_table */
#define NVFP4_ROPE_PLAIN 0  /* f_i = base^(-2i / rot_dim)                           */
#define NVFP4_ROPE_LINEAR 1 /* f_i / factor: positions interpolated                 */
#define NVFP4_ROPE_BASE 2   /* base * factor^(rot_dim / (rot_dim - 2)) as the base   */
#define NVFP4_ROPE_PARTS 3  /* by wavelength: f_i (w + (1 - w) / factor), with       */
                            /* w = clamp((n_i - low) / (high - low), 0, 1) and       */
                            /* n_i = original_len f_i / 2 pi the pair's turns over   */
                            /* the length that the model was trained on              */

/* Size of the workspace nvfp4_kv_attention takes. */
#define NVFP4_KV_WORKSPACE_BYTES (64 << 20)

/*
 * nvfp4_rope_table -- the cosines and sines of the rotation's angles:
 *   table  float [max_pos][2][rot_dim / 2]: amplitude cos(p f_i), then
 *          amplitude sin(p f_i), computed in 64 bits and rounded once.
 * rot_dim: a positive multiple of 16. base > 1, factor >= 1, amplitude
 * finite. original_len > 0 and low < high are read by NVFP4_ROPE_PARTS only.
 * A base change needs rot_dim > 2, which the multiple of 16 gives.
 */
int nvfp4_rope_table(int64_t max_pos, int64_t rot_dim, double base, int scaling, double factor,
                     double original_len, double low, double high, double amplitude, float* table,
                     hipStream_t stream);

/*
 * nvfp4_rope -- rotary positions. With c, s = table[positions[t]] and (a, b)
 * pair i of a head's first rot_dim elements,
 *     a' = fl(fl(a c) - fl(b s)),  b' = fl(fl(b c) + fl(a s))
 * in binary32, rounded once to the dtype; the other elements are copied.
 * NVFP4_ROPE_ADJOINT takes -s for s: the transpose of the rotation, i.e. its
 * gradient (dx from dy), and its inverse where the amplitude is 1.
 *   x, y       [tokens][heads][head_dim] of dtype (F32, BF16 or F16); y may
 *              be x (same strides), otherwise they must not overlap; its heads
 *              must not overlap each other either (x may be a broadcast view)
 *   positions  int32 [tokens]; one outside [0, max_pos) gives NaN in the
 *              rotated elements
 *   table      from nvfp4_rope_table (or the caller's own), 16-byte aligned
 * tokens >= 0, heads >= 1, head_dim and rot_dim multiples of 16, rot_dim <=
 * head_dim.
 */
int nvfp4_rope(const void* x, int dtype, int64_t tokens, int64_t heads, int64_t head_dim,
               int64_t x_token_stride, int64_t x_head_stride, const int32_t* positions,
               const float* table, int64_t max_pos, int64_t rot_dim, uint32_t flags, void* y,
               int64_t y_token_stride, int64_t y_head_stride, hipStream_t stream);

/*
 * nvfp4_kv_append -- quantizes new keys and values into the cache, the keys
 * rotated on the way; with q, also rotates the queries (one launch for all
 * that stands between the projection and the attention).
 *   k, v       [tokens][kv_heads][head_dim] of dtype (F32, BF16 or F16), both
 *              with kv_token_stride and kv_head_stride
 *   q, q_out   [tokens][heads][head_dim] of dtype, or both NULL (heads 0);
 *              q_out may be q (same strides); as y of nvfp4_rope otherwise
 *   positions  int32 [tokens]: place in the sequence, and the rotation's
 *              position. A negative one marks padding: nothing is cached, and
 *              its row of q_out is zero.
 *   seq        int32 [tokens]: each token's sequence (row of page_table), or
 *              NULL: token t belongs to sequence t (then tokens <= batch,
 *              padding among them)
 *   page_table int32 [batch][table_stride]
 *   table      rotation table (max_pos, rot_dim as nvfp4_rope), or NULL with
 *              rot_dim 0: no rotation (then q must be NULL too)
 *   flags      0 or NVFP4_ROPE_INTERLEAVED
 * Keys are quantized from the binary32 result of the rotation (not rounded
 * to dtype in between), values from their binary32 value, each 16-element
 * block as nvfp4_quantize_1d's: s = e4m3_rne(b / (6 S)), codes
 * e2m1_rne(|x| (1 / (s S))). A position past the table gives keys whose
 * scales are NaN. Two tokens of one call must not have the same place.
 * tokens >= 0.
 */
int nvfp4_kv_append(const void* k, const void* v, int dtype, int64_t tokens,
                    int64_t kv_token_stride, int64_t kv_head_stride, const void* q, void* q_out,
                    int64_t heads, int64_t q_token_stride, int64_t q_head_stride,
                    int64_t q_out_token_stride, int64_t q_out_head_stride, const int32_t* positions,
                    const int32_t* seq, const int32_t* page_table, int64_t batch,
                    int64_t table_stride, const float* table, int64_t max_pos, int64_t rot_dim,
                    uint32_t flags, uint8_t* data, int64_t num_pages, int64_t kv_heads,
                    int64_t page_size, int64_t head_dim, const float* k_amax, const float* v_amax,
                    hipStream_t stream);

/*
 * nvfp4_kv_read -- the keys and values that the cache holds for a list of
 * tokens, x = fl(fl(e2m1 * e4m3) * S) as nvfp4_dequantize gives it, rounded
 * once to out_dtype (F32, BF16 or F16).
 *   k_out, v_out  [tokens][kv_heads][head_dim], contiguous; either may be NULL
 *   positions, seq, page_table, data, ...: as nvfp4_kv_append. A negative
 *   position reads as zero, a hole as NaN.
 */
int nvfp4_kv_read(const uint8_t* data, int64_t num_pages, int64_t kv_heads, int64_t page_size,
                  int64_t head_dim, const float* k_amax, const float* v_amax, int64_t tokens,
                  const int32_t* positions, const int32_t* seq, const int32_t* page_table,
                  int64_t batch, int64_t table_stride, void* k_out, void* v_out, int out_dtype,
                  hipStream_t stream);

/*
 * nvfp4_kv_attention -- attention of new queries over the cached tokens,
 *     o = sum_t p_t v_t,  p = softmax(scale q . k_t)
 * over the tokens that the query sees. Query i of the nq of sequence b has
 * position lens[b] - nq + i (its own key is cached before the call); it sees
 * the cached tokens t < lens[b], with NVFP4_KV_CAUSAL only t <= its position,
 * and with window > 0 only t > its position - window. Without NVFP4_KV_CAUSAL
 * every query sees all of them (cross attention to an encoder's states,
 * cached once). A query that sees nothing gives o = 0 and lse = -inf; one with
 * an infinite or NaN element that sees something gives NaN.
 *   q       [total_q][heads][head_dim] of dtype (BF16 or F16), strided
 *   cu_q    int32 [batch + 1]: sequence b has the queries cu_q[b] ..
 *           cu_q[b + 1] - 1, at most max_q; or NULL: max_q each (total_q =
 *           batch * max_q). It rises from 0 to total_q (at most batch * max_q):
 *           rows of out that belong to no sequence are not written. Queries of
 *           a sequence past its first max_q give NaN (o and lse). The rows of a kv head that
 *           max_q allows choose the kernel (more than 32 to 128, by head_dim,
 *           are a prompt's), so prompts and single tokens go better in calls
 *           of their own.
 *   lens    int32 [batch], cached tokens including the new ones; one of at
 *           most 0 is an empty sequence, one past the page table's row is
 *           taken as the row's capacity
 *   heads   a multiple of kv_heads: query heads h G .. h G + G - 1 read
 *           key/value head h (G = heads / kv_heads)
 *   out     [total_q][heads][head_dim] of dtype, contiguous
 *   lse     optional float [total_q][heads]: ln sum_t exp(scale q . k_t)
 *   workspace  NVFP4_KV_WORKSPACE_BYTES bytes, zero-filled before its first
 *           use and then reused as is (each call leaves it ready for the
 *           next); calls that overlap in time need different ones
 * Rounding: scores from exact products in binary32 (q of BF16 is scaled by a
 * power of two per head, which binary16 then holds exactly down to 2^-30 of
 * the head's largest element), softmax statistics and sums in binary32, the
 * weights p in binary16 (11 bits) for their products with the values.
 * scale: finite and positive. 1 <= max_q, total_q >= 0, batch >= 0 (0: no
 * sequences and no queries, nothing is done).
 */
int nvfp4_kv_attention(const void* q, int dtype, int64_t total_q, int64_t heads,
                       int64_t q_token_stride, int64_t q_head_stride, const int32_t* cu_q,
                       int64_t max_q, const uint8_t* data, int64_t num_pages, int64_t kv_heads,
                       int64_t page_size, int64_t head_dim, const float* k_amax,
                       const float* v_amax, const int32_t* page_table, int64_t batch,
                       int64_t table_stride, const int32_t* lens, float scale, int64_t window,
                       uint32_t flags, void* out, float* lse, void* workspace, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* NVFP4_KV_H */
