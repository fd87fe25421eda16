/*
 * libtq, serving from a compressed KV cache: rotary positions, writing new tokens into a paged
 * cache of packed rows, reading tokens back, and attention over the packed codes. The entry
 * points follow the conventions of tq.h (memory, streams, errors, dtypes, formats, signs); the
 * exceptions are stated with each of them.
 */
#ifndef TQ_KV_H
#define TQ_KV_H

#include "tq.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A paged KV cache of packed rows: the two halves are tq_qweight descriptors of the same
 * rows, keys and values. Page p holds heads * page_tokens rows, row h * page_tokens + t being
 * token t of the page for (key/value) head h, so one head's tokens of a page are contiguous:
 *     codes [E pages][heads][page_tokens][words_per_row], scales [E][heads][page_tokens][K / group].
 * K is the head dimension, 64, 128 or 256 (the same for both halves); n_levels 4, 8, 16 or
 * 256 and group 32, 64 or 128 (dividing K) per half; N = heads * page_tokens; E pages, up to
 * 2^31 - 1 (the limit of 8192 experts does not apply). page_tokens is a multiple of 16 up to
 * 65536, heads at most 1024. codes are 16-byte aligned and scales 8-byte aligned. A token's
 * place is its slot, page * page_tokens + (index in the page), counted in 64 bits. The row of
 * a slot holds what tq_encode would store for that key or value with the signs of its half
 * (of a group with NaN or infinities only the same scale, NaN or 65504; its codes may be
 * others), so a cache of up to 8192 pages can also be read by tq_kv_fetch. Both halves may be
 * rotated by different signs. */
typedef struct {
  tq_qweight k, v;
  int32_t heads, page_tokens;
} tq_kv_cache;

/* Rotary positions: the first rot_dim elements of a head vector in pairs, each pair (a, b)
 * turned by the angle position * inv_freq[i] and scaled:
 *     (a cos - b sin, b cos + a sin) * gain,
 * pair i being elements (i, i + rot_dim / 2), or (2 i, 2 i + 1) when interleaved. Elements from
 * rot_dim on are left as they are. The angle is formed and reduced in fp64, so far positions
 * keep their precision. */
typedef struct {
  const double *inv_freq; /* device, [rot_dim / 2], radians per position, 8-byte aligned */
  int32_t rot_dim;        /* even, in [2, head_dim] */
  int32_t interleaved;    /* 0 or 1 */
  double gain;            /* 1 for none */
} tq_rope_params;

/* How tq_rope_frequencies stretches the frequencies f_i = base^(-2 i / rot_dim) for texts
 * `stretch` times as long as the `original` ones (stretch 1: no change in any of them):
 *   NONE    f_i
 *   LINEAR  f_i / stretch                                        (position interpolation)
 *   NTK     the frequencies of base * stretch^(rot_dim / (rot_dim - 2))      (rot_dim > 2)
 *   YARN    f_i (g + (1 - g) / stretch), g = clamp((turns - 1) / 31, 0, 1) with turns =
 *           original * f_i / (2 pi), and gain 0.1 ln(stretch) + 1 (Peng et al. 2023; turns
 *           below 1 are interpolated, above 32 kept)
 * YARN's ramp g is linear in the turns, as published. Programs that make it linear in the pair's
 * index i (in the logarithm of the turns) get other frequencies in between, by up to 2.3 times at
 * 128 dimensions and stretch 8: for a model trained with those, fill inv_freq by its own rule. */
enum { TQ_ROPE_NONE = 0, TQ_ROPE_LINEAR = 1, TQ_ROPE_NTK = 2, TQ_ROPE_YARN = 3 };

/* The frequencies into HOST memory inv_freq[rot_dim / 2] (fp64) and the gain (1 but for YARN)
 * into *gain. base > 0, stretch >= 1, original > 0 (read by YARN only). Copy them to the
 * device once for tq_rope_params. */
int tq_rope_frequencies(int32_t rot_dim, double base, int32_t scaling, double stretch,
                        double original, double *inv_freq, double *gain);

/* flags of tq_rope */
enum { TQ_ROPE_TRANSPOSED = 1 }; /* turn by the negative angle: the gradient of the call, and
                                    its inverse where gain is 1 */

/* out[t][h] = rotary(x[t][h]) at positions[t] for `tokens` x `heads` vectors of head_dim
 * elements of one dtype (device). x and out are addressed by their strides in elements
 * (token, head; the elements of a head are contiguous), so a slice of a fused projection's
 * output can be turned where it lies: out may be x itself with the same strides, and may not
 * overlap x otherwise, nor itself. head_dim even, in [2, 1024]; positions device int32 [tokens],
 * any sign. Sine and cosine (times the gain) are formed in fp64 and rounded to fp32; the products are
 * fp32, rounded to the type once. x and out need the alignment of their dtype (16-byte loads are used
 * where pointers, strides and sizes allow). */
int tq_rope(const void *x, tq_dtype dtype, int64_t tokens, int32_t heads, int32_t head_dim,
            int64_t x_token_stride, int64_t x_head_stride, const int32_t *positions,
            const tq_rope_params *rope, uint32_t flags, void *out, int64_t out_token_stride,
            int64_t out_head_stride, void *stream);

/* Writes `tokens` new tokens into the cache: for every token t with a slot in [0, E *
 * page_tokens), each head's key (value) is rotated, quantized and packed into its row, as
 * tq_encode does (fp64 rotation, RMS and, with `rope`, rotary turn; binary32 decision). A
 * slot outside that range is skipped, which is how padding is passed (-1). Each slot must
 * appear at most once in a call: of a slot given twice the row may hold a mix of both
 * tokens. k and v: device, [tokens][heads][K] of `dtype`, addressed by their strides in
 * elements (the elements of a head are contiguous). rope: NULL, or the rotary positions
 * applied to the keys first, at positions[t] (device int32). Both halves go in one launch;
 * nothing but the rows of the given slots is written. Workspace: none. */
int tq_kv_store(const tq_kv_cache *cache, const void *k, const void *v, tq_dtype dtype,
                int64_t tokens, int64_t k_token_stride, int64_t k_head_stride,
                int64_t v_token_stride, int64_t v_head_stride, const int64_t *slots,
                const tq_rope_params *rope, const int32_t *positions, void *stream);

/* Reads tokens back: k_out[t][h] = the dequantized, rotated-back key of slots[t] (v_out the
 * value), device [tokens][heads][K] of `dtype`, contiguous, 16-byte aligned; either may be
 * NULL, and they may not overlap. A slot outside [0, E * page_tokens) gives NaN rows; slots
 * may repeat. Computed in fp32 and rounded once, as tq_kv_fetch. Workspace: none. */
int tq_kv_load(const tq_kv_cache *cache, const int64_t *slots, int64_t tokens, void *k_out,
               void *v_out, tq_dtype dtype, void *stream);

/* Attention of ragged queries over the packed cache. Sequence b < B has kv_lens[b] tokens in
 * the cache, token j in page page_table[b][j / page_tokens], and the last n_b of them are its
 * queries' own: query i of sequence b is row q_offsets[b] + i of q and token kv_lens[b] - n_b +
 * i of the cache (store them first). It sees
 *   without tree   the tokens up to and including its own;
 *   with tree      every token before kv_lens[b] - n_b, and of the n_b last ones token j where
 *                  bit j % 32 of word j / 32 of its mask row is set (drafted tokens that see
 *                  only their ancestors); bits past tree_words * 32 count as unset.
 *     out = sum_j p_j v_j,  p = softmax_j(scale * q . k_j),
 * over the tokens it sees; a query that sees none gets zeros. The rotation is orthonormal, so
 * q is rotated once, scored against the decoded codes, and the sum of decoded values is
 * rotated back once: the cache is never unpacked in memory.
 *   q            device, rows of q_heads * K elements at q_token_stride (elements), bf16 or
 *                fp16, 16-byte aligned rows (the stride a multiple of 8); q_heads a multiple of
 *                cache->heads, query head h reading key head h / (q_heads / heads)
 *   q_offsets    device int32 [B + 1], non-decreasing, q_offsets[0] = 0, at most M; NULL for
 *                M / B queries per sequence (B must divide M). Rows of out behind
 *                q_offsets[B] are left as they were.
 *   kv_lens      device int32 [B]; lengths are cut to [0, table_width * page_tokens]
 *   page_table   device int32 [B][table_width]; entries behind a sequence's last page are not
 *                read; a page outside [0, E) makes the rows that see its tokens NaN
 *   tree         device uint32 [M][tree_words], or NULL
 *   out          device [M][q_heads][K], bf16 or fp16 (its own dtype), contiguous, 16-byte aligned; it
 *                may be q (with q's dtype and q_token_stride = q_heads * K), not overlap it otherwise
 * Scores, softmax statistics and sums are fp32; the operands of the matrix cores (rotated
 * q, centroids, p, decoded values) are fp16, scaled so that none overflows and so that no token's
 * scales, seen or not, take bits from another's: a token's part of an output is off by some 2^-11
 * of itself and 2^-32 of the token's value (weights below 2^-21 of the largest lose bits). So fp16
 * outputs are good to about 8e-4 of their norm and bf16 outputs to their rounding (the
 * quantization of an 8-bit cache costs 6e-3; tq_kv_load reads rows in fp32). Rows of the
 * last page behind kv_lens[b] may hold anything. A token whose scale is NaN makes the rows that
 * see it NaN, and no others. Deterministic; the last bits of a row depend on the batch it is in
 * (what else is in it decides where its tokens are cut into parts).
 * Workspace: tq_kv_attend_workspace(cache, q_heads, B, M) bytes (at most 69 MB, whatever the
 * lengths), 256-byte aligned; its contents need not be kept, and two calls that can run at the
 * same time need one each. M is at most 2^24, B at most 65536, (M + B) * q_heads below 2^31, and
 * times (table_width * page_tokens + 256) below 2^53. */
int tq_kv_attend(const tq_kv_cache *cache, const void *q, tq_dtype q_dtype, int32_t q_heads,
                 int64_t q_token_stride, int32_t B, const int32_t *q_offsets, int64_t M,
                 const int32_t *kv_lens, const int32_t *page_table, int32_t table_width,
                 const uint32_t *tree, int32_t tree_words, float scale, void *out,
                 tq_dtype out_dtype, void *ws, size_t ws_bytes, void *stream);

/* Bytes of workspace tq_kv_attend needs (SIZE_MAX for invalid arguments). */
size_t tq_kv_attend_workspace(const tq_kv_cache *cache, int32_t q_heads, int32_t B, int64_t M);

#ifdef __cplusplus
}
#endif

#endif /* TQ_KV_H */
