/*
 * libtq, a decoding step around the attention of tq_kv.h: page tables, slots and masks made from
 * the requests' lengths (tq_kv_plan), the choice of the drafted tokens that stay (tq_verify), and
 * what stays with them in the cache (tq_kv_keep). Nothing of a step has to pass through the host:
 *
 *     tq_kv_plan    counts new tokens of each sequence -> slots, positions, offsets, masks, lengths
 *     tq_rope, tq_kv_store, tq_kv_attend    the layers
 *     tq_verify     the target's last layer and the drafted tokens -> the tokens that stay, a new one
 *     tq_kv_keep    -> rows of the accepted branch together, new lengths, unused pages given back
 *
 * so one step can be captured into a graph and replayed. The entry points follow the conventions of
 * tq.h. Outputs may not overlap inputs or each other but where it is said (TQ_ERR_ARG).
 */
#ifndef TQ_STEP_H
#define TQ_STEP_H

#include "tq_kv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* The pages of a cache that no sequence holds: the first state[0] entries of free_pages, the last of
 * them given out first. Calls that change one pool are ordered by the caller (one stream). */
typedef struct {
  int32_t *free_pages; /* device, [pages], 4-byte aligned */
  int32_t *state;      /* device, [2]: the number of free pages, and 0 (the calls count arrivals there) */
  int32_t pages;       /* of the cache, in [1, 2^30] */
} tq_kv_pool;

/* status of a sequence */
enum {
  TQ_PLAN_OK = 0,
  TQ_PLAN_NO_PAGES = 1, /* the pool has too few pages for it, or had for one before it */
  TQ_PLAN_TABLE = 2,    /* its tokens do not fit its row of the page table */
  TQ_PLAN_ROWS = 3      /* its rows do not fit M */
};

/* The step's tables. Sequence b < B holds lens[b] tokens and gets counts[b] rows (negative values
 * count as 0), rows o_b .. o_b + counts[b] of the step with o_b = sum of the counts before. Row i of a
 * sequence is its token lens[b] + i. Pages that it needs for them, ceil((lens + counts) / page_tokens)
 * - ceil(lens / page_tokens) of them, come off the pool in the order of the sequences and go into its
 * row of the page table. A sequence is served whole or refused: status[b] says why. Who asks for pages
 * behind a sequence that was refused for lack of pages is refused too.
 *   page_table   device int32 [B][table_width], entries of held pages read, of new pages written
 *   parents      device int32 [M], or NULL for chains: row i of a sequence follows its row parents[i]
 *                (in [0, i); another value ends the walk to the root there). Row 0 is the root. Prompts among
 *                trees are chains of parents; a tree of thousands of rows that does not begin as a chain is made by
 *                one workgroup from there on (0.1 ms for 4000 rows, 0.6 with their masks)
 *   shift        device int32 [B] or NULL: added to the positions
 * Outputs, device:
 *   slots        int64 [M]   page * page_tokens + place; -1 for rows of refused sequences, rows behind
 *                            the last sequence's and pages outside [0, pages)
 *   positions    int32 [M]   lens[b] + depth + shift[b], depth the row's steps to the root (a chain: i);
 *                            0 for rows without a sequence that is served
 *   q_offsets    int32 [B+1] min(o_b, M), for tq_kv_attend and tq_verify
 *   kv_lens      int32 [B]   lens + counts, for tq_kv_attend; 0 where refused (its rows see nothing)
 *   status       int32 [B]
 *   tree         uint32 [M][tree_words] or NULL (then tree_words is 0): a row's mask for tq_kv_attend,
 *                            itself and its ancestors (bits past tree_words * 32 are dropped), 0 for
 *                            rows without a sequence that is served
 *   left         int32 [1]: the free pages that are left. NULL: pool->state[0], the pages are taken.
 *                            Another address leaves the pool as it is, to look ahead.
 * B at most 65536, M at most 2^24, table_width * page_tokens below 2^31 - 65536, page_tokens in [1, 65536],
 * tree_words at most 65536. Workspace: none. */
int tq_kv_plan(const tq_kv_pool *pool, int32_t page_tokens, int32_t B, const int32_t *lens,
               const int32_t *counts, int32_t *page_table, int32_t table_width, int64_t M,
               const int32_t *parents, const int32_t *shift, int64_t *slots, int32_t *positions,
               int32_t *q_offsets, int32_t *kv_lens, int32_t *status, uint32_t *tree,
               int32_t tree_words, int32_t *left, void *stream);

/* What stays of a step. Of the n_b = q_offsets[b + 1] - q_offsets[b] rows planned behind lens[b]
 * tokens, kept[b] stay (cut to [0, n_b]; negative: the sequence ends, none of its tokens stays). The
 * sequence's new length is lens[b] + kept[b] (0 if it ends), and the pages behind it go back to the
 * pool: keeping nothing leaves the pool's list as it was before tq_kv_plan.
 *   q_offsets    device int32 [B + 1], or NULL: no rows (to end sequences)
 *   status       device int32 [B] of tq_kv_plan, or NULL: a refused sequence has no rows
 *   path         device int32, or NULL: row j of those kept stays where it is. Else the cache rows of
 *                token lens[b] + path[q_offsets[b] + j] are moved to token lens[b] + j, for 0 < j <
 *                kept[b]; the path of tq_verify: path >= j, ascending, below n_b (a row that is not
 *                is not moved; of a path that does not ascend the rows may hold each other's)
 *   M            elements of path (the step's rows): q_offsets are cut to [0, M]; without a path M is not used
 *   cache        read and written where path is not NULL, else it may be NULL
 *   page_table   device int32 [B][table_width], read; pages outside [0, pages) are not moved
 *   lens_out     device int32 [B], may be lens itself
 *   left         as in tq_kv_plan; the list is written either way (behind state[0])
 * Limits as for tq_kv_plan. Workspace: none. */
int tq_kv_keep(const tq_kv_pool *pool, const tq_kv_cache *cache, int32_t page_tokens, int32_t B,
               const int32_t *lens, const int32_t *q_offsets, const int32_t *status,
               const int32_t *kept, const int32_t *path, int64_t M, const int32_t *page_table,
               int32_t table_width, int32_t *lens_out, int32_t *left, void *stream);

/* flags of tq_verify: the rows are probabilities (not negative), not logits */
enum { TQ_TARGET_PROBS = 1, TQ_DRAFT_PROBS = 2 };

/* Which drafted tokens stay, and the token after them, so that the tokens are distributed as the
 * target's own (speculative sampling: Leviathan, Kalman, Matias 2023; Chen et al. 2023; several
 * children of a row one after another, each against what the ones before have left).
 * Rows offsets[b] .. offsets[b + 1] are sequence b's: row 0 the root (its last token, kept already),
 * the others drafted tokens, row i following row parents[i] < i (NULL: row i - 1). Row r of `target`
 * is the target's distribution of the token after r: softmax(x / temperature[b]), or the values as
 * they are with TQ_TARGET_PROBS. Row r of `draft` is the distribution that the tokens of r's children
 * were drawn from, softmax(x / temperature[b]) or the values with TQ_DRAFT_PROBS; rows without children
 * are not read. draft NULL: the drafted tokens are fixed (point
 * masses), such as the target's own most likely ones or tokens looked up in the text.
 * From c = the root on, with p, q of row c, a = 0, S = 1, the children x of c in their order, each
 * with its number u = uniforms[its row] in [0, 1):
 *     draft        u S q(x) < p(x) - a q(x): x stays, c = its row;  else a += S, S = sum_i (p_i - a q_i)+
 *     no draft     u S < p(x): x stays, c = its row;                else S -= p(x), p(x) = 0
 * When no child stays, the new token is the first i with w_0 + .. + w_i > u sum(w), u the root's
 * number, w_i = (p_i - a q_i)+ or the p that is left (if that is 0 everywhere, p itself).
 * temperature[b] not above 0: greedy, a child stays if it is the target's largest value (the lowest
 * index of equal ones), and the new token is that; draft is not read. A token outside [0, vocab) is
 * passed over (padding).
 *   target, draft  device, rows of vocab elements at their strides (elements), any alignment of their type
 *   temperature    device fp32 [B], or NULL: 1
 * Outputs, device int32:
 *   kept         [B]  rows that stay, the root among them (0 for a sequence without rows)
 *   out_tokens   [M]  from offsets[b]: the drafted tokens that stay, then the new one (kept[b] in all);
 *                     -1 behind them
 *   path         [M]  from offsets[b]: the rows that stay in the sequence, 0 first; -1 behind them
 * Rows behind offsets[B] are left as they were. Logits of -infinity are probabilities of 0. Where a row
 * of c's makes no distribution (logits with NaN, +infinity or nothing but -infinity; probabilities that
 * are looked at, a child's when it is tested and all of the row when S or w is summed, and are NaN or infinity;
 * a target's that are 0 throughout; greedy: NaN, +infinity or no value above 0 resp. -infinity), none of its
 * children stays (but one that stayed before the value was looked at) and the new token is -1.
 * Tests are as with sums of fp64 exponentials: u S q and p - a q (u S and p) are told apart where they differ by more
 * than about 1e-12 of what they are made of. A border of the cumulative sum of w lies where the definition has it to
 * about 1e-12 of the sum of p + a q; where most of p is within 4e-6 of a q, S and the borders are off by 1e-9 of that
 * sum at most. With a draft, sum(w) or S below 1e-12 (both sides probabilities: 1e-14) is nothing
 * left: no sibling stays, the new token is one of p. Weights below 1e-280 of the row's largest are 0. Deterministic.
 * Of a sequence that tq_kv_plan refused the results mean nothing; tq_kv_keep keeps none of its rows.
 * Time grows with the children that are turned away: with a draft each takes a sum over the vocabulary, by one
 * workgroup from a sequence's fifth on (0.05 ms for 60000 tokens); without one the k-th of a row is compared with the
 * k - 1 before it. Trees are meant to have tens of children to a row, not tens of thousands.
 * Workspace: tq_verify_workspace bytes, 256-byte aligned; its contents need not be kept, and two calls
 * that can run at the same time need one each. vocab in [1, 2^28], B at most 65536, M at most 2^24;
 * offsets non-decreasing, offsets[0] = 0, at most M. */
int tq_verify(const void *target, tq_dtype target_dtype, int64_t target_stride, const void *draft,
              tq_dtype draft_dtype, int64_t draft_stride, uint32_t flags, int64_t vocab, int32_t B,
              const int32_t *offsets, int64_t M, const int32_t *tokens, const int32_t *parents,
              const float *uniforms, const float *temperature, int32_t *kept, int32_t *out_tokens,
              int32_t *path, void *ws, size_t ws_bytes, void *stream);

/* Bytes of workspace tq_verify needs; drafted: 1 with a draft, else 0 (SIZE_MAX for invalid arguments). */
size_t tq_verify_workspace(int64_t vocab, int32_t B, int64_t M, int32_t drafted, uint32_t flags);

#ifdef __cplusplus
}
#endif

#endif /* TQ_STEP_H */
