/*
 * cccl_step.h -- C ABI of libcccl, third part: one step of a serving program
 * that drafts tokens, over the paged cache of cccl_kv.h.  A draft proposes a
 * tree of tokens a sequence (a chain is a tree); the target model computes all
 * of them at once; what it would have said itself is kept.
 *
 *   cccl_step_plan       block tables, slots, positions and masks from the
 *                        sequences' lengths and their trees;
 *   cccl_step_write      rotary positions for queries and keys; keys and
 *                        values go to their pages;
 *   cccl_step_attention  attention of the drafted tokens over what was cached
 *                        before them and their own ancestors;
 *   cccl_step_verify     which of them are kept, and the token after them,
 *                        from the target's probabilities and given random
 *                        numbers;
 *   cccl_step_keep       the kept ones' keys and values, moved together.
 *
 * The conventions of cccl_kv.h hold: caller-owned buffers, the workspace's
 * 16-byte status header zeroed once by the caller (cccl_kv_clear_status), host
 * checks before anything is enqueued, every call capturable in a CUDA graph,
 * and no input that makes a call read or write out of range.  Lengths, trees
 * and results stay on the device: a step needs no host synchronisation.
 *
 * In a sequence's tree token 0 is the root: the last token that the program is
 * sure of, whose keys and values are not cached yet.  Every other token has an
 * earlier one as its parent.
 */
#ifndef CCCL_STEP_H
#define CCCL_STEP_H

#include "cccl_kv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Limits: tokens of a tree that a mask of cccl_step_plan can hold (32 a word)
 * or that cccl_step_verify goes through, and values of a row of probabilities. */
#define CCCL_STEP_MAX_DRAFT 1024
#define CCCL_STEP_MAX_VOCAB (1 << 20)

/* Who holds which page.  Sequence b holds the pages page_table[b *
 * table_stride + 0 .. held[b] - 1]; free_pages[0 .. free_count[0] - 1] are
 * nobody's. */
typedef struct {
    int32_t *page_table;       /* device, [batch][table_stride], 4-byte aligned */
    const int32_t *held;       /* device, [batch] */
    const int32_t *free_pages; /* device, [free_capacity] */
    const int32_t *free_count; /* device, one number */
    int64_t table_stride;      /* >= table_pages */
    int64_t free_capacity;     /* 1..2^31 - 1 */
    int32_t batch;             /* 0..CCCL_KV_MAX_BATCH; 0 makes the call a no-op */
    int32_t table_pages;       /* usable entries of a table row, >= 1 */
    int32_t page_tokens;       /* slots of a page, >= 1 */
    int32_t reserved;          /* 0 */
} cccl_step_tables;

/* What a plan writes, all on the device; the first four are required. */
typedef struct {
    int32_t *cu_tokens;   /* [batch + 1] */
    int32_t *kv_lens;     /* [batch]; may be the lengths given */
    int32_t *held;        /* [batch]; may be the tables' held */
    int32_t *free_count;  /* one number; may be the tables' free_count */
    int64_t *slots;       /* [rows] or NULL; 8-byte aligned */
    int32_t *positions;   /* [rows] or NULL */
    uint32_t *mask;       /* [rows][mask_stride] or NULL */
    int64_t mask_stride;  /* >= mask_words */
    int64_t rows;         /* rows of the packed tensors, 0..2^31 - 1 */
    int32_t mask_words;   /* words of a mask, 1..CCCL_STEP_MAX_DRAFT / 32 (0 without mask) */
    int32_t reserved;     /* 0 */
} cccl_step_out;

/* d_new[b] tokens join the d_lens[b] that sequence b has cached.  Sequence b's
 * rows of the packed tensors are cu_tokens[b] .. cu_tokens[b + 1] - 1
 * (cu_tokens is the running sum of d_new from 0 on), kv_lens[b] = d_lens[b] +
 * d_new[b].  Where it holds fewer than ceil(kv_lens[b] / page_tokens) pages it
 * gets the missing ones, from the end of free_pages on, sequence by sequence:
 * with n pages given to the sequences before it, its first is
 * free_pages[free_count - 1 - n].  held and free_count count them.
 * Row cu_tokens[b] + i gets
 *   slots      page * page_tokens + slot of position d_lens[b] + i;
 *   positions  d_lens[b] + its depth: 0 for a token without a parent, else its
 *              parent's + 1 (d_parents NULL: i);
 *   mask       bit k % 32 of word k / 32 for itself and its ancestors k.
 * d_parents (NULL: every token's parent is the one before it) has a row's
 * parent as its number in the sequence's tree, -1 for none; one that is not
 * earlier is reported and taken as none.  Rows behind the last sequence's stay
 * as they are.
 * When the lengths, counts or pages do not fit (a negative number, more rows
 * than `rows`, more pages than a table row or free_pages has, with mask a
 * sequence of more than 32 * mask_words tokens, with d_parents one of more than
 * CCCL_STEP_MAX_DRAFT) nothing is given to anyone: cu_tokens is all 0,
 * kv_lens, held and free_count are what came in, the rest is untouched, and
 * CCCL_ERR_INVALID_ARG (too few free pages: CCCL_ERR_CAPACITY) is reported on
 * the device.  Outputs may not overlap inputs other than as said above.
 * d_ws: 16 bytes.  Returns INVALID_ARG, CUDA or OK. */
cccl_status cccl_step_plan(const cccl_step_tables *h_tables, const int32_t *d_lens, const int32_t *d_new,
                           const int32_t *d_parents, const cccl_step_out *h_out, void *d_ws, size_t ws_bytes,
                           cccl_stream_t stream);

/* Rotary positions of a model, on the host.  Of the first rot_dim values of a
 * head pair i is (x_i, x_{i + rot_dim / 2}), or (x_2i, x_{2i + 1}) when
 * interleaved; at position p it is turned by p * turns[i] / 2^64 full turns
 * (modulo whole ones, exactly) and multiplied by magnitude:
 *   (a, b) -> magnitude (a cos t - b sin t, b cos t + a sin t).
 * The other values stay as they are. */
typedef struct {
    const uint64_t *turns; /* device, [rot_dim / 2], 8-byte aligned (cccl_step_rotary_turns) */
    float magnitude;       /* finite */
    int32_t rot_dim;       /* a multiple of 16, 16..the cache's head_dim */
    int32_t interleaved;   /* 0 or 1 */
    int32_t reserved;      /* 0 */
} cccl_step_rotary;

/* The usual frequencies, computed on the host: pair i turns by f_i = base^(-2 i
 * / rot_dim) radians a position.  For contexts that are longer than the model
 * was trained on, by `factor`:
 *   original_length 0: f_i / factor, every pair alike;
 *   else by parts: with r_i = original_length f_i / (2 pi) turns over the
 *   original length and g = (r_i - few) / (many - few), limited to 0..1,
 *   g f_i + (1 - g) f_i / factor.
 * In binary64: with base and factor of 1 or more, and many not below 4/3 few, a
 * pair's turns are off by less than 2^-51 of a turn a position (the usual bases,
 * up to 10^6: 2^-55).
 * h_turns: [rot_dim / 2], on the host.  Returns INVALID_ARG (base, factor not
 * positive and finite, few not below many with a length) or OK. */
cccl_status cccl_step_rotary_turns(int rot_dim, double base, double factor, double original_length, double few,
                                   double many, uint64_t *h_turns);

/* Rotate the batch's queries and keys and store its keys and values: as
 * cccl_kv_write, with d_k rotated first.  Row t stands at position
 * d_positions[t] (NULL: its place in the sequence, as in cccl_kv_batch); where
 * it is stored goes by the batch alone, so drafted siblings may share a
 * position.  Rotated values are binary32, rounded once: to the cache's dtype
 * in d_q_out and a 16-bit cache, to codes in an 8-bit one (no rounding before
 * the scale is taken).  Angles are off by less than 2^-21 radians from the given
 * turns', at any position.  d_q and d_q_out: [n_tokens, q_heads, head_dim] with strides as in
 * cccl_kv_write; they may be the same tensor and may not overlap in another
 * way; q_heads 0: no queries (both NULL).  Rows of no sequence stay as they
 * are in d_q_out; one at a negative place (cccl_kv_batch) is rotated there and
 * stored nowhere.
 * d_ws: 16 bytes.  Returns INVALID_ARG, CUDA or OK. */
cccl_status cccl_step_write(const cccl_kv_cache *h_cache, const cccl_kv_batch *h_batch, const cccl_step_rotary *h_rotary,
                            const int32_t *d_positions, const void *d_q, int q_heads, int64_t q_token_stride,
                            int64_t q_head_stride, void *d_q_out, int64_t qo_token_stride, int64_t qo_head_stride,
                            const void *d_k, int64_t k_token_stride, int64_t k_head_stride, const void *d_v,
                            int64_t v_token_stride, int64_t v_head_stride, void *d_ws, size_t ws_bytes,
                            cccl_stream_t stream);

/* Attention of drafted tokens: as cccl_kv_attention, but a sequence's new
 * token i sees the cached tokens before the new ones (positions below
 * kv_lens[b] - n, all of them) and of the new ones those k whose bit (k % 32
 * of word k / 32) is set in row t of d_mask, t its row of the packed tensors:
 * itself only if its own bit is set.  d_mask has n_tokens rows of mask_words
 * words, mask_stride from one to the next; tokens from 32 * mask_words on are
 * seen by none.  window > 0: of what a token sees without it, the last
 * `window` (those cached before the draft first, then drafted ones by their
 * number): with masks of ancestors, the window of its own path.
 * Workspace: cccl_kv_workspace_bytes(h_cache, h_batch, q_heads).  Rounding,
 * empty rows, hidden places and overlaps as in cccl_kv_attention: so the size of
 * the program's trees (max_new, times the query heads that share a kv head: up to
 * 24 such rows, 32 over an 8-bit cache, are few) says whether probabilities meet
 * the values with 16 bits or more or are rounded once to 16-bit floating point.
 * Returns INVALID_ARG, CUDA or OK. */
cccl_status cccl_step_attention(const cccl_kv_cache *h_cache, const cccl_kv_batch *h_batch, const void *d_q, int q_heads,
                                int64_t q_token_stride, int64_t q_head_stride, float scale, const uint32_t *d_mask,
                                int64_t mask_stride, int mask_words, int64_t window, void *d_out,
                                int64_t o_token_stride, int64_t o_head_stride, float *d_lse, void *d_ws,
                                size_t ws_bytes, cccl_stream_t stream);

/* The drafts of one call, on the host.  Rows cu_tokens[b] .. cu_tokens[b + 1]
 * - 1 are sequence b's tree.  Row t of p holds the target's probabilities of
 * the token after the path that ends in token t, row t of q the probabilities
 * that the draft drew t's children from (q NULL: the draft chose them without
 * chance).  Rows of p and q have `vocab` binary32 values side by side. */
typedef struct {
    const float *p, *q;          /* device, 4-byte aligned; q may be NULL */
    int64_t p_stride, q_stride;  /* values from one row to the next, >= vocab */
    const int32_t *tokens;       /* device, [rows]; a root's is not looked at */
    const int32_t *parents;      /* device, [rows]: a token's parent by its number in the tree (NULL: the one before) */
    const float *uniform;        /* device, [rows]: independent random numbers, 0 <= u < 1 */
    const int32_t *cu_tokens;    /* device, [batch + 1] */
    int64_t rows;                /* 0..2^31 - 1 */
    int32_t batch;               /* 0..CCCL_KV_MAX_BATCH */
    int32_t vocab;               /* 1..CCCL_STEP_MAX_VOCAB */
} cccl_step_draft;

/* Which drafted tokens are kept, so that the kept ones and the next token are
 * distributed as if the target had drawn them one by one.  The root is kept.
 * Then the tree is gone through in order, with a current token c (the root at
 * first) and a number A (0 at first):
 *   a token x whose parent is c is tried.  With
 *     R(y) = max(p_c(y) - A q_c(y), 0),  S = 1 when A = 0, else sum R,
 *   it is kept when u S q_c(x) < R(x), u its own random number: c becomes this
 *   token and A 0.  Else A becomes A + S.
 *   Without q: R is p_c without the tokens that were refused here, S is 1 less
 *   their p_c; kept when u S < R(x).
 * At the end the next token is drawn from R at the last c by the root's random
 * number u: the first y with R(0) + .. + R(y) > u sum R (from p_c itself where
 * R is 0 throughout).
 * Probabilities enter sums as multiples of 2^-56, cut off below, and sums of those
 * are exact.  A is held in multiples of 2^-53 and A q_c(y) in multiples of 2^-56,
 * both cut off below; u q_c(x) < p_c(x) is decided exactly, u S q_c(x) < R(x) at
 * A > 0 in binary64.  So results depend on nothing but the inputs.  Values that
 * are not numbers or negative count as 0, values above 1 as 1; where a row adds
 * up to more than 2 the next token is any (and may be reported).  A token outside
 * 0..vocab - 1, or whose parent is not earlier, is passed over; a tree's tokens
 * from CCCL_STEP_MAX_DRAFT on are passed over and reported.
 * d_path [rows]: rows cu_tokens[b] + k, k < n_kept[b], the number of the k-th
 * kept token (the root's 0 first), -1 in the others of the sequence.
 * d_next [batch]: the next token.  A sequence without rows has 0 kept and -1
 * next; one whose row of p has no positive value 0 next (reported).
 * Outputs may not overlap inputs.
 * d_ws: 16 bytes.  Returns INVALID_ARG, CUDA or OK. */
cccl_status cccl_step_verify(const cccl_step_draft *h_draft, int32_t *d_path, int32_t *d_n_kept, int32_t *d_next,
                             void *d_ws, size_t ws_bytes, cccl_stream_t stream);

/* Kept tokens moved together in one layer's cache: for k < d_n_kept[b], what
 * the cache holds (codes and scales as they are) at the place of sequence b's
 * new token d_path[cu_tokens[b] + k] goes to the place of its k-th; nothing else
 * in the cache changes.  d_lens [batch] (NULL: not wanted) gets the length
 * without the others: kv_lens[b] - n + n_kept[b] (0 where that is negative),
 * also where n_tokens is 0: other than in the calls above only batch 0 makes
 * this one a no-op, since every sequence has a length.
 * A path's entries k have to lie in k .. n - 1; others are not moved, and
 * reported, as is a count outside 0..n (clamped).  d_lens may not overlap the
 * batch's arrays, d_path or d_n_kept, which the call's blocks read while it is
 * written (and which further calls need, one a layer): refused.
 * d_ws: 16 bytes.  Returns INVALID_ARG, CUDA or OK. */
cccl_status cccl_step_keep(const cccl_kv_cache *h_cache, const cccl_kv_batch *h_batch, const int32_t *d_path,
                           const int32_t *d_n_kept, int32_t *d_lens, void *d_ws, size_t ws_bytes, cccl_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* CCCL_STEP_H */
