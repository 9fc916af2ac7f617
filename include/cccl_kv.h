/*
 * cccl_kv.h -- C ABI of libcccl, second part: the paged key/value cache that
 * a compressed payload (cccl_decompress_paged) arrives in, and what a serving
 * program does with it next: append tokens, take tokens out, attend.
 *
 *   cccl_kv_write      stores new tokens' keys and values, as they are or as
 *                      8-bit codes with a binary32 scale per token and head;
 *   cccl_kv_read       takes tokens out again as 16-bit values;
 *   cccl_kv_attention  attention of every sequence's new tokens (a chunk of a
 *                      prompt, or one token each) over its cached tokens.
 *
 * The conventions of cccl.h hold (caller-owned buffers, 16-byte alignment
 * unless stated, one allocation per buffer, host-checked argument errors
 * before anything is enqueued), with one difference: a workspace's 16-byte
 * status header is not cleared by these calls, so that a step of many calls
 * needs no clearing launch.  The caller zeroes those 16 bytes once
 * (cccl_kv_clear_status); a device error then stays readable with
 * cccl_get_result until the header is zeroed again.  Calls that run at the
 * same time need workspaces of their own; calls on one stream may share one.
 * All three calls can be captured in a CUDA graph.
 *
 * Device errors, reported as CCCL_ERR_INVALID_ARG: a page table entry outside
 * 0..pages-1 for a position that is used (that position is skipped, or read
 * as zeros), a length that is negative or longer than the table's pages hold,
 * cu_tokens that decrease or pass n_tokens (the range is clamped).  No such
 * input makes a call read or write out of range.
 */
#ifndef CCCL_KV_H
#define CCCL_KV_H

#include "cccl.h"

#ifdef __cplusplus
extern "C" {
#endif

/* How a cache holds its values. */
#define CCCL_KV_16BIT 0 /* the values themselves (bf16 or fp16) */
#define CCCL_KV_INT8 1  /* int8 codes in -127..127, value = code * scale */
#define CCCL_KV_E4M3 2  /* 8-bit floats (4 exponent, 3 fraction bits, no infinity, largest 448), value = code * scale */

/* Limits: sequences of one call, values of a head, query heads. */
#define CCCL_KV_MAX_BATCH 1024
#define CCCL_KV_MAX_DIM 128
#define CCCL_KV_MAX_HEADS 4096

/* One layer's paged cache, described on the host.  Value (page, slot, head,
 * i) of k is at k + page * page_stride + slot * token_stride +
 * head * head_stride + i, counted in elements (2 bytes for CCCL_KV_16BIT,
 * else 1), and v has the same strides: tokens or heads may lie outermost in
 * a page, and K and V may be interleaved.  Offsets may pass 32 bits.
 * Scale (page, slot, head) of k is k_scale[page * scale_page_stride +
 * slot * scale_token_stride + head * scale_head_stride] (8-bit formats only;
 * NULL otherwise), likewise v_scale. */
typedef struct {
    void *k, *v;
    float *k_scale, *v_scale;
    int32_t dtype;       /* CCCL_DTYPE_BF16 or CCCL_DTYPE_FP16: the type of values passed in and out */
    int32_t format;      /* CCCL_KV_* */
    int32_t kv_heads;    /* 1..CCCL_KV_MAX_HEADS */
    int32_t head_dim;    /* a multiple of 16, 16..CCCL_KV_MAX_DIM */
    int32_t page_tokens; /* slots of a page, >= 1 */
    int32_t reserved;    /* 0 */
    int64_t pages;
    int64_t page_stride, token_stride, head_stride; /* elements; multiples of 16 bytes, not negative */
    int64_t scale_page_stride, scale_token_stride, scale_head_stride; /* floats, not negative */
} cccl_kv_cache;

/* The sequences of one call.  Sequence b holds kv_lens[b] tokens; position p
 * lies in page page_table[b * table_stride + p / page_tokens], slot
 * p % page_tokens.  Its tokens of this call are rows cu_tokens[b] ..
 * cu_tokens[b + 1] - 1 of the packed tensors, and they are its last ones:
 * with n of them, row cu_tokens[b] + i is position kv_lens[b] - n + i.  A row
 * whose position is negative (n above kv_lens[b]) is in no page: a write
 * skips it, a read gives zeros, and in causal attention it sees no key (without
 * causal it sees all of them, whatever the window).  kv_lens counts the new tokens, so one batch serves a write and
 * the attention after it.  The arrays must not change while a call runs: its
 * blocks read them more than once and rely on seeing the same. */
typedef struct {
    const int32_t *page_table; /* device, [batch][table_stride], 4-byte aligned */
    const int32_t *cu_tokens;  /* device, [batch + 1], 4-byte aligned */
    const int32_t *kv_lens;    /* device, [batch], 4-byte aligned */
    int64_t table_stride;      /* >= table_pages */
    int64_t n_tokens;          /* rows of the packed tensors; 0 makes every call a no-op */
    int32_t batch;             /* 0..CCCL_KV_MAX_BATCH; 0 makes every call a no-op */
    int32_t table_pages;       /* usable entries of a table row, >= 1 */
    int32_t max_new, max_len;  /* what the program expects as the most new tokens and the longest length of a
                                * sequence, both >= 1: they choose kernels and how work is divided, so that results
                                * may differ in their rounding and no more */
} cccl_kv_batch;

/* Zero the status header of a workspace, on `stream`. */
cccl_status cccl_kv_clear_status(void *d_ws, size_t ws_bytes, cccl_stream_t stream);

/* Workspace bytes of any call below on this cache and batch: the status
 * header, and for attention the partial results of sequences whose cached
 * tokens are divided among SMs.  q_heads 0: for write and read alone.
 * Returns 0 for arguments that the calls refuse. */
size_t cccl_kv_workspace_bytes(const cccl_kv_cache *h_cache, const cccl_kv_batch *h_batch, int q_heads);

/* Store keys and values of the batch's tokens.  Token t, head h of d_k starts
 * at d_k + t * k_token_stride + h * k_head_stride (elements of the cache's
 * dtype; strides multiples of 8, not negative), likewise d_v: both may be
 * slices of one fused tensor.
 * 8-bit formats, per token and head, in binary32: a = max |x|, L = 127 or
 * 448, scale = a / L, inv = min(L / a, largest finite) (0 when a = 0); the
 * code is x * inv rounded to the nearest integer, ties to even, or to the
 * nearest E4M3 value, limited to +-L.  A vector with a NaN or an infinity gets
 * a NaN as its scale, and reads back as NaN throughout.
 * Two rows of one call that name the same page and slot: what that slot holds
 * afterwards is undefined (in 8-bit formats one row's codes may meet the other's
 * scale); nothing else is affected.
 * Returns INVALID_ARG, CUDA or OK. */
cccl_status cccl_kv_write(const cccl_kv_cache *h_cache, const cccl_kv_batch *h_batch, const void *d_k,
                          int64_t k_token_stride, int64_t k_head_stride, const void *d_v, int64_t v_token_stride,
                          int64_t v_head_stride, void *d_ws, size_t ws_bytes, cccl_stream_t stream);

/* The reverse: the cached keys and values of the batch's tokens, code * scale
 * rounded once to the cache's dtype, to d_k and d_v (strides as above). */
cccl_status cccl_kv_read(const cccl_kv_cache *h_cache, const cccl_kv_batch *h_batch, void *d_k, int64_t k_token_stride,
                         int64_t k_head_stride, void *d_v, int64_t v_token_stride, int64_t v_head_stride, void *d_ws,
                         size_t ws_bytes, cccl_stream_t stream);

/* Attention of the batch's tokens over the cached tokens of their sequences.
 * Row t, query head h of d_q starts at d_q + t * q_token_stride +
 * h * q_head_stride (the cache's dtype; strides multiples of 8); it reads the
 * cache's head h / (q_heads / kv_heads) (q_heads a multiple of kv_heads;
 * n_tokens * q_heads below 2^31).
 * With the row's position p and s_j = scale * q . k_j over the visible keys j
 *     j < kv_lens[b];  j <= p when causal;  j > p - window when window > 0
 * the result is  sum_j exp(s_j - m) v_j / sum_j exp(s_j - m),  m = max s_j,
 * rounded once to the cache's dtype at d_out + t * o_token_stride +
 * h * o_head_stride; d_lse (NULL, or n_tokens * q_heads floats, 4-byte
 * aligned) receives m + ln sum_j exp(s_j - m) at t * q_heads + h.
 * A row with no visible key gives zeros and -infinity.  What lies in a hidden
 * or unwritten place has no effect, NaN and infinities included.
 * Scores, maxima, sums and accumulators are binary32; 16-bit operands enter
 * the tensor cores as they are, 8-bit codes exactly (their scales are applied
 * in binary32), queries for 8-bit caches exactly down to 2^-29 of a row's
 * largest value.  A probability meets the values with 16 bits or more in calls
 * with few rows a kv head, rounded once to 16-bit floating point in others;
 * over fp16 and 8-bit caches that is fp16, whose smallest step is off by up to
 * 2^-39 (few rows), 2^-34 (others) or 2^-30 (others, 8-bit caches) of the row's
 * largest probability (times its value's scale).  Value scales may have either
 * sign; those smaller than 2^-90 may lose bits.  The same call gives the same
 * bits.  d_out may not overlap d_q or the cache.
 * Returns INVALID_ARG, CUDA or OK. */
cccl_status cccl_kv_attention(const cccl_kv_cache *h_cache, const cccl_kv_batch *h_batch, const void *d_q, int q_heads,
                              int64_t q_token_stride, int64_t q_head_stride, float scale, int causal, int64_t window,
                              void *d_out, int64_t o_token_stride, int64_t o_head_stride, float *d_lse, void *d_ws,
                              size_t ws_bytes, cccl_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* CCCL_KV_H */
