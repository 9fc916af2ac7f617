// cccl_kv_check.h -- host-side checks of the paged cache calls' arguments
// (internal), and the kernels' form of a cache and a batch.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "cccl.h"
#include "cccl_kv.cuh"
#include "cccl_kv.h"
#include "cccl_launch.h"

namespace cccl {

constexpr int64_t kMaxExtent = (int64_t)1 << 46;  // bytes of one buffer: keeps every product below 2^63

inline bool aligned(const void* p, uintptr_t to) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

// last byte offset + 1 of a strided view, in elements; false when a stride is
// negative or the extent passes kMaxExtent
inline bool extent(const int64_t* n, const int64_t* stride, int axes, int64_t inner, int64_t* out) {
    __int128 e = inner;
    for (int i = 0; i < axes; ++i) {
        if (stride[i] < 0) return false;
        e += (__int128)(n[i] - 1) * stride[i];
        if (e > kMaxExtent) return false;
    }
    *out = (int64_t)e;
    return true;
}

// Sizes of a cache and a batch that need no GPU to check.
inline bool shapes_ok(const cccl_kv_cache* c, const cccl_kv_batch* b) {
    if (c == nullptr || b == nullptr) return false;
    if (c->dtype != CCCL_DTYPE_BF16 && c->dtype != CCCL_DTYPE_FP16) return false;
    if (c->format != CCCL_KV_16BIT && c->format != CCCL_KV_INT8 && c->format != CCCL_KV_E4M3) return false;
    if (c->kv_heads < 1 || c->kv_heads > CCCL_KV_MAX_HEADS || c->reserved != 0) return false;
    if (c->head_dim < 16 || c->head_dim > CCCL_KV_MAX_DIM || c->head_dim % 16 != 0) return false;
    if (c->page_tokens < 1 || c->pages < 1 || c->pages > INT32_MAX) return false;
    if (b->batch < 0 || b->batch > CCCL_KV_MAX_BATCH || b->n_tokens < 0 || b->n_tokens > INT32_MAX) return false;
    return b->table_pages >= 1 && b->table_stride >= b->table_pages && b->max_new >= 1 && b->max_len >= 1;
}

// The remaining checks of a cache and batch, and the kernels' form of them.
inline bool fill(const cccl_kv_cache* c, const cccl_kv_batch* b, void* d_ws, size_t ws_bytes, size_t need, KvArgs* a) {
    DeviceRanges at;
    const int64_t elem = c->format == CCCL_KV_16BIT ? 2 : 1;
    const int64_t n[3] = {c->pages, c->page_tokens, c->kv_heads};
    const int64_t st[3] = {c->page_stride, c->token_stride, c->head_stride};
    int64_t values = 0;
    for (const int64_t s : st)
        if ((s * elem) % 16 != 0) return false;
    if (!extent(n, st, 3, c->head_dim, &values)) return false;
    if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(d_ws, 16) || ws_bytes < need) return false;
    if (!aligned(b->page_table, 4) || !aligned(b->cu_tokens, 4) || !aligned(b->kv_lens, 4)) return false;
    const int64_t rows[1] = {b->batch}, ts[1] = {b->table_stride};
    int64_t entries = 0, scales = 0;
    if (!extent(rows, ts, 1, b->table_pages, &entries)) return false;
    if (c->format != CCCL_KV_16BIT) {
        const int64_t ss[3] = {c->scale_page_stride, c->scale_token_stride, c->scale_head_stride};
        if (!aligned(c->k_scale, 4) || !aligned(c->v_scale, 4) || !extent(n, ss, 3, 1, &scales)) return false;
        if (!at.ok(c->k_scale, 4 * (size_t)scales) || !at.ok(c->v_scale, 4 * (size_t)scales))
            return false;
    }
    if (!at.ok(c->k, (size_t)(values * elem)) || !at.ok(c->v, (size_t)(values * elem)) ||
        !at.ok(d_ws, need) || !at.ok(b->page_table, 4 * (size_t)entries) ||
        !at.ok(b->cu_tokens, 4 * ((size_t)b->batch + 1)) || !at.ok(b->kv_lens, 4 * (size_t)b->batch))
        return false;
    a->k = static_cast<uint8_t*>(c->k);
    a->v = static_cast<uint8_t*>(c->v);
    a->k_scale = c->k_scale;
    a->v_scale = c->v_scale;
    a->page_stride = c->page_stride * elem;
    a->token_stride = c->token_stride * elem;
    a->head_stride = c->head_stride * elem;
    a->s_page = c->scale_page_stride;
    a->s_token = c->scale_token_stride;
    a->s_head = c->scale_head_stride;
    a->pages = c->pages;
    a->table = b->page_table;
    a->cu = b->cu_tokens;
    a->lens = b->kv_lens;
    a->table_stride = b->table_stride;
    a->n_tokens = b->n_tokens;
    a->ws = static_cast<WsHeader*>(d_ws);
    a->page_tokens = fast_div((uint32_t)c->page_tokens);
    a->kv_heads = c->kv_heads;
    a->dim = c->head_dim;
    a->batch = b->batch;
    a->table_pages = b->table_pages;
    return true;
}

// A packed 16-bit tensor [n_tokens, heads, dim] with two strides in elements.
inline bool packed_ok(const void* p, int64_t tokens, int64_t heads, int64_t dim, int64_t token_stride, int64_t head_stride) {
    const int64_t n[2] = {tokens, heads}, st[2] = {token_stride, head_stride};
    int64_t values = 0;
    return aligned(p, 16) && token_stride % 8 == 0 && head_stride % 8 == 0 && extent(n, st, 2, dim, &values) &&
           device_range(p, 2 * (size_t)values);
}

inline bool empty(const cccl_kv_batch* b) { return b->batch == 0 || b->n_tokens == 0; }

}  // namespace cccl
