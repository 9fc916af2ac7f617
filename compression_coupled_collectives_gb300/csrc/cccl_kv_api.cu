// cccl_kv_api.cu -- the C ABI of the paged cache (include/cccl_kv.h): argument
// checks and launches.  Nothing here allocates memory or waits.
#include <cuda_runtime.h>

#include <cstdint>

#include "cccl.h"
#include "cccl_kv.cuh"
#include "cccl_kv.h"
#include "cccl_kv_launch.h"
#include "cccl_launch.h"

namespace {

using cccl::device_range;

constexpr int64_t kMaxExtent = (int64_t)1 << 46;  // bytes of one buffer: keeps every product below 2^63

bool aligned(const void* p, uintptr_t to) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

// last byte offset + 1 of a strided view, in elements; false when a stride is
// negative or the extent passes kMaxExtent
bool extent(const int64_t* n, const int64_t* stride, int axes, int64_t inner, int64_t* out) {
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
bool shapes_ok(const cccl_kv_cache* c, const cccl_kv_batch* b) {
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
bool fill(const cccl_kv_cache* c, const cccl_kv_batch* b, void* d_ws, size_t ws_bytes, size_t need, cccl::KvArgs* a) {
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
        if (!device_range(c->k_scale, 4 * (size_t)scales) || !device_range(c->v_scale, 4 * (size_t)scales))
            return false;
    }
    if (!device_range(c->k, (size_t)(values * elem)) || !device_range(c->v, (size_t)(values * elem)) ||
        !device_range(d_ws, need) || !device_range(b->page_table, 4 * (size_t)entries) ||
        !device_range(b->cu_tokens, 4 * ((size_t)b->batch + 1)) || !device_range(b->kv_lens, 4 * (size_t)b->batch))
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
    a->ws = static_cast<cccl::WsHeader*>(d_ws);
    a->page_tokens = cccl::fast_div((uint32_t)c->page_tokens);
    a->kv_heads = c->kv_heads;
    a->dim = c->head_dim;
    a->batch = b->batch;
    a->table_pages = b->table_pages;
    return true;
}

// A packed 16-bit tensor [n_tokens, heads, dim] with two strides in elements.
bool packed_ok(const void* p, int64_t tokens, int64_t heads, int64_t dim, int64_t token_stride, int64_t head_stride) {
    const int64_t n[2] = {tokens, heads}, st[2] = {token_stride, head_stride};
    int64_t values = 0;
    return aligned(p, 16) && token_stride % 8 == 0 && head_stride % 8 == 0 && extent(n, st, 2, dim, &values) &&
           device_range(p, 2 * (size_t)values);
}

bool empty(const cccl_kv_batch* b) { return b->batch == 0 || b->n_tokens == 0; }

}  // namespace

extern "C" {

cccl_status cccl_kv_clear_status(void* d_ws, size_t ws_bytes, cccl_stream_t stream) {
    if (!aligned(d_ws, 16) || ws_bytes < sizeof(cccl::WsHeader) || !device_range(d_ws, sizeof(cccl::WsHeader)))
        return CCCL_ERR_INVALID_ARG;
    return cudaMemsetAsync(d_ws, 0, sizeof(cccl::WsHeader), reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
               ? CCCL_OK
               : CCCL_ERR_CUDA;
}

size_t cccl_kv_workspace_bytes(const cccl_kv_cache* h_cache, const cccl_kv_batch* h_batch, int q_heads) {
    if (!shapes_ok(h_cache, h_batch) || q_heads < 0 || q_heads > CCCL_KV_MAX_HEADS) return 0;
    if (q_heads == 0) return sizeof(cccl::WsHeader);
    if (q_heads % h_cache->kv_heads != 0) return 0;
    return sizeof(cccl::WsHeader) + cccl::kv_attention_scratch(h_cache->format, h_cache->head_dim,
                                                               q_heads / h_cache->kv_heads, h_batch->max_new);
}

static cccl_status copy_call(bool write, const cccl_kv_cache* c, const cccl_kv_batch* b, const void* d_k, int64_t kt,
                             int64_t kh, const void* d_v, int64_t vt, int64_t vh, void* d_ws, size_t ws_bytes,
                             cccl_stream_t stream) {
    if (!shapes_ok(c, b)) return CCCL_ERR_INVALID_ARG;
    if (empty(b)) return CCCL_OK;
    cccl::KvArgs a{};
    if (!fill(c, b, d_ws, ws_bytes, sizeof(cccl::WsHeader), &a) ||
        !packed_ok(d_k, b->n_tokens, c->kv_heads, c->head_dim, kt, kh) ||
        !packed_ok(d_v, b->n_tokens, c->kv_heads, c->head_dim, vt, vh))
        return CCCL_ERR_INVALID_ARG;
    const cccl::KvPacked x{static_cast<uint8_t*>(const_cast<void*>(d_k)), static_cast<uint8_t*>(const_cast<void*>(d_v)),
                           2 * kt, 2 * kh, 2 * vt, 2 * vh};
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = write ? cccl::launch_kv_write(c->dtype, c->format, a, x, s)
                                : cccl::launch_kv_read(c->dtype, c->format, a, x, s);
    return e == cudaSuccess ? CCCL_OK : CCCL_ERR_CUDA;
}

cccl_status cccl_kv_write(const cccl_kv_cache* h_cache, const cccl_kv_batch* h_batch, const void* d_k,
                          int64_t k_token_stride, int64_t k_head_stride, const void* d_v, int64_t v_token_stride,
                          int64_t v_head_stride, void* d_ws, size_t ws_bytes, cccl_stream_t stream) {
    return copy_call(true, h_cache, h_batch, d_k, k_token_stride, k_head_stride, d_v, v_token_stride, v_head_stride,
                     d_ws, ws_bytes, stream);
}

cccl_status cccl_kv_read(const cccl_kv_cache* h_cache, const cccl_kv_batch* h_batch, void* d_k, int64_t k_token_stride,
                         int64_t k_head_stride, void* d_v, int64_t v_token_stride, int64_t v_head_stride, void* d_ws,
                         size_t ws_bytes, cccl_stream_t stream) {
    return copy_call(false, h_cache, h_batch, d_k, k_token_stride, k_head_stride, d_v, v_token_stride, v_head_stride,
                     d_ws, ws_bytes, stream);
}

cccl_status cccl_kv_attention(const cccl_kv_cache* h_cache, const cccl_kv_batch* h_batch, const void* d_q, int q_heads,
                              int64_t q_token_stride, int64_t q_head_stride, float scale, int causal, int64_t window,
                              void* d_out, int64_t o_token_stride, int64_t o_head_stride, float* d_lse, void* d_ws,
                              size_t ws_bytes, cccl_stream_t stream) {
    const cccl_kv_cache* c = h_cache;
    const cccl_kv_batch* b = h_batch;
    if (!shapes_ok(c, b) || q_heads < 1 || q_heads > CCCL_KV_MAX_HEADS || q_heads % c->kv_heads != 0 || window < 0 ||
        (causal != 0 && causal != 1) || !(scale >= -3.402823466e+38f && scale <= 3.402823466e+38f))
        return CCCL_ERR_INVALID_ARG;
    if (empty(b)) return CCCL_OK;
    if (b->n_tokens > INT32_MAX / q_heads) return CCCL_ERR_INVALID_ARG;
    cccl::KvArgs a{};
    if (!fill(c, b, d_ws, ws_bytes, cccl_kv_workspace_bytes(c, b, q_heads), &a) ||
        !packed_ok(d_q, b->n_tokens, q_heads, c->head_dim, q_token_stride, q_head_stride) ||
        !packed_ok(d_out, b->n_tokens, q_heads, c->head_dim, o_token_stride, o_head_stride))
        return CCCL_ERR_INVALID_ARG;
    if (d_lse != nullptr &&
        (!aligned(d_lse, 4) || !device_range(d_lse, 4 * (size_t)b->n_tokens * (size_t)q_heads)))
        return CCCL_ERR_INVALID_ARG;
    cccl::AttnArgs t{};
    t.q = static_cast<const uint8_t*>(d_q);
    t.out = static_cast<uint8_t*>(d_out);
    t.lse = d_lse;
    t.q_token = 2 * q_token_stride;
    t.q_head = 2 * q_head_stride;
    t.o_token = 2 * o_token_stride;
    t.o_head = 2 * o_head_stride;
    t.window = window < INT32_MAX ? (int32_t)window : 0;  // one that hides nothing is none
    t.scale = scale;
    t.causal = causal;
    t.group = cccl::fast_div((uint32_t)(q_heads / c->kv_heads));
    t.q_heads = q_heads;
    const cudaError_t e = cccl::launch_kv_attention(c->dtype, c->format, a, t, b->max_new, b->max_len,
                                                    reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? CCCL_OK : CCCL_ERR_CUDA;
}

}  // extern "C"
