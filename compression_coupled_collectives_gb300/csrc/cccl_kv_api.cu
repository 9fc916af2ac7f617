// cccl_kv_api.cu -- the C ABI of the paged cache (include/cccl_kv.h): argument
// checks and launches.  Nothing here allocates memory or waits.
#include <cuda_runtime.h>

#include <cstdint>

#include "cccl.h"
#include "cccl_kv.cuh"
#include "cccl_kv.h"
#include "cccl_kv_check.h"
#include "cccl_kv_launch.h"
#include "cccl_launch.h"

using cccl::aligned;
using cccl::device_range;
using cccl::empty;
using cccl::fill;
using cccl::packed_ok;
using cccl::shapes_ok;

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
