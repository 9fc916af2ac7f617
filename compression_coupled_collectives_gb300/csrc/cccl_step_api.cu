// cccl_step_api.cu -- the C ABI of a step with drafted tokens
// (include/cccl_step.h): argument checks and launches.  Nothing here allocates
// memory or waits.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "cccl.h"
#include "cccl_kv_check.h"
#include "cccl_kv_launch.h"
#include "cccl_launch.h"
#include "cccl_step.cuh"
#include "cccl_step.h"

using cccl::aligned;
using cccl::empty;
using cccl::extent;
using cccl::fill;
using cccl::packed_ok;
using cccl::shapes_ok;

namespace {

// The pointers of one call.
struct Pointers {
    cccl::DeviceRanges ranges;
    // n numbers of `bytes` each, aligned to their size
    bool numbers(const void* p, int64_t n, int bytes) {
        return aligned(p, (uintptr_t)bytes) && ranges.ok(p, (size_t)n * (size_t)bytes);
    }
    // rows of `inner` numbers, `stride` apart
    bool rows(const void* p, int64_t rows, int64_t stride, int64_t inner, int bytes) {
        const int64_t n[1] = {rows}, st[1] = {stride};
        int64_t values = 0;
        return extent(n, st, 1, inner, &values) && numbers(p, values, bytes);
    }
    bool workspace(void* d_ws, size_t ws_bytes) {
        return aligned(d_ws, 16) && ws_bytes >= sizeof(cccl::WsHeader) && ranges.ok(d_ws, sizeof(cccl::WsHeader));
    }
};
// whether n numbers have none in common with `rows` rows of m, `stride` (>= m) apart
bool apart(const int32_t* a, int64_t n, const int32_t* b, int64_t m, int64_t rows = 1, int64_t stride = 1) {
    const int64_t at = ((int64_t)reinterpret_cast<uintptr_t>(a) - (int64_t)reinterpret_cast<uintptr_t>(b)) / 4;
    const int64_t row = at < m ? 0 : (at - m) / stride + 1;  // the first that ends behind `at`
    return m == 0 || row >= rows || row * stride >= at + n;
}
cccl_status status_of(cudaError_t e) {
    if (e == cudaSuccess) return CCCL_OK;
    cudaGetLastError();  // a refused launch is not the next call's error
    return CCCL_ERR_CUDA;
}

}  // namespace

extern "C" {

cccl_status cccl_step_plan(const cccl_step_tables* h_tables, const int32_t* d_lens, const int32_t* d_new,
                           const int32_t* d_parents, const cccl_step_out* h_out, void* d_ws, size_t ws_bytes,
                           cccl_stream_t stream) {
    const cccl_step_tables* t = h_tables;
    const cccl_step_out* o = h_out;
    if (t == nullptr || o == nullptr || t->batch < 0 || t->batch > CCCL_KV_MAX_BATCH || t->table_pages < 1 ||
        t->table_stride < t->table_pages || t->page_tokens < 1 || t->free_capacity < 1 ||
        t->free_capacity > INT32_MAX || t->reserved != 0 || o->reserved != 0 || o->rows < 0 || o->rows > INT32_MAX)
        return CCCL_ERR_INVALID_ARG;
    if (o->mask != nullptr ? o->mask_words < 1 || o->mask_words > CCCL_STEP_MAX_DRAFT / 32 || o->mask_stride < o->mask_words
                           : o->mask_words != 0)
        return CCCL_ERR_INVALID_ARG;
    if (t->batch == 0) return CCCL_OK;
    Pointers at;
    if (!at.workspace(d_ws, ws_bytes) || !at.rows(t->page_table, t->batch, t->table_stride, t->table_pages, 4) ||
        !at.numbers(t->held, t->batch, 4) || !at.numbers(t->free_pages, t->free_capacity, 4) ||
        !at.numbers(t->free_count, 1, 4) ||
        !at.numbers(d_lens, t->batch, 4) || !at.numbers(d_new, t->batch, 4) ||
        !at.numbers(o->cu_tokens, (int64_t)t->batch + 1, 4) || !at.numbers(o->kv_lens, t->batch, 4) ||
        !at.numbers(o->held, t->batch, 4) || !at.numbers(o->free_count, 1, 4))
        return CCCL_ERR_INVALID_ARG;
    if (o->rows > 0 && ((d_parents != nullptr && !at.numbers(d_parents, o->rows, 4)) ||
                        (o->slots != nullptr && !at.numbers(o->slots, o->rows, 8)) ||
                        (o->positions != nullptr && !at.numbers(o->positions, o->rows, 4)) ||
                        (o->mask != nullptr && !at.rows(o->mask, o->rows, o->mask_stride, o->mask_words, 4))))
        return CCCL_ERR_INVALID_ARG;
    cccl::PlanArgs a{};
    a.lens = d_lens;
    a.fresh = d_new;
    a.held = t->held;
    a.free_pages = t->free_pages;
    a.free_count = t->free_count;
    a.parents = d_parents;
    a.table = t->page_table;
    a.table_stride = t->table_stride;
    a.free_capacity = t->free_capacity;
    a.rows = o->rows;
    a.cu = o->cu_tokens;
    a.lens_out = o->kv_lens;
    a.held_out = o->held;
    a.count_out = o->free_count;
    a.positions = o->positions;
    a.slots = o->slots;
    a.mask = o->mask;
    a.mask_stride = o->mask_stride;
    a.ws = static_cast<cccl::WsHeader*>(d_ws);
    a.page_tokens = cccl::fast_div((uint32_t)t->page_tokens);
    a.batch = t->batch;
    a.table_pages = t->table_pages;
    a.words = o->mask_words;
    return status_of(cccl::launch_step_plan(a, reinterpret_cast<cudaStream_t>(stream)));
}

cccl_status cccl_step_rotary_turns(int rot_dim, double base, double factor, double original_length, double few,
                                   double many, uint64_t* h_turns) {
    if (rot_dim < 16 || rot_dim > CCCL_KV_MAX_DIM || rot_dim % 16 != 0 || h_turns == nullptr || !(base > 0) ||
        !std::isfinite(base) || !(factor > 0) || !std::isfinite(factor) || !(original_length >= 0) ||
        !std::isfinite(original_length) ||
        (original_length > 0 && !(few < many && std::isfinite(few) && std::isfinite(many))))
        return CCCL_ERR_INVALID_ARG;
    const double two_pi = 6.283185307179586476925;
    for (int i = 0; i < rot_dim / 2; ++i) {
        const double f = std::pow(base, -2.0 * i / rot_dim);
        double stay = 0.0;
        if (original_length > 0) {
            stay = (original_length * f / two_pi - few) / (many - few);
            stay = stay < 0.0 ? 0.0 : (stay > 1.0 ? 1.0 : stay);
        }
        // whole turns a position change nothing
        double turn = (stay * f + (1.0 - stay) * (f / factor)) / two_pi;
        if (!std::isfinite(turn)) return CCCL_ERR_INVALID_ARG;
        turn -= std::floor(turn);
        const double scaled = std::ldexp(turn, 64);
        h_turns[i] = scaled >= 18446744073709551616.0 ? 0 : (uint64_t)scaled;
    }
    return CCCL_OK;
}

cccl_status cccl_step_write(const cccl_kv_cache* h_cache, const cccl_kv_batch* h_batch, const cccl_step_rotary* h_rotary,
                            const int32_t* d_positions, const void* d_q, int q_heads, int64_t q_token_stride,
                            int64_t q_head_stride, void* d_q_out, int64_t qo_token_stride, int64_t qo_head_stride,
                            const void* d_k, int64_t k_token_stride, int64_t k_head_stride, const void* d_v,
                            int64_t v_token_stride, int64_t v_head_stride, void* d_ws, size_t ws_bytes,
                            cccl_stream_t stream) {
    const cccl_kv_cache* c = h_cache;
    const cccl_kv_batch* b = h_batch;
    const cccl_step_rotary* r = h_rotary;
    if (!shapes_ok(c, b) || r == nullptr || r->reserved != 0 || r->rot_dim < 16 || r->rot_dim > c->head_dim ||
        r->rot_dim % 16 != 0 || (r->interleaved != 0 && r->interleaved != 1) || q_heads < 0 ||
        q_heads > CCCL_KV_MAX_HEADS || !std::isfinite(r->magnitude))
        return CCCL_ERR_INVALID_ARG;
    if (empty(b)) return CCCL_OK;
    cccl::KvArgs a{};
    Pointers at;
    if (!fill(c, b, d_ws, ws_bytes, sizeof(cccl::WsHeader), &a) || !at.numbers(r->turns, r->rot_dim / 2, 8) ||
        (d_positions != nullptr && !at.numbers(d_positions, b->n_tokens, 4)) ||
        !packed_ok(d_k, b->n_tokens, c->kv_heads, c->head_dim, k_token_stride, k_head_stride) ||
        !packed_ok(d_v, b->n_tokens, c->kv_heads, c->head_dim, v_token_stride, v_head_stride))
        return CCCL_ERR_INVALID_ARG;
    if (q_heads > 0 && (!packed_ok(d_q, b->n_tokens, q_heads, c->head_dim, q_token_stride, q_head_stride) ||
                        !packed_ok(d_q_out, b->n_tokens, q_heads, c->head_dim, qo_token_stride, qo_head_stride)))
        return CCCL_ERR_INVALID_ARG;
    const cccl::KvPacked x{static_cast<uint8_t*>(const_cast<void*>(d_k)), static_cast<uint8_t*>(const_cast<void*>(d_v)),
                           2 * k_token_stride, 2 * k_head_stride, 2 * v_token_stride, 2 * v_head_stride};
    cccl::RotaryArgs q{};
    q.turns = r->turns;
    q.positions = d_positions;
    q.q = static_cast<const uint8_t*>(d_q);
    q.q_out = static_cast<uint8_t*>(d_q_out);
    q.q_token = 2 * q_token_stride;
    q.q_head = 2 * q_head_stride;
    q.o_token = 2 * qo_token_stride;
    q.o_head = 2 * qo_head_stride;
    q.magnitude = r->magnitude;
    q.rot_dim = r->rot_dim;
    q.q_heads = q_heads;
    return status_of(cccl::launch_step_write(c->dtype, c->format, a, x, q, r->interleaved != 0,
                                             reinterpret_cast<cudaStream_t>(stream)));
}

cccl_status cccl_step_attention(const cccl_kv_cache* h_cache, const cccl_kv_batch* h_batch, const void* d_q, int q_heads,
                                int64_t q_token_stride, int64_t q_head_stride, float scale, const uint32_t* d_mask,
                                int64_t mask_stride, int mask_words, int64_t window, void* d_out,
                                int64_t o_token_stride, int64_t o_head_stride, float* d_lse, void* d_ws,
                                size_t ws_bytes, cccl_stream_t stream) {
    const cccl_kv_cache* c = h_cache;
    const cccl_kv_batch* b = h_batch;
    if (!shapes_ok(c, b) || q_heads < 1 || q_heads > CCCL_KV_MAX_HEADS || q_heads % c->kv_heads != 0 || window < 0 ||
        mask_words < 1 || mask_words > (1 << 20) || mask_stride < mask_words || !std::isfinite(scale))
        return CCCL_ERR_INVALID_ARG;
    if (empty(b)) return CCCL_OK;
    if (b->n_tokens > INT32_MAX / q_heads) return CCCL_ERR_INVALID_ARG;
    cccl::KvArgs a{};
    Pointers at;
    if (!fill(c, b, d_ws, ws_bytes, cccl_kv_workspace_bytes(c, b, q_heads), &a) ||
        !packed_ok(d_q, b->n_tokens, q_heads, c->head_dim, q_token_stride, q_head_stride) ||
        !packed_ok(d_out, b->n_tokens, q_heads, c->head_dim, o_token_stride, o_head_stride) ||
        !at.rows(d_mask, b->n_tokens, mask_stride, mask_words, 4) ||
        (d_lse != nullptr && !at.numbers(d_lse, b->n_tokens * q_heads, 4)))
        return CCCL_ERR_INVALID_ARG;
    cccl::TreeArgs t{};
    t.q = static_cast<const uint8_t*>(d_q);
    t.out = static_cast<uint8_t*>(d_out);
    t.lse = d_lse;
    t.q_token = 2 * q_token_stride;
    t.q_head = 2 * q_head_stride;
    t.o_token = 2 * o_token_stride;
    t.o_head = 2 * o_head_stride;
    t.window = window < INT32_MAX ? (int32_t)window : 0;  // one that hides nothing is none
    t.scale = scale;
    t.causal = 0;
    t.group = cccl::fast_div((uint32_t)(q_heads / c->kv_heads));
    t.q_heads = q_heads;
    t.mask = d_mask;
    t.mask_stride = mask_stride;
    t.words = mask_words;
    return status_of(cccl::launch_step_attention(c->dtype, c->format, a, t, b->max_new, b->max_len,
                                                 reinterpret_cast<cudaStream_t>(stream)));
}

cccl_status cccl_step_verify(const cccl_step_draft* h_draft, int32_t* d_path, int32_t* d_n_kept, int32_t* d_next,
                             void* d_ws, size_t ws_bytes, cccl_stream_t stream) {
    const cccl_step_draft* d = h_draft;
    if (d == nullptr || d->batch < 0 || d->batch > CCCL_KV_MAX_BATCH || d->rows < 0 || d->rows > INT32_MAX ||
        d->vocab < 1 || d->vocab > CCCL_STEP_MAX_VOCAB)
        return CCCL_ERR_INVALID_ARG;
    if (d->batch == 0) return CCCL_OK;
    Pointers at;
    if (!at.workspace(d_ws, ws_bytes) || !at.numbers(d->cu_tokens, (int64_t)d->batch + 1, 4) ||
        !at.numbers(d_n_kept, d->batch, 4) || !at.numbers(d_next, d->batch, 4))
        return CCCL_ERR_INVALID_ARG;
    if (d->rows > 0 &&
        (d->p_stride < d->vocab || !at.rows(d->p, d->rows, d->p_stride, d->vocab, 4) || !at.numbers(d->tokens, d->rows, 4) ||
         !at.numbers(d->uniform, d->rows, 4) || !at.numbers(d_path, d->rows, 4) ||
         (d->parents != nullptr && !at.numbers(d->parents, d->rows, 4)) ||
         (d->q != nullptr && (d->q_stride < d->vocab || !at.rows(d->q, d->rows, d->q_stride, d->vocab, 4)))))
        return CCCL_ERR_INVALID_ARG;
    cccl::VerifyArgs a{};
    a.p = d->p;
    a.q = d->q;
    a.p_stride = d->p_stride;
    a.q_stride = d->q_stride;
    a.rows = d->rows;
    a.tokens = d->tokens;
    a.parents = d->parents;
    a.cu = d->cu_tokens;
    a.uniform = d->uniform;
    a.path = d_path;
    a.n_kept = d_n_kept;
    a.next = d_next;
    a.ws = static_cast<cccl::WsHeader*>(d_ws);
    a.batch = d->batch;
    a.vocab = d->vocab;
    return status_of(cccl::launch_step_verify(a, reinterpret_cast<cudaStream_t>(stream)));
}

cccl_status cccl_step_keep(const cccl_kv_cache* h_cache, const cccl_kv_batch* h_batch, const int32_t* d_path,
                           const int32_t* d_n_kept, int32_t* d_lens, void* d_ws, size_t ws_bytes, cccl_stream_t stream) {
    const cccl_kv_cache* c = h_cache;
    const cccl_kv_batch* b = h_batch;
    if (!shapes_ok(c, b)) return CCCL_ERR_INVALID_ARG;
    if (b->batch == 0) return CCCL_OK;
    cccl::KvArgs a{};
    Pointers at;
    if (!fill(c, b, d_ws, ws_bytes, sizeof(cccl::WsHeader), &a) || !at.numbers(d_n_kept, b->batch, 4) ||
        (d_lens != nullptr &&
         (!at.numbers(d_lens, b->batch, 4) || !apart(d_lens, b->batch, b->kv_lens, b->batch) ||
          !apart(d_lens, b->batch, b->cu_tokens, (int64_t)b->batch + 1) ||
          !apart(d_lens, b->batch, d_n_kept, b->batch) || !apart(d_lens, b->batch, d_path, b->n_tokens) ||
          !apart(d_lens, b->batch, b->page_table, b->table_pages, b->batch, b->table_stride))) ||
        (b->n_tokens > 0 && !at.numbers(d_path, b->n_tokens, 4)))
        return CCCL_ERR_INVALID_ARG;
    const cccl::KeepArgs x{d_path, d_n_kept, d_lens};
    return status_of(cccl::launch_step_keep(c->format, a, x, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
