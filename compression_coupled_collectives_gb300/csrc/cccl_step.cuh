// cccl_step.cuh -- the launch arguments of the calls of a step with drafted
// tokens (include/cccl_step.h); attention's are in cccl_kv.cuh.
#pragma once

#include "cccl_kv.cuh"

namespace cccl {

constexpr int kMaxDraft = 1024;          // CCCL_STEP_MAX_DRAFT
constexpr int kMaxSequences = 1024;      // CCCL_KV_MAX_BATCH
constexpr uint32_t kStatusCapacity = 2;  // too few free pages

struct PlanArgs {
    const int32_t *lens, *fresh, *held, *free_pages, *free_count, *parents;
    int32_t* table;
    int64_t table_stride, free_capacity, rows;
    int32_t *cu, *lens_out, *held_out, *count_out, *positions;
    int64_t* slots;
    uint32_t* mask;
    int64_t mask_stride;
    WsHeader* ws;
    FastDiv page_tokens;
    int32_t batch, table_pages, words;
};

// Rotary positions, and the queries of a write (strides in bytes).
struct RotaryArgs {
    const uint64_t* turns;
    const int32_t* positions;  // or null
    const uint8_t* q;
    uint8_t* q_out;
    int64_t q_token, q_head, o_token, o_head;
    float magnitude;
    int32_t rot_dim, q_heads;
};

struct VerifyArgs {
    const float *p, *q;
    int64_t p_stride, q_stride, rows;
    const int32_t *tokens, *parents, *cu;
    const float* uniform;
    int32_t *path, *n_kept, *next;
    WsHeader* ws;
    int32_t batch, vocab;
};

struct KeepArgs {
    const int32_t *path, *n_kept;
    int32_t* lens;  // or null
};

}  // namespace cccl
