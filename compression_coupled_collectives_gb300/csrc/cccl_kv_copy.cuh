// cccl_kv_copy.cuh -- what the kernels share that bring packed tokens to the
// cache's pages and back: a block's tokens and where each of them lies.
#pragma once

#include "cccl_kv.cuh"

namespace cccl {

constexpr int kCopyThreads = 256;
constexpr int kMaxTokensPerBlock = 16;  // at most 32: a lane each when they are looked up

// Tokens t0 .. t0 + count - 1 of a block: where each lies in the cache, and
// whether it lies there at all.
struct TokenSlots {
    int64_t at[kMaxTokensPerBlock], scale_at[kMaxTokensPerBlock];
    int32_t pos[kMaxTokensPerBlock];   // its place in the sequence (may be negative)
    int8_t state[kMaxTokensPerBlock];  // 0 no sequence's row, 1 in the cache, 2 not in the cache
};
// Warp 0, a token a lane.  The first block's other warps meanwhile look at every
// sequence, for what no row leads to (a length, rows in no order).
__device__ __forceinline__ void find_slots(const KvArgs& a, int64_t t0, int count, TokenSlots& s) {
    const int lane = threadIdx.x & 31;
    if (threadIdx.x >= 32) {
        if (blockIdx.x == 0)
            for (int b = (int)threadIdx.x - 32; b < a.batch; b += kCopyThreads - 32) load_sequence(a, b);
        return;
    }
    // the last sequence that starts at or before t0: 32 candidates a step
    int lo = 0, hi = a.batch;  // starts at lo, or no sequence does
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32;
        const int c = lo + lane * step;
        const uint32_t le = __ballot_sync(0xFFFFFFFFu, c < hi && (lane == 0 || a.cu[c] <= t0));
        const int at = 31 - __clz(le);
        lo += at * step;
        hi = min(hi, lo + step);
    }
    if (lane >= count) return;
    const int64_t t = t0 + lane;
    while (lo + 1 < a.batch && a.cu[lo + 1] <= t) ++lo;
    const Sequence q = load_sequence(a, lo);
    int state = 0;
    int64_t at = 0, sat = 0, pos = 0;
    if (t >= q.row && t < q.row + q.n) {
        pos = (int64_t)q.len - q.n + (t - q.row);
        state = pos >= 0 && slot_of(a, lo, (uint32_t)pos, at, sat) ? 1 : 2;
    }
    s.at[lane] = at;
    s.scale_at[lane] = sat;
    s.pos[lane] = (int32_t)pos;
    s.state[lane] = (int8_t)state;
}

__device__ __forceinline__ uint4 load_stream(const void* p) {
    return __ldcs(reinterpret_cast<const uint4*>(p));
}

// Tokens of one block: 1 while that fills the GPU's 152 SMs with 8 blocks
// each, more (fewer searches of the batch per byte) beyond: reading 131072
// tokens took 130 us at 32, 126.5 at 16, 138 at 8.
inline int tokens_per_block(int64_t n) {
    const int64_t t = n / (152 * 8);
    return (int)(t < 1 ? 1 : (t > kMaxTokensPerBlock ? kMaxTokensPerBlock : t));
}

}  // namespace cccl
