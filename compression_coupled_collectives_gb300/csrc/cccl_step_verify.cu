// cccl_step_verify.cu -- which drafted tokens the target keeps, and the next one.
//
// A cluster of blocks a sequence.  Its first block's first warp goes through the
// tree; what needs a whole row of probabilities is done by all blocks, each over
// its part of the row: a pass adds up R = max(p - A q, 0) warp by warp, and for
// the next token the warp in whose part the sum passes u S looks its values
// through again.  The first block says what to do next (Order); the others follow,
// so that all meet at the same barriers whatever is in memory.
//
// Most steps take one pass: sums before it are only needed for a second child's
// chance where the draft gave probabilities.  So the time is one read of a row of
// p (and q) a sequence, behind the chain of loads that leads to it (rows, tokens
// and parents, probabilities of the tokens): one sequence takes 7.4 to 8.9 us (128000
// values, with q), every further one 0.16, its 1 MB at 6.2 TB/s.  64 chains of 4
// drafted: 19.6 us (45 MB: q only where a child was refused; floor 6.7); 16 trees of
// up to 33, 50257 values, no q: 9.0.  A second refused child and each one after it
// takes a pass and two barriers more, 9 to 10 us (16 sequences: 12).  On
// the way there, of 33.1: four blocks of 256 threads an SM instead of two of 512
// 30.6; a search of 16 values a lane, tests in whole numbers 25.4; loads a step
// ahead of their use, the search from the step that holds it 23.4; code for each
// form of R 19.5.
//
// Sums: a value is taken as an integer multiple of 2^-56 (a binary32 number has 24
// bits, so those above 2^-33 lose nothing and 2^17 smaller ones lose 2^-39 in all),
// and integer sums do not depend on their order: neither on how a row is divided
// nor on the number of blocks.
#include "cccl_kv_launch.h"
#include "cccl_kv_schedule.cuh"
#include "cccl_step.cuh"

namespace cccl {

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32, kMostBlocks = 8;
constexpr int kBlocksPerSm = 4;
// Values are gone through 512 at a time.  kSteps: of the longest part (2^20 values
// in 64 parts, or 2^12 or less in 8).
constexpr int kFlight = 4, kStep = 128 * kFlight, kSteps = (1 << 20) / (kMostBlocks * kWarps) / kStep;
constexpr uint64_t kOne = 1ull << 53;    // A of 1
constexpr uint64_t kWhole = 1ull << 56;  // a sum of 1

// x limited to 0..1, what is not a number to 0 (as __saturatef has it), and the
// same in multiples of 2^-56, cut off: 2^(e - 127) m / 2^23 2^56 with e the
// exponent's and m the fraction's bits (subnormals fall off).
__device__ __forceinline__ float limited(float x) { return __saturatef(x); }
__device__ __forceinline__ uint64_t fixed(float x) {
    const uint32_t b = __float_as_uint(limited(x)), e = b >> 23, m = (b & 0x7FFFFFu) | 0x800000u;
    return ((uint64_t)m << 33) >> min(127u - e, 63u);
}
// a b < c 2^56 for factors of up to 64 bits and c below 2^64
__device__ __forceinline__ bool product_below(uint64_t a, uint64_t b, uint64_t c) {
    const uint64_t hi = __umul64hi(a, b), lo = a * b;
    return hi < c >> 8 || (hi == c >> 8 && lo < c << 56);
}
// u q < p, exactly (u q = h + e)
__device__ __forceinline__ bool product_below(float u, float q, float p) {
    const float h = u * q, e = fmaf(u, q, -h);
    return h < p || (h == p && e < 0.f);
}
// A (in multiples of 2^-53, up to one for every token) times q, at most 2^60:
// that is 16, and p is at most 1
__device__ __forceinline__ uint64_t times(uint64_t A, uint64_t q) {
    const uint64_t hi = __umul64hi(A, q);
    return hi >= 1ull << 49 ? 1ull << 60 : (hi << 11) | ((A * q) >> 53);
}
// R of one value.  Most rows are taken as they are (A = 0) or without one q (A =
// 1); code for those alone saves a third of the instructions.
enum Mode { kPlain, kLessOne, kLessA };
template <Mode MODE>
__device__ __forceinline__ uint64_t weight(float p, float q, uint64_t A) {
    const uint64_t x = fixed(p);
    if (MODE == kPlain) return x;
    const uint64_t y = fixed(q);
    const int64_t d = (int64_t)(x - (MODE == kLessOne ? y : times(A, y)));
    return (uint64_t)(d & ~(d >> 63));
}
__device__ __forceinline__ uint64_t warp_sum64(uint64_t x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
    return x;
}

struct alignas(16) Order {
    int64_t row;       // of p and q; -1: the sequence has none
    uint64_t A;
    uint64_t u;        // of the next token, in multiples of 2^-56
    int32_t last;      // the next token is drawn (else only the sum is wanted)
    int32_t refused;   // how many tokens p is taken without
};
struct Shared {
    Order order;                    // the first block's
    uint64_t totals[kMostBlocks];   // of every block, in every block
    uint64_t warps[kWarps];
    uint64_t upto[kWarps][kSteps];  // of each warp's part, after every step
    int32_t refused[kMaxDraft];     // the first block's; then every block's copy
    int32_t parent[kMaxDraft], token[kMaxDraft], kept[kMaxDraft];
    float p[kMaxDraft], q[kMaxDraft], u[kMaxDraft];
};

// The first warp's way through the tree.
struct Way {
    int32_t at, next, kept;  // current token, the next to look at, how many are kept
    uint64_t A;
    uint64_t left;   // without q: S, in multiples of 2^-56
    int32_t refused;
    bool known;      // the sum at A has been taken
    uint64_t sum;
};
// On to the end (true) or to where a sum is needed.
template <bool DRAFT>
__device__ __forceinline__ bool advance(Shared& s, int32_t n, Way& w) {
    const int lane = threadIdx.x & 31;
    for (;;) {
        // the next token whose parent is the current one
        int32_t i = -1;
        for (int32_t base = w.next & ~31; base < n && i < 0; base += 32) {
            const int32_t k = base + lane;
            const uint32_t mine = __ballot_sync(0xFFFFFFFFu, k >= w.next && k < n && s.parent[k] == w.at);
            if (mine != 0) i = base + __ffs(mine) - 1;
        }
        if (i < 0) return true;
        const int32_t x = s.token[i];
        const float p = limited(s.p[i]), u = s.u[i];
        bool keep, again = false;
        if (DRAFT) {
            const float q = limited(s.q[i]);
            if (w.A == 0) {
                keep = product_below(u, q, p);
            } else {
                if (!w.known) {
                    w.next = i;
                    return false;
                }
                keep = (double)u * ((double)w.sum * 0x1p-56) * (double)q < (double)weight<kLessA>(p, q, w.A) * 0x1p-56;
            }
        } else {
            for (int32_t k = lane; k < w.refused; k += 32) again |= s.refused[k] == x;
            again = __any_sync(0xFFFFFFFFu, again) != 0;
            keep = !again && product_below(fixed(u), w.left, fixed(p));
        }
        w.next = i + 1;
        if (keep) {
            if (lane == 0) s.kept[w.kept] = i;
            ++w.kept;
            w.at = i;
            w.A = 0;
            w.left = kWhole;
            w.refused = 0;
        } else if (DRAFT) {
            w.A += w.A == 0 ? kOne : w.sum >> 3;
        } else if (!again) {
            if (lane == 0) s.refused[w.refused] = x;
            ++w.refused;
            w.left -= min(w.left, fixed(p));
        }
        w.known = false;
        __syncwarp();
    }
}

// A warp's part of a row: values from .. to - 1.
struct Part {
    int32_t from, to;
};
__device__ __forceinline__ Part part_of(int32_t vocab, int blocks, int rank, int warp) {
    const int32_t each = ((vocab + blocks * kWarps - 1) / (blocks * kWarps) + 127) & ~127;
    const int64_t from = (int64_t)(rank * kWarps + warp) * each;
    return Part{(int32_t)min(from, (int64_t)vocab), (int32_t)min(from + each, (int64_t)vocab)};
}
// Values at .. at + 3 (VEC; lanes side by side) or at, at + 32, at + 64, at + 96.
template <bool VEC>
__device__ __forceinline__ void load4(const float* row, int32_t at, int32_t to, float* x) {
    if (VEC && at + 4 <= to) {
        const float4 v = *reinterpret_cast<const float4*>(row + at);
        x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
        return;
    }
    constexpr int kStep = VEC ? 1 : 32;
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = at + i * kStep < to ? row[at + i * kStep] : 0.f;
}

// The part's sum, and after every step the sum so far.  A load follows the use of
// what it replaces, so that most of a step's loads are always on their way.
template <Mode MODE, bool VEC>
__device__ __forceinline__ uint64_t add_up(const float* p, const float* q, const Order& o, const Part& part,
                                           uint64_t* upto) {
    const int lane = threadIdx.x & 31;
    constexpr bool both = MODE != kPlain;
    float x[kFlight][4], y[kFlight][4] = {};
    int32_t at = part.from + (VEC ? 4 * lane : lane);
#pragma unroll
    for (int k = 0; k < kFlight; ++k) {
        load4<VEC>(p, at + 128 * k, part.to, x[k]);
        if (both) load4<VEC>(q, at + 128 * k, part.to, y[k]);
    }
    uint64_t sum = 0;
    int step = 0;
    for (int32_t base = part.from; base < part.to; base += kStep, ++step) {
        at += kStep;
#pragma unroll
        for (int k = 0; k < kFlight; ++k) {
#pragma unroll
            for (int i = 0; i < 4; ++i) sum += weight<MODE>(x[k][i], y[k][i], o.A);
            load4<VEC>(p, at + 128 * k, part.to, x[k]);
            if (both) load4<VEC>(q, at + 128 * k, part.to, y[k]);
        }
        const uint64_t all = warp_sum64(sum);
        if (lane == 0) upto[step] = all;
    }
    __syncwarp();
    return step > 0 ? upto[step - 1] : 0;
}

// The first value of the part at which the running sum passes `goal` (it does so
// within the part), by one warp: 16 values in a row a lane, from the step on whose
// sum passes it (upto counts refused tokens too: an earlier step may hold it, never
// a later one, so with refused tokens the search begins at the front).
template <Mode MODE, bool VEC>
__device__ __forceinline__ int32_t find(const float* p, const float* q, const Order& o, const int32_t* refused,
                                        const Part& part, uint64_t goal, const uint64_t* upto) {
    constexpr int kEach = 16;
    static_assert(32 * kEach == kStep, "");
    const int lane = threadIdx.x & 31;
    int step = 0;
    if (o.refused == 0) {
        const int steps = (part.to - part.from + kStep - 1) / kStep;
        const uint32_t below = __ballot_sync(0xFFFFFFFFu, lane < steps && upto[min(lane, kSteps - 1)] <= goal);
        step = __popc(below);
        if (step > 0) goal -= upto[step - 1];
    }
    for (int32_t base = part.from + step * kStep; base < part.to; base += kStep) {
        const int32_t at = base + kEach * lane;
        float x[kEach], y[kEach] = {};
        if constexpr (VEC) {
#pragma unroll
            for (int k = 0; k < kEach; k += 4) {
                load4<true>(p, at + k, part.to, x + k);
                if (MODE != kPlain) load4<true>(q, at + k, part.to, y + k);
            }
        } else {
#pragma unroll
            for (int k = 0; k < kEach; ++k) {
                x[k] = at + k < part.to ? p[at + k] : 0.f;
                if (MODE != kPlain) y[k] = at + k < part.to ? q[at + k] : 0.f;
            }
        }
        for (int32_t i = 0; i < o.refused; ++i) {
            const int32_t k0 = refused[i] - at;
#pragma unroll
            for (int k = 0; k < kEach; ++k) x[k] = k == k0 ? 0.f : x[k];
        }
        uint64_t all = 0;
#pragma unroll
        for (int k = 0; k < kEach; ++k) all += weight<MODE>(x[k], y[k], o.A);
        uint64_t run_to = all;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const uint64_t z = __shfl_up_sync(0xFFFFFFFFu, run_to, d);
            if (lane >= d) run_to += z;
        }
        const uint32_t past = __ballot_sync(0xFFFFFFFFu, run_to > goal);
        if (past == 0) {
            goal -= __shfl_sync(0xFFFFFFFFu, run_to, 31);
            continue;
        }
        // the lane's first value at which its own sum passes what is left
        const uint64_t left = goal - (run_to - all);
        int32_t mine = kEach;
        uint64_t run = 0;
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            run += weight<MODE>(x[k], y[k], o.A);
            if (run > left && mine == kEach) mine = k;
        }
        return __shfl_sync(0xFFFFFFFFu, at + mine, __ffs(past) - 1);
    }
    return part.from;  // (not reached: the part's sum is above the goal)
}

template <bool DRAFT, bool VEC>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm) verify_kernel(const __grid_constant__ VerifyArgs a, int blocks) {
    __shared__ Shared s;
    const int rank = (int)cluster_rank(), b = (int)blockIdx.x / blocks;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int64_t row0 = 0;
    int32_t rows = 0, n = 0;
    Way w{0, 1, 1, 0, kWhole, 0, false, 0};
    if (rank == 0) {
        const int64_t lo = a.cu[b], hi = a.cu[b + 1];
        row0 = min(max(lo, (int64_t)0), a.rows);
        const int64_t end = min(max(hi, row0), a.rows);
        rows = (int32_t)(end - row0);
        n = min(rows, kMaxDraft);
        if (threadIdx.x == 0 && (row0 != lo || end != hi || n < rows)) record_error(a.ws, kStatusInvalidArg);
        for (int32_t i = threadIdx.x; i < n; i += kThreads) {
            int32_t up = -1;
            float p = 0.f, q = 0.f;
            const int32_t x = a.tokens[row0 + i];
            if (i > 0 && x >= 0 && x < a.vocab) {
                up = a.parents != nullptr ? a.parents[row0 + i] : i - 1;
                if (up < 0 || up >= i) up = -1;
                if (up >= 0) {
                    p = a.p[(row0 + up) * a.p_stride + x];
                    if (DRAFT) q = a.q[(row0 + up) * a.q_stride + x];
                }
            }
            s.parent[i] = up;
            s.token[i] = x;
            s.p[i] = p;
            s.q[i] = q;
            s.u[i] = a.uniform[row0 + i];
        }
        if (threadIdx.x == 0) s.kept[0] = 0;
        __syncthreads();
    }
    for (;;) {
        if (rank == 0 && warp == 0) {
            Order o{-1, 0, 0, 1, 0};
            if (n > 0) {
                o.last = advance<DRAFT>(s, n, w) ? 1 : 0;
                o.row = row0 + w.at;
                o.A = w.A;
                o.u = fixed(s.u[0]);
                o.refused = DRAFT ? 0 : w.refused;
            }
            if (lane == 0) {
                s.order = o;
                a.next[b] = n > 0 ? 0 : -1;  // (some token also where a row's sum leaves 64 bits)
            }
        }
        __syncthreads();
        cluster_sync();
        Order o;
        {
            const uint32_t at = in_block(smem_addr(&s.order), 0);
            const float4 lo = load_cluster4(at), hi = load_cluster4(at + 16);
            memcpy(&o, &lo, 16);
            memcpy(reinterpret_cast<char*>(&o) + 16, &hi, 16);
            if (rank != 0)
                for (int32_t i = threadIdx.x; i < o.refused; i += kThreads)
                    s.refused[i] = __float_as_int(load_cluster(in_block(smem_addr(&s.refused[i]), 0)));
        }
        __syncthreads();
        if (o.row < 0) {  // no rows at all
            if (rank == 0 && threadIdx.x == 0) a.n_kept[b] = 0;
            __syncwarp();
            cluster_sync();  // the first block's order has been read
            return;
        }
        const float* p = a.p + o.row * a.p_stride;
        const float* q = DRAFT ? a.q + o.row * a.q_stride : nullptr;
        const Part part = part_of(a.vocab, blocks, rank, warp);
        uint64_t total = 0;
        for (int turn = 0; turn < 2; ++turn) {
            const Mode mode = !DRAFT || o.A == 0 ? kPlain : (o.A == kOne ? kLessOne : kLessA);
            uint64_t sum = mode == kPlain     ? add_up<kPlain, VEC>(p, q, o, part, s.upto[warp])
                           : mode == kLessOne ? add_up<kLessOne, VEC>(p, q, o, part, s.upto[warp])
                                              : add_up<kLessA, VEC>(p, q, o, part, s.upto[warp]);
            if (o.refused > 0) {
                uint64_t off = 0;
                for (int32_t k = lane; k < o.refused; k += 32)
                    if (s.refused[k] >= part.from && s.refused[k] < part.to) off += fixed(p[s.refused[k]]);
                __syncwarp();
                sum -= warp_sum64(off);
            }
            if (lane == 0) s.warps[warp] = sum;
            __syncthreads();
            if (threadIdx.x < (uint32_t)blocks) {
                uint64_t mine = 0;
                for (int i = 0; i < kWarps; ++i) mine += s.warps[i];
                const uint32_t to = in_block(smem_addr(&s.totals[rank]), threadIdx.x);
                asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(to), "l"(mine) : "memory");
            }
            __syncwarp();
            cluster_sync();
            total = 0;
            for (int i = 0; i < blocks; ++i) total += s.totals[i];
            if (!o.last || total != 0) break;
            // nothing is left of p: the next token comes from p itself
            if (o.A == 0 && o.refused == 0) break;
            o.A = 0;
            o.refused = 0;
            cluster_sync();  // everyone has the totals
        }
        if (!o.last) {
            w.sum = total;
            w.known = true;
            continue;
        }
        if (total == 0) {
            if (rank == 0 && threadIdx.x == 0) record_error(a.ws, kStatusInvalidArg);
        } else {
            uint64_t goal = (__umul64hi(total, o.u) << 8) | ((total * o.u) >> 56);
            if (goal >= total) goal = total - 1;
            uint64_t before = 0;  // of the values before this warp's
            for (int i = 0; i < rank; ++i) before += s.totals[i];
            for (int i = 0; i < warp; ++i) before += s.warps[i];
            if (before <= goal && goal - before < s.warps[warp]) {
                const uint64_t left = goal - before;
                const int32_t y =
                    !DRAFT || o.A == 0 ? find<kPlain, VEC>(p, q, o, s.refused, part, left, s.upto[warp])
                    : o.A == kOne      ? find<kLessOne, VEC>(p, q, o, s.refused, part, left, s.upto[warp])
                                       : find<kLessA, VEC>(p, q, o, s.refused, part, left, s.upto[warp]);
                if (lane == 0) a.next[b] = y;
            }
        }
        break;
    }
    if (rank == 0) {
        for (int32_t i = threadIdx.x; i < rows; i += kThreads) a.path[row0 + i] = -1;
        __syncthreads();
        if (warp == 0) {  // the one that knows
            for (int32_t i = lane; i < w.kept; i += 32) a.path[row0 + i] = s.kept[i];
            if (lane == 0) a.n_kept[b] = w.kept;
        }
    }
}

template <bool DRAFT, bool VEC>
cudaError_t launch_one(const VerifyArgs& a, cudaStream_t s) {
    // a warp's part is at least 128 values; 8 blocks a sequence while that leaves them some
    int blocks = kMostBlocks;
    while (blocks > 1 && a.vocab <= blocks * kWarps * 64) blocks /= 2;
    return launch_clusters(verify_kernel<DRAFT, VEC>, a.batch * blocks, blocks, kThreads, 0, s, a, blocks);
}

}  // namespace

cudaError_t launch_step_verify(const VerifyArgs& a, cudaStream_t s) {
    const bool wide = (reinterpret_cast<uintptr_t>(a.p) & 15) == 0 && a.p_stride % 4 == 0;
    if (a.q == nullptr) return wide ? launch_one<false, true>(a, s) : launch_one<false, false>(a, s);
    const bool both = wide && (reinterpret_cast<uintptr_t>(a.q) & 15) == 0 && a.q_stride % 4 == 0;
    return both ? launch_one<true, true>(a, s) : launch_one<true, false>(a, s);
}

}  // namespace cccl
