// cccl_step_plan.cu -- block tables, slot maps, positions and masks of one step.
//
// A few numbers a sequence and a few bytes a row: the time is the launch and the
// chain of loads behind one another.  One cluster of 8 blocks does it all.  Every
// block reads the batch (a thread a sequence) and works out the running sums of
// rows and of pages given, so that only one barrier is needed: after it nothing
// that was read is needed again, and the results may lie where the inputs did.
// Rows and pages are then divided among all of the cluster's threads; a row's
// page is looked up in the table where the sequence held it before, else among
// the free ones, so that nobody waits for the table's new entries.  64 trees of up to
// 33 tokens: 5.9 us, of which an empty launch is half; 32 prompts, 63588 rows: 7.2.
// A row of a tree walks to its root, a load a level, so deep ones take long: a chain
// of 64 given as parents 7.1 us, of 256 27.5, of 1024 287, eight of those 2270 (the
// same chains as none given: 4.7).
#include "cccl_kv_launch.h"
#include "cccl_kv_schedule.cuh"
#include "cccl_step.cuh"

namespace cccl {

namespace {

constexpr int kBlocks = 8, kThreads = 1024;

struct Sums {
    uint32_t rows[kMaxSequences + 1], pages[kMaxSequences + 1];  // before sequence b
    int32_t lens[kMaxSequences], held[kMaxSequences];
    uint64_t warp_rows[32], warp_pages[32];
};

// The sequence of place x of a line: first[b] <= x < first[b + 1].
__device__ __forceinline__ int owner(const uint32_t* first, int batch, uint32_t x) {
    int lo = 0, hi = batch;
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (first[mid] <= x)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

// LANES lanes a row of a tree: each holds one word of its mask.
template <int LANES>
__device__ __forceinline__ void trees(const PlanArgs& a, const Sums& s, uint32_t rows, int me, int all) {
    const int lane = me % LANES;
    for (uint32_t row = (uint32_t)me / LANES; row < rows; row += (uint32_t)(all / LANES)) {
        const int b = owner(s.rows, a.batch, row);
        const uint32_t first = s.rows[b];
        int32_t k = (int32_t)(row - first), depth = 0;
        uint32_t bits = 0;
        if (a.parents == nullptr) {  // every token before it
            const int32_t n = k + 1 - 32 * lane;
            bits = n <= 0 ? 0u : (n >= 32 ? ~0u : (1u << n) - 1u);
            depth = k;
        } else {
            while (true) {  // k falls with every turn
                if (k >> 5 == lane) bits |= 1u << (k & 31);
                const int32_t up = a.parents[(int64_t)first + k];
                if (up >= k || up < -1) record_error(a.ws, kStatusInvalidArg);
                if (up >= k || up < 0) break;
                k = up;
                ++depth;
            }
        }
        if (a.mask != nullptr && lane < a.words) a.mask[(int64_t)row * a.mask_stride + lane] = bits;
        if (a.positions != nullptr && lane == 0) a.positions[row] = s.lens[b] + depth;
    }
}

// Slots, and positions where no tree gives them: 32 ROWS rows a warp at a time, one
// search, then a step or two, ROWS rows' loads in flight.  (32 prompts, 63588 rows:
// 8.7 us with one, 7.2 with four; 64 trees, 1378 rows: 5.9 and 7.0.)
template <int ROWS>
__device__ __forceinline__ void places(const PlanArgs& a, const Sums& s, uint32_t rows, int64_t count, bool walk, int me,
                                       int all) {
    const int lane = me & 31;
    for (uint32_t base = (uint32_t)(me >> 5) * 32 * ROWS; base < rows; base += (uint32_t)all * ROWS) {
        int o = owner(s.rows, a.batch, base);
        int64_t page[ROWS];
        uint32_t slot[ROWS];
#pragma unroll
        for (int k = 0; k < ROWS; ++k) {
            const uint32_t row = base + 32 * k + (uint32_t)lane;
            page[k] = slot[k] = 0;
            if (row >= rows) continue;
            while (s.rows[o + 1] <= row) ++o;
            const int32_t pos = s.lens[o] + (int32_t)(row - s.rows[o]);
            if (!walk && a.positions != nullptr) a.positions[row] = pos;
            if (a.slots == nullptr) continue;
            const uint32_t pi = div_by(a.page_tokens, (uint32_t)pos);
            slot[k] = (uint32_t)pos - pi * a.page_tokens.d;
            const int32_t ahead = (int32_t)pi - s.held[o];
            page[k] = ahead < 0 ? a.table[(int64_t)o * a.table_stride + pi]
                                : a.free_pages[count - 1 - (int64_t)s.pages[o] - ahead];
        }
        if (a.slots == nullptr) continue;
#pragma unroll
        for (int k = 0; k < ROWS; ++k) {
            const uint32_t row = base + 32 * k + (uint32_t)lane;
            if (row < rows) a.slots[row] = page[k] * (int64_t)a.page_tokens.d + slot[k];
        }
    }
}

__global__ void __launch_bounds__(kThreads) plan_kernel(const __grid_constant__ PlanArgs a) {
    __shared__ Sums s;
    __shared__ uint32_t wrong;
    const int b = threadIdx.x, warp = b >> 5, lane = b & 31;
    if (b == 0) wrong = 0;
    __syncthreads();
    const int64_t count = *a.free_count;
    int64_t fresh = 0, need = 0;
    int32_t len = 0, held = 0;
    if (b < a.batch) {
        len = a.lens[b];
        held = a.held[b];
        fresh = a.fresh[b];
        const int64_t most = min((int64_t)a.table_pages * a.page_tokens.d, (int64_t)0x7FFF0000);
        bool bad = len < 0 || held < 0 || held > a.table_pages || fresh < 0 || fresh > a.rows || len + fresh > most;
        if (a.mask != nullptr && fresh > 32 * a.words) bad = true;
        if (a.parents != nullptr && fresh > kMaxDraft) bad = true;  // (a walk up a chain takes as many loads)
        if (bad) {
            wrong = 1;
            fresh = 0;
        } else {
            const uint32_t after = (uint32_t)(len + fresh);
            need = max((after == 0 ? 0 : (int64_t)div_by(a.page_tokens, after - 1) + 1) - held, (int64_t)0);
        }
        s.lens[b] = len;
        s.held[b] = held;
    }
    uint64_t r = (uint64_t)fresh, g = (uint64_t)need;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint64_t x = __shfl_up_sync(0xFFFFFFFFu, r, o), y = __shfl_up_sync(0xFFFFFFFFu, g, o);
        if (lane >= o) {
            r += x;
            g += y;
        }
    }
    if (lane == 31) {
        s.warp_rows[warp] = r;
        s.warp_pages[warp] = g;
    }
    __syncthreads();
    if (warp == 0) {
        uint64_t x = s.warp_rows[lane], y = s.warp_pages[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint64_t u = __shfl_up_sync(0xFFFFFFFFu, x, o), v = __shfl_up_sync(0xFFFFFFFFu, y, o);
            if (lane >= o) {
                x += u;
                y += v;
            }
        }
        s.warp_rows[lane] = x;
        s.warp_pages[lane] = y;
    }
    __syncthreads();
    const uint64_t all_rows = s.warp_rows[31], all_pages = s.warp_pages[31];
    const bool counted = wrong == 0 && all_rows <= (uint64_t)a.rows && count >= 0 && count <= a.free_capacity;
    const bool fits = counted && all_pages <= (uint64_t)count;
    if (b < a.batch) {
        if (warp > 0) {
            r += s.warp_rows[warp - 1];
            g += s.warp_pages[warp - 1];
        }
        s.rows[b + 1] = fits ? (uint32_t)r : 0u;
        s.pages[b + 1] = fits ? (uint32_t)g : 0u;
    }
    if (b == 0) s.rows[0] = s.pages[0] = 0;
    __syncthreads();
    cluster_sync();  // everyone has read what the results may lie over
    const uint32_t rank = cluster_rank();
    if (rank == 0) {
        if (b < a.batch) {
            a.cu[b + 1] = (int32_t)s.rows[b + 1];
            a.lens_out[b] = fits ? (int32_t)(len + fresh) : len;
            a.held_out[b] = fits ? (int32_t)(held + need) : held;
        }
        if (b == 0) {
            a.cu[0] = 0;
            *a.count_out = (int32_t)(fits ? count - (int64_t)all_pages : count);
            if (!fits) record_error(a.ws, counted ? kStatusCapacity : kStatusInvalidArg);
        }
    }
    if (!fits) return;
    const int me = (int)rank * kThreads + b, all = kBlocks * kThreads;
    for (uint32_t i = (uint32_t)me; i < (uint32_t)all_pages; i += (uint32_t)all) {
        const int o = owner(s.pages, a.batch, i);
        a.table[(int64_t)o * a.table_stride + s.held[o] + (int64_t)(i - s.pages[o])] = a.free_pages[count - 1 - i];
    }
    const uint32_t rows = (uint32_t)all_rows;
    const bool walk = a.mask != nullptr || (a.parents != nullptr && a.positions != nullptr);
    if (walk) {
        if (a.words <= 1)
            trees<1>(a, s, rows, me, all);
        else if (a.words <= 2)
            trees<2>(a, s, rows, me, all);
        else if (a.words <= 4)
            trees<4>(a, s, rows, me, all);
        else if (a.words <= 8)
            trees<8>(a, s, rows, me, all);
        else
            trees<32>(a, s, rows, me, all);
    }
    if (a.slots == nullptr && (walk || a.positions == nullptr)) return;
    if (rows > 2u * (uint32_t)all)
        places<4>(a, s, rows, count, walk, me, all);
    else
        places<1>(a, s, rows, count, walk, me, all);
}

}  // namespace

cudaError_t launch_step_plan(const PlanArgs& a, cudaStream_t s) {
    return launch_clusters(plan_kernel, kBlocks, kBlocks, kThreads, 0, s, a);
}

}  // namespace cccl
