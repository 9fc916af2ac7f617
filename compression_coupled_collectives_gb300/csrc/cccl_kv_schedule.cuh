// cccl_kv_schedule.cuh -- how attention's work is divided among thread blocks.
//
// Item: one sequence, one kv head and one tile of ROWS rows (a row is a new
// token and one of the `group` query heads that share the kv head, tokens
// outermost).  An item walks the cached tokens that any of its rows sees, in
// tiles of TOKENS aligned to multiples of TOKENS; one that sees none still
// counts as one tile, so that its zeros get written.  All items' tiles form
// one line, sequence by sequence, head by head, row tile by row tile, and each
// of C blocks takes an equal share of the line: sequences of any lengths load
// the GPU evenly, and one sequence's long context is shared by many blocks.
// An item that a share's end cuts leaves partial results (an unnormalised
// accumulator, its maximum and its sum for each row) that a second kernel
// joins, in the order of the line, so that results do not vary.  Few items are
// instead shared by a cluster of blocks each, which joins their parts itself.
//
// The lengths are in device memory, so every block works the division out
// itself (a few loads a sequence).
#pragma once

#include "cccl_kv.cuh"

namespace cccl {

constexpr int kMaxBatch = 1024;  // CCCL_KV_MAX_BATCH

// Row tile rt of a sequence: its visible tiles.
struct TileRange {
    int32_t first, last;  // visible tokens of any row: first .. last - 1
    int32_t lo, n;        // tiles lo .. lo + n - 1 (n >= 1)
};
// What any row of tile rt may see.
template <int ROWS>
__device__ __forceinline__ void tile_visible(const AttnArgs& t, const Sequence& s, int32_t rt, int32_t& first,
                                             int32_t& last) {
    const uint32_t rows = (uint32_t)s.n * t.group.d, r0 = (uint32_t)rt * ROWS;
    const int32_t base = s.len - s.n;
    int32_t ignore;
    visible_range(t, s, 0, base + (int32_t)div_by(t.group, r0), first, ignore);
    visible_range(t, s, 0, base + (int32_t)div_by(t.group, min(r0 + ROWS, rows) - 1), ignore, last);
}
// (Drafted tokens: whatever the masks say.  A row that sees none of them sees the
// last `window` tokens before them.)
template <int ROWS>
__device__ __forceinline__ void tile_visible(const TreeArgs& t, const Sequence& s, int32_t, int32_t& first,
                                             int32_t& last) {
    first = t.window > 0 ? (int32_t)max((int64_t)before_draft(s) - t.window, (int64_t)0) : 0;
    last = s.len;
}
// (A call's rows are below 2^31: n_tokens * q_heads is.)  TOKENS of 0 counts
// every item as one tile.
template <int ROWS, int TOKENS, class Args>
__device__ __forceinline__ TileRange tile_range(const Args& t, const Sequence& s, int32_t rt) {
    TileRange r;
    tile_visible<ROWS>(t, s, rt, r.first, r.last);
    if (r.first >= r.last) {
        r.first = r.last = r.lo = 0;
        r.n = 1;
    } else if constexpr (TOKENS == 0) {
        r.lo = 0;
        r.n = 1;
    } else {
        r.lo = r.first / TOKENS;
        r.n = (r.last + TOKENS - 1) / TOKENS - r.lo;
    }
    return r;
}
template <int ROWS>
__device__ __forceinline__ int32_t row_tiles(const AttnArgs& t, const Sequence& s) {
    return (int32_t)(((uint32_t)s.n * t.group.d + ROWS - 1) / ROWS);
}

// Block-wide: prefix[b] = tiles before sequence b on the line, prefix[batch] =
// all.  Ends with a barrier.  2^32 tiles would take hours: such lengths are
// reported as invalid and the line is empty.
template <int ROWS, int TOKENS, class Args>
__device__ __forceinline__ void build_prefix(const KvArgs& a, const Args& t, uint32_t* prefix) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    // a thread a sequence; those of many row tiles are left to a warp each
    constexpr int32_t kFew = 4;
    constexpr uint32_t kLeft = 0xFFFFFFFFu;
    for (int b = threadIdx.x; b < a.batch; b += blockDim.x) {
        const Sequence s = load_sequence(a, b);
        const int32_t rts = row_tiles<ROWS>(t, s);
        uint64_t sum = 0;
        for (int32_t rt = 0; rt < min(rts, kFew); ++rt) sum += (uint64_t)tile_range<ROWS, TOKENS>(t, s, rt).n;
        prefix[b + 1] = rts > kFew ? kLeft : (uint32_t)min(sum * (uint32_t)a.kv_heads, (uint64_t)(kLeft - 1));
    }
    __syncthreads();
    for (int b = warp; b < a.batch; b += warps) {
        if (prefix[b + 1] != kLeft) continue;
        const Sequence s = load_sequence(a, b);
        const int32_t rts = row_tiles<ROWS>(t, s);
        uint64_t sum = 0;
        for (int32_t rt = lane; rt < rts; rt += 32) sum += (uint64_t)tile_range<ROWS, TOKENS>(t, s, rt).n;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
        if (lane == 0) prefix[b + 1] = (uint32_t)min(sum * (uint32_t)a.kv_heads, (uint64_t)(kLeft - 1));
    }
    __syncthreads();
    if (warp == 0) {
        uint64_t carry = 0;
        for (int base = 0; base < a.batch; base += 32) {
            const int b = base + lane;
            uint64_t x = b < a.batch ? prefix[b + 1] : 0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint64_t y = __shfl_up_sync(0xFFFFFFFFu, x, o);
                if (lane >= o) x += y;
            }
            if (b < a.batch) prefix[b + 1] = (uint32_t)min(carry + x, (uint64_t)0xFFFFFFFFu);
            carry += __shfl_sync(0xFFFFFFFFu, x, 31);
        }
        if (lane == 0) prefix[0] = 0;
        if (carry >= kLeft - 1) {
            if (lane == 0) record_error(a.ws, kStatusInvalidArg);
            for (int b = lane; b < a.batch; b += 32) prefix[b + 1] = 0;
        }
    }
    __syncthreads();
}

// One block's part of one item.
struct Piece {
    Sequence seq;
    TileRange range;
    int32_t b, kv_head, rt;
    uint32_t item;        // the item's start on the line
    int32_t from, count;  // its tiles range.lo + from .. + count - 1
};

// Share c of a line of T = each * shares + rest tiles begins at
// floor(T c / shares).
struct Line {
    uint32_t each, rest, shares;
};
__device__ __forceinline__ uint32_t share_start(const Line& l, uint32_t c) {
    return l.each * c + l.rest * c / l.shares;  // rest, c < 2^9
}

// One block's share of the line, piece by piece (a whole warp at a time).
struct Walk {
    Line line;
    uint32_t x, x1, share;
    int32_t whole;  // items are not cut: the block that an item begins in does all of it
    int32_t begun;  // the caller's piece is the one before
};
__device__ __forceinline__ Walk make_walk(uint32_t T, uint32_t share, uint32_t blocks, int whole) {
    Walk w;
    w.share = share;
    w.line.shares = max(min(blocks, T), 1u);  // a tile each at least
    w.line.each = T / w.line.shares;
    w.line.rest = T - w.line.each * w.line.shares;
    w.x = share < w.line.shares ? share_start(w.line, share) : T;
    w.x1 = share < w.line.shares ? share_start(w.line, share + 1) : T;
    w.whole = whole;
    w.begun = 0;
    return w;
}
// The next piece; false at the share's end.  p is the piece before, once there
// was one.  (Items after the first are reached by stepping on; what finds the
// first shares its code with that, since all of it runs cold.)
template <int ROWS, int TOKENS, class Args>
__device__ __forceinline__ bool next_piece(const KvArgs& a, const Args& t, const uint32_t* prefix, Walk& w,
                                           Piece& p) {
    const int lane = threadIdx.x & 31;
    while (w.x < w.x1) {
        bool enter = w.begun == 0;  // another sequence
        if (w.begun == 0) {
            int lo = 0, hi = a.batch;  // prefix[lo] <= x < prefix[hi]
#pragma unroll 1
            while (hi - lo > 1) {
                const int mid = (lo + hi) / 2;
                if (prefix[mid] <= w.x)
                    lo = mid;
                else
                    hi = mid;
            }
            p.b = lo;
        } else {
            p.item += (uint32_t)p.range.n;
            if (++p.rt >= row_tiles<ROWS>(t, p.seq)) {
                p.rt = 0;
                if (++p.kv_head >= a.kv_heads) {
                    p.kv_head = 0;
                    enter = true;
                    do ++p.b;
                    while (prefix[p.b + 1] == prefix[p.b]);  // no new tokens
                }
            }
        }
        if (enter) p.seq = load_sequence(a, p.b);
        if (w.begun == 0) {
            const uint32_t per_head = (prefix[p.b + 1] - prefix[p.b]) / (uint32_t)a.kv_heads;
            p.kv_head = (int32_t)((w.x - prefix[p.b]) / per_head);
            p.item = prefix[p.b] + (uint32_t)p.kv_head * per_head;
            // the first row tile whose tiles reach past x: 32 row tiles at a time
            const int32_t rts = row_tiles<ROWS>(t, p.seq);
#pragma unroll 1
            for (int32_t base = 0;; base += 32) {
                const uint32_t n = base + lane < rts ? (uint32_t)tile_range<ROWS, TOKENS>(t, p.seq, base + lane).n : 0;
                uint32_t upto = n;
#pragma unroll 1
                for (int o = 1; o < 32; o <<= 1) {
                    const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, upto, o);
                    if (lane >= o) upto += y;
                }
                const uint32_t past = __ballot_sync(0xFFFFFFFFu, p.item + upto > w.x);
                const int at = past != 0 ? __ffs(past) - 1 : 31;
                p.item += __shfl_sync(0xFFFFFFFFu, past != 0 ? upto - n : upto, at);
                p.rt = base + at;
                if (past != 0 || base + 32 >= rts) break;
            }
        }
        p.range = tile_range<ROWS, TOKENS>(t, p.seq, p.rt);
        w.begun = 1;
        const uint32_t end = p.item + (uint32_t)p.range.n;
        if (w.whole) {
            const bool before = p.item < w.x;
            w.x = end;
            if (before) continue;  // the share before does it
            p.from = 0;
            p.count = p.range.n;
        } else {
            p.from = (int32_t)(w.x - p.item);
            p.count = (int32_t)(min(end, w.x1) - w.x);
            w.x += (uint32_t)p.count;
        }
        return true;
    }
    return false;
}

// What the joining kernel needs to know about the end of share c - 1 (the
// start of share c): whether an item is cut there for the first time, and
// which shares hold its parts: the last part of share c - 1, then the first
// part of shares c .. last.
struct Cut {
    int32_t b, kv_head, rt, last;  // last < 0: nothing to join here
    Sequence seq;
};
// Written by block c (one thread) for its first piece.
template <int ROWS, int TOKENS>
__device__ __forceinline__ Cut cut_of(const Piece& p, const Line& l, uint32_t c) {
    Cut u{p.b, p.kv_head, p.rt, -1, p.seq};
    if (c > 0 && p.item < share_start(l, c) && share_start(l, c - 1) <= p.item) {
        const uint32_t end = p.item + (uint32_t)p.range.n;
        uint32_t last = c;
        while (last + 1 < l.shares && share_start(l, last + 1) < end) ++last;
        u.last = (int32_t)last;
    }
    return u;
}

// Partial results in the workspace, after the header: C cuts, then two parts
// for each share, ROWS * (dim + 2) floats each: the accumulators, row by row
// (items of few rows) or column by column (256 rows, whose threads hold a row
// each and so write whole lines), then every row's reference (base 2), then
// every row's sum.
struct PartLayout {
    Cut* cuts;
    float* parts;
    int32_t rows, dim;
    __device__ __forceinline__ float* acc(uint32_t share, int which) const {
        return parts + ((size_t)share * 2 + which) * (size_t)rows * (dim + 2);
    }
    __device__ __forceinline__ float* stats(uint32_t share, int which) const {
        return acc(share, which) + (size_t)rows * dim;
    }
};
__device__ __forceinline__ PartLayout part_layout(const KvArgs& a, int shares, int rows) {
    uint8_t* p = reinterpret_cast<uint8_t*>(a.ws) + sizeof(WsHeader);
    return PartLayout{reinterpret_cast<Cut*>(p), reinterpret_cast<float*>(p + (size_t)shares * sizeof(Cut)), rows,
                      a.dim};
}
inline size_t part_bytes(int shares, int rows, int dim) {
    return (size_t)shares * (sizeof(Cut) + 2 * (size_t)rows * (size_t)(dim + 2) * sizeof(float));
}

// Rows of the piece's tile that exist.
template <int ROWS>
__device__ __forceinline__ int live_rows(const AttnArgs& t, const Piece& p) {
    return min(ROWS, (int)((uint32_t)p.seq.n * t.group.d) - p.rt * ROWS);
}
// Row `row` of an item's tile: its place in the packed tensors.
struct RowPlace {
    int64_t token;  // row of the packed tensors
    int32_t pos;    // position in the sequence
    int32_t head;   // query head
};
__device__ __forceinline__ RowPlace row_place(const AttnArgs& t, const Piece& p, int rows, int row) {
    const uint32_t r = (uint32_t)(p.rt * rows + row), i = div_by(t.group, r);
    return RowPlace{p.seq.row + i, p.seq.len - p.seq.n + (int32_t)i,
                    (int32_t)((uint32_t)p.kv_head * t.group.d + (r - i * t.group.d))};
}
// Values d .. d + 7 of a finished row: v / sum, and with d = 0 its log-sum-exp
// (m in base 2).  True when something is not finite, though the row sees keys:
// the row is then worked out by fix_row.
template <class T, class Args>
__device__ __forceinline__ bool store_row_part(const Args& t, const Piece& p, int rows, int row, int d,
                                               const float* v, float m, float sum) {
    const RowPlace at = row_place(t, p, rows, row);
    const bool none = sees_none(t, p.seq, at.token, at.pos, sum);
    const float inv = none ? 0.f : 1.f / sum;
    float y[8];
    bool odd = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        y[i] = none ? 0.f : v[i] * inv;
        odd |= !(fabsf(y[i]) <= 3.402823466e+38f);
    }
    const uint4 w = make_uint4(round_pair<T>(y[0], y[1]), round_pair<T>(y[2], y[3]), round_pair<T>(y[4], y[5]),
                               round_pair<T>(y[6], y[7]));
    *reinterpret_cast<uint4*>(t.out + at.token * t.o_token + (int64_t)at.head * t.o_head + 2 * d) = w;
    if (d == 0 && t.lse != nullptr)
        t.lse[at.token * t.q_heads + at.head] = none ? -INFINITY : (m + log2f(sum)) * 0.6931471805599453f;
    return odd;
}
// One warp: the row from the definition.
template <class T, int FMT, class Args>
__device__ __forceinline__ void fix_row(const KvArgs& a, const Args& t, const Piece& p, int rows, int row) {
    const RowPlace at = row_place(t, p, rows, row);
    attend_row<T, FMT>(a, t, p.b, p.seq, at.token, at.pos, at.head);
}

// What the joining kernels of share blockIdx.x begin with: the cut, and for the
// block's rows row0 .. row0 + JOIN - 1 the parts' weights and what they add up to.
template <int JOIN, int PARTS>
struct JoinShared {
    float weight[JOIN][PARTS + 1], sums[JOIN][PARTS + 1];
    float total[JOIN], top[JOIN];
    uint32_t odd_rows;
};
template <int ROWS, int JOIN, int PARTS>
__device__ __forceinline__ bool join_begin(const KvArgs& a, const AttnArgs& t, const PartLayout& parts,
                                           JoinShared<JOIN, PARTS>& sh, Piece& p, int& live, int& first, int& n) {
    const Cut cut = parts.cuts[blockIdx.x];
    if (cut.last < 0) return false;
    p.b = cut.b;
    p.kv_head = cut.kv_head;
    p.rt = cut.rt;
    p.seq = cut.seq;
    const int row0 = blockIdx.y * JOIN;
    live = live_rows<ROWS>(t, p) - row0;
    if (live <= 0) return false;
    first = (int)blockIdx.x - 1;
    n = cut.last - first + 1;
    if (threadIdx.x == 0) sh.odd_rows = 0;
    for (int i = threadIdx.x; i < n * JOIN; i += blockDim.x) {
        const int part = i / JOIN, r = i % JOIN;
        const float* st = parts.stats(first + part, part == 0);
        sh.weight[r][part] = r < live ? st[row0 + r] : -INFINITY;
        sh.sums[r][part] = r < live ? st[ROWS + row0 + r] : 0.f;
    }
    __syncthreads();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int r = warp; r < JOIN; r += blockDim.x >> 5) {
        float m = -INFINITY;
        for (int i = lane; i < n; i += 32) m = fmaxf(m, sh.weight[r][i]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        const float from = m == -INFINITY ? 0.f : m;
        float sum = 0.f;
        for (int i = lane; i < n; i += 32) {
            const float f = exp2f(sh.weight[r][i] - from);
            sum += f * sh.sums[r][i];
            sh.weight[r][i] = f;
        }
        sum = warp_sum(sum);
        if (lane == 0) {
            sh.total[r] = sum;
            sh.top[r] = m;
        }
    }
    __syncthreads();
    return true;
}
template <class T, int FMT, int ROWS, int JOIN, int PARTS, class Args>
__device__ __forceinline__ void join_end(const KvArgs& a, const Args& t, JoinShared<JOIN, PARTS>& sh,
                                         const Piece& p) {
    __syncthreads();
    for (uint32_t odd = sh.odd_rows; odd != 0; odd &= odd - 1) {
        const int r = __ffs(odd) - 1;
        if (r % (int)(blockDim.x >> 5) == (int)(threadIdx.x >> 5))
            fix_row<T, FMT>(a, t, p, ROWS, (int)blockIdx.y * JOIN + r);
    }
}

// Items of few rows, up to hundreds of parts: 4 rows a block, 4 warps a row,
// each taking every 4th part; a row's warps are added in their order.
constexpr int kMaxShares = 456;
constexpr int kJoinFew = 4, kJoinFewThreads = 512;
template <class T, int FMT, int ROWS, class Args>
__global__ void __launch_bounds__(kJoinFewThreads) join_rows_kernel(const __grid_constant__ KvArgs a,
                                                                    const __grid_constant__ Args t, int shares) {
    __shared__ JoinShared<kJoinFew, kMaxShares> sh;
    __shared__ float4 meet[4][kJoinFew][32];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const PartLayout parts = part_layout(a, shares, ROWS);
    Piece p;
    int live, first, n;
    if (!join_begin<ROWS>(a, t, parts, sh, p, live, first, n)) return;
    const int lane = threadIdx.x & 31, r = threadIdx.x >> 7, stride = (threadIdx.x >> 5) & 3;
    const int row = blockIdx.y * kJoinFew + r;
    const bool mine = r < live && 4 * lane < a.dim;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int i = stride; i < n; i += 4) {
        if (mine) {
            const float* src = parts.acc(first + i, i == 0) + (size_t)row * a.dim + 4 * lane;
            const float4 x = *reinterpret_cast<const float4*>(src);
            const float f = sh.weight[r][i];
            v.x += f * x.x;
            v.y += f * x.y;
            v.z += f * x.z;
            v.w += f * x.w;
        }
    }
    meet[stride][r][lane] = v;
    __syncthreads();
    if (stride == 0) {
#pragma unroll
        for (int i = 1; i < 4; ++i) {
            const float4 x = meet[i][r][lane];
            v.x += x.x;
            v.y += x.y;
            v.z += x.z;
            v.w += x.w;
        }
        // pairs of lanes hold 8 values together: the even one stores them
        const float y[8] = {v.x, v.y, v.z, v.w, __shfl_down_sync(0xFFFFFFFFu, v.x, 1),
                            __shfl_down_sync(0xFFFFFFFFu, v.y, 1), __shfl_down_sync(0xFFFFFFFFu, v.z, 1),
                            __shfl_down_sync(0xFFFFFFFFu, v.w, 1)};
        if (mine && (lane & 1) == 0 && store_row_part<T>(t, p, ROWS, row, 4 * lane, y, sh.top[r], sh.total[r]))
            atomicOr(&sh.odd_rows, 1u << r);
    }
    join_end<T, FMT, ROWS>(a, t, sh, p);
}

// Items of 256 rows, few parts: 32 rows a block, a row a lane, 16 columns a
// warp; the rows go out through shared memory.
constexpr int kJoinMany = 32, kJoinManyThreads = 256, kManyShares = 152;
template <class T, int FMT, int ROWS, class Args>
__global__ void __launch_bounds__(kJoinManyThreads) join_columns_kernel(const __grid_constant__ KvArgs a,
                                                                        const __grid_constant__ Args t,
                                                                        int shares) {
    __shared__ JoinShared<kJoinMany, kManyShares> sh;
    extern __shared__ float tile[];  // [32][dim + 1]
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const PartLayout parts = part_layout(a, shares, ROWS);
    Piece p;
    int live, first, n;
    if (!join_begin<ROWS>(a, t, parts, sh, p, live, first, n)) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int row0 = blockIdx.y * kJoinMany;
    if (16 * warp < a.dim) {
        float v[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) v[k] = 0.f;
        for (int i = 0; i < n; ++i) {
            const float f = sh.weight[lane][i];
            const float* src = parts.acc(first + i, i == 0) + (size_t)(16 * warp) * ROWS + row0 + lane;
            float x[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) x[k] = lane < live ? src[k * ROWS] : 0.f;
#pragma unroll
            for (int k = 0; k < 16; ++k) v[k] += f * x[k];
        }
#pragma unroll
        for (int k = 0; k < 16; ++k) tile[lane * (a.dim + 1) + 16 * warp + k] = v[k];
    }
    __syncthreads();
    const int groups = a.dim / 8;
    for (int k = threadIdx.x; k < min(live, kJoinMany) * groups; k += kJoinManyThreads) {
        const int r = k / groups, d = 8 * (k - r * groups);
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = tile[r * (a.dim + 1) + d + e];
        if (store_row_part<T>(t, p, ROWS, row0 + r, d, y, sh.top[r], sh.total[r])) atomicOr(&sh.odd_rows, 1u << r);
    }
    join_end<T, FMT, ROWS>(a, t, sh, p);
}

// Clusters of blocks.
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Shared memory of another of the cluster's blocks.
__device__ __forceinline__ uint32_t in_block(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ float4 load_cluster4(uint32_t a) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(a)
                 : "memory");
    return v;
}
__device__ __forceinline__ float load_cluster(uint32_t a) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
    return v;
}
template <class... Params, class... Args>
cudaError_t launch_clusters(void (*kernel)(Params...), int blocks, int cluster, int threads, size_t shared,
                            cudaStream_t s, Args... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = shared;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)cluster;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Shares that a call can need, at most `most`: the tiles of a batch whose
// sequences keep to the program's expectations.
inline int shares_for(const KvArgs& a, const AttnArgs& t, int max_new, int max_len, int rows, int tokens, int most) {
    const double row_tiles = ((double)max_new * t.group.d + rows - 1) / rows;
    const double tiles = ((double)max_len + 2 * tokens - 1) / tokens;
    const double all = (double)a.batch * a.kv_heads * row_tiles * tiles;
    return all < most ? (int)all : most;
}

// Launched so that its blocks may start while the kernel before it still runs;
// they wait for its end before they read.
template <class Args>
cudaError_t launch_join(void (*kernel)(KvArgs, Args, int), const KvArgs& a, const Args& t, int shares, int blocks_y,
                        int threads, size_t shared, cudaStream_t s) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)shares, (unsigned)blocks_y);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = shared;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a, t, shares);
}

}  // namespace cccl
