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
// joins, in the order of the line, so that results do not vary.
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
// (A call's rows are below 2^31: n_tokens * q_heads is.)
template <int ROWS, int TOKENS>
__device__ __forceinline__ TileRange tile_range(const AttnArgs& t, const Sequence& s, int32_t rt) {
    const uint32_t rows = (uint32_t)s.n * t.group.d, r0 = (uint32_t)rt * ROWS;
    const int32_t base = s.len - s.n;
    TileRange r;
    int32_t ignore;
    visible_range(t, s.len, base + (int32_t)div_by(t.group, r0), r.first, ignore);
    visible_range(t, s.len, base + (int32_t)div_by(t.group, min(r0 + ROWS, rows) - 1), ignore, r.last);
    if (r.first >= r.last) {
        r.first = r.last = r.lo = 0;
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
template <int ROWS, int TOKENS>
__device__ __forceinline__ void build_prefix(const KvArgs& a, const AttnArgs& t, uint32_t* prefix) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    for (int b = warp; b < a.batch; b += warps) {
        const Sequence s = load_sequence(a, b);
        const int32_t rts = row_tiles<ROWS>(t, s);
        uint64_t sum = 0;
        for (int32_t rt = lane; rt < rts; rt += 32) sum += (uint64_t)tile_range<ROWS, TOKENS>(t, s, rt).n;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
        if (lane == 0) prefix[b + 1] = (uint32_t)min(sum * (uint32_t)a.kv_heads, (uint64_t)0xFFFFFFFFu);
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
        if (carry >= 0xFFFFFFFFu) {
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

// The item that holds place x of the line (a whole warp, all lanes alike).
template <int ROWS, int TOKENS>
__device__ __forceinline__ void find_item(const KvArgs& a, const AttnArgs& t, const uint32_t* prefix, uint32_t x,
                                          Piece& p) {
    const int lane = threadIdx.x & 31;
    int lo = 0, hi = a.batch;  // prefix[lo] <= x < prefix[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (prefix[mid] <= x)
            lo = mid;
        else
            hi = mid;
    }
    p.b = lo;
    p.seq = load_sequence(a, lo);
    const uint32_t per_head = (prefix[lo + 1] - prefix[lo]) / (uint32_t)a.kv_heads;
    p.kv_head = (int32_t)((x - prefix[lo]) / per_head);
    const uint32_t start = prefix[lo] + (uint32_t)p.kv_head * per_head;
    // the first row tile whose tiles reach past x: 32 row tiles at a time
    uint32_t before = 0;
    p.rt = 0;
    const int32_t rts = row_tiles<ROWS>(t, p.seq);
    for (int32_t base = 0; base < rts; base += 32) {
        const int32_t rt = base + lane;
        const uint32_t n = rt < rts ? (uint32_t)tile_range<ROWS, TOKENS>(t, p.seq, rt).n : 0;
        uint32_t upto = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, upto, o);
            if (lane >= o) upto += y;
        }
        const uint32_t past = __ballot_sync(0xFFFFFFFFu, start + before + upto > x);
        if (past != 0) {
            const int at = __ffs(past) - 1;
            p.rt = base + at;
            before += __shfl_sync(0xFFFFFFFFu, upto - n, at);
            break;
        }
        before += __shfl_sync(0xFFFFFFFFu, upto, 31);
    }
    p.range = tile_range<ROWS, TOKENS>(t, p.seq, p.rt);
    p.item = start + before;
}
// The item after p's on the line (there is one).
template <int ROWS, int TOKENS>
__device__ __forceinline__ void next_item(const KvArgs& a, const AttnArgs& t, Piece& p) {
    p.item += (uint32_t)p.range.n;
    if (++p.rt >= row_tiles<ROWS>(t, p.seq)) {
        p.rt = 0;
        if (++p.kv_head >= a.kv_heads) {
            p.kv_head = 0;
            do {
                p.seq = load_sequence(a, ++p.b);
            } while (p.seq.n == 0);
        }
    }
    p.range = tile_range<ROWS, TOKENS>(t, p.seq, p.rt);
}

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
__device__ __forceinline__ Walk make_walk(uint32_t T, uint32_t share, uint32_t blocks, uint32_t min_tiles, int whole) {
    Walk w;
    w.share = share;
    // no more shares than give each min_tiles tiles
    w.line.shares = min(blocks, max((T - 1) / min_tiles + 1, 1u));
    if (T == 0) w.line.shares = 1;
    w.line.each = T / w.line.shares;
    w.line.rest = T - w.line.each * w.line.shares;
    w.x = share < w.line.shares ? share_start(w.line, share) : T;
    w.x1 = share < w.line.shares ? share_start(w.line, share + 1) : T;
    w.whole = whole;
    w.begun = 0;
    return w;
}
template <int ROWS, int TOKENS>
__device__ __forceinline__ bool next_piece(const KvArgs& a, const AttnArgs& t, const uint32_t* prefix, Walk& w,
                                           Piece& p) {
    while (w.x < w.x1) {
        if (w.begun == 0)
            find_item<ROWS, TOKENS>(a, t, prefix, w.x, p);
        else
            next_item<ROWS, TOKENS>(a, t, p);
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
// for each share, ROWS * (dim + 2) floats each: per row the accumulator, then
// the maximum (base 2) and the sum of every row.
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
template <class T>
__device__ __forceinline__ bool store_row_part(const AttnArgs& t, const Piece& p, int rows, int row, int d,
                                               const float* v, float m, float sum) {
    const RowPlace at = row_place(t, p, rows, row);
    int32_t first, last;
    visible_range(t, p.seq.len, at.pos, first, last);
    const bool none = last <= first;
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
template <class T, int FMT>
__device__ __forceinline__ void fix_row(const KvArgs& a, const AttnArgs& t, const Piece& p, int rows, int row) {
    const RowPlace at = row_place(t, p, rows, row);
    attend_row<T, FMT>(a, t, p.b, p.seq.len, at.token, at.pos, at.head);
}

// Joins the parts of the item cut at the start of share blockIdx.x.  A block has
// GROUPS groups of STRIDES warps; a group joins EACH rows at a time, its warps
// taking every STRIDES-th part (items of few rows can have hundreds of parts,
// items of many have few), and adds its warps' sums in their order.
constexpr int kMaxShares = 456;
template <int GROUPS_, int STRIDES_, int EACH_, int PARTS_>
struct JoinShape {
    static constexpr int GROUPS = GROUPS_, STRIDES = STRIDES_, EACH = EACH_, PARTS = PARTS_;
    static constexpr int kRows = GROUPS * EACH, kThreads = 32 * GROUPS * STRIDES;
};
template <class T, int FMT, int ROWS, class J>
__global__ void __launch_bounds__(J::kThreads) join_parts_kernel(const __grid_constant__ KvArgs a,
                                                                 const __grid_constant__ AttnArgs t, int shares) {
    __shared__ float weight[J::kRows][J::PARTS + 1], sums[J::kRows][J::PARTS + 1];
    __shared__ float total[J::kRows], top[J::kRows];
    __shared__ float4 meet[J::STRIDES > 1 ? J::STRIDES : 1][J::STRIDES > 1 ? J::kRows : 1][32];
    __shared__ uint32_t odd_rows;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const PartLayout parts = part_layout(a, shares, ROWS);
    const Cut cut = parts.cuts[blockIdx.x];
    if (cut.last < 0) return;
    Piece p;
    p.b = cut.b;
    p.kv_head = cut.kv_head;
    p.rt = cut.rt;
    p.seq = cut.seq;
    const int row0 = blockIdx.y * J::kRows, live = live_rows<ROWS>(t, p) - row0;
    if (live <= 0) return;
    const int first = (int)blockIdx.x - 1, n = cut.last - first + 1;
    if (threadIdx.x == 0) odd_rows = 0;
    for (int i = threadIdx.x; i < n * J::kRows; i += J::kThreads) {
        const int part = i / J::kRows, r = i % J::kRows;
        if (r < live) {
            const float* st = parts.stats(first + part, part == 0);
            weight[r][part] = st[row0 + r];
            sums[r][part] = st[ROWS + row0 + r];
        }
    }
    __syncthreads();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int r = warp; r < min(J::kRows, live); r += J::kThreads / 32) {
        float m = -INFINITY;
        for (int i = lane; i < n; i += 32) m = fmaxf(m, weight[r][i]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        const float from = m == -INFINITY ? 0.f : m;
        float sum = 0.f;
        for (int i = lane; i < n; i += 32) {
            const float f = exp2f(weight[r][i] - from);
            sum += f * sums[r][i];
            weight[r][i] = f;
        }
        sum = warp_sum(sum);
        if (lane == 0) {
            total[r] = sum;
            top[r] = m;
        }
    }
    __syncthreads();
    const int group = warp / J::STRIDES, stride = warp % J::STRIDES;
    const int r0 = group * J::EACH;
    float4 v[J::EACH];
#pragma unroll
    for (int k = 0; k < J::EACH; ++k) v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    const bool inside = 4 * lane < a.dim;
#pragma unroll 4
    for (int i = stride; i < n; i += J::STRIDES) {
        const float* src = parts.acc(first + i, i == 0) + (size_t)(row0 + r0) * a.dim + 4 * lane;
#pragma unroll
        for (int k = 0; k < J::EACH; ++k) {
            if (r0 + k < live && inside) {
                const float4 x = *reinterpret_cast<const float4*>(src + (size_t)k * a.dim);
                const float f = weight[r0 + k][i];
                v[k].x += f * x.x;
                v[k].y += f * x.y;
                v[k].z += f * x.z;
                v[k].w += f * x.w;
            }
        }
    }
    if (J::STRIDES > 1) {
#pragma unroll
        for (int k = 0; k < J::EACH; ++k) meet[stride][r0 + k][lane] = v[k];
        __syncthreads();
        if (stride == 0) {
#pragma unroll
            for (int k = 0; k < J::EACH; ++k)
#pragma unroll
                for (int i = 1; i < J::STRIDES; ++i) {
                    const float4 x = meet[i][r0 + k][lane];
                    v[k].x += x.x;
                    v[k].y += x.y;
                    v[k].z += x.z;
                    v[k].w += x.w;
                }
        }
    }
    if (stride == 0) {
#pragma unroll
        for (int k = 0; k < J::EACH; ++k) {
            // pairs of lanes hold 8 values together: the even one stores them
            const float y[8] = {v[k].x, v[k].y, v[k].z, v[k].w, __shfl_down_sync(0xFFFFFFFFu, v[k].x, 1),
                                __shfl_down_sync(0xFFFFFFFFu, v[k].y, 1), __shfl_down_sync(0xFFFFFFFFu, v[k].z, 1),
                                __shfl_down_sync(0xFFFFFFFFu, v[k].w, 1)};
            const int r = r0 + k;
            if (r < live && inside && (lane & 1) == 0 &&
                store_row_part<T>(t, p, ROWS, row0 + r, 4 * lane, y, top[r], total[r]))
                atomicOr(&odd_rows, 1u << r);
        }
    }
    __syncthreads();
    for (uint32_t odd = odd_rows; odd != 0; odd &= odd - 1) {
        const int r = __ffs(odd) - 1;
        if (r % (J::kThreads / 32) == warp) fix_row<T, FMT>(a, t, p, ROWS, row0 + r);
    }
}

// Launched so that its blocks may start while the kernel before it still runs;
// they wait for its end before they read.
template <class T, int FMT, int ROWS, class J>
cudaError_t launch_join(const KvArgs& a, const AttnArgs& t, int shares, cudaStream_t s) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)shares, ROWS / J::kRows);
    cfg.blockDim = dim3(J::kThreads);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, join_parts_kernel<T, FMT, ROWS, J>, a, t, shares);
}

}  // namespace cccl
