// cccl_kv_chunk.cuh -- attention of many rows a kv head (chunks of prompts) on
// the 5th-generation tensor cores.
//
// An item is 256 rows (new tokens x the query heads that share a kv head), two
// tiles of 128; it walks its cached tokens 128 at a time.  Per tile of tokens
// and tile of rows: S = Q K^T (tcgen05, both operands in shared memory, S in
// TMEM), the softmax's step by a warpgroup that holds one row a thread, P back
// to TMEM over S, O += P V (A from TMEM, V in shared memory).  While one tile
// of rows is in its softmax the tensor core works on the other.
//
// Warps: 0-3 and 4-7 softmax of row tiles 0 and 1 (they also bring in their
// rows of Q and write the result); 8-11 bring K and V in, or widen 8-bit codes
// that 13 and 15 bring in; 12 issues the products; 14 walks along the block's
// share of the line and hands the pieces to the others.  One block an SM: it
// needs all 512 columns of TMEM (S0, S1, O0, O1).  Where there are few items a
// cluster's blocks share each and join their parts through shared memory.
//
// With ref_i a row's reference, x_ij = s_ij scale log2(e) and p_ij =
// 2^(x_ij - ref_i), a row's result is sum_j p_ij v_j / sum_j p_ij for any ref_i.
// So the reference is only moved when a score exceeds it by more than some slack
// (the accumulator is then rescaled in TMEM): binary32 sums and 16-bit
// probabilities hold that factor (kSlack, kLower).  The products of one thread execute
// in order, so a full S also means that the previous O is done, and S may be
// written over the P that the product before it reads.
//
// What bounds it, 16-bit caches: a row's 128 scores a tile cost its thread the
// loads from TMEM, a maximum, the exponentials (4 clocks a warp each on an SMSP),
// the sum, the rounding and the stores, about as long as the tensor core takes
// for the other tile of rows; under the power limit the clock is what gives.
// 4096 new tokens at the end of 32768 cached, 32 heads over 8 kv heads of 128:
// 1302 to 1339 us from a graph of a few calls, 1540 to 1580 TFLOP/s with the clock,
// 1443 us in a loop, where the power limit holds it at 1430 (a library product:
// 1931 and 1740); tensor pipe 59 % busy in a short call (1024 over 8192: 100 us).
// Half a row a thread, 16 softmax warps: 1590 us against 1389.  Exponentials
// taken a block of 16 late: the same.
// 8-bit caches, 5 x 2048 new tokens with windows of 4096: 702 to 712 us, 710 to
// 720 TFLOP/s; the long chunk over E4M3 1896 to 1909 us, 1085.  Where it goes, by
// leaving parts out, of 717: widening 86, the scales' loads and products, a
// column's for each of a row's scores, 92, and the tiles at a range's ends, with
// one slot less for tiles, 130.  Rows held in the products' own layout, which
// loads a quarter of the scales: 797.
// Moving a reference rescales the accumulator, 32 columns at a time in a loop that
// is not unrolled: 16 columns, unrolled, took 763 us for 710 (INT8, above) and 1329
// for 1315 (the long chunk), not unrolled 718 and 1344.
#pragma once

#include <cuda.h>

#include <type_traits>

#include "cccl_kv.cuh"
#include "cccl_kv_launch.h"
#include "cccl_kv_schedule.cuh"
#include "cccl_launch.h"

namespace cccl {

namespace {

constexpr int kRows = 256, kTileRows = 128, kTokens = 128;
constexpr int kThreads = 512;
constexpr int kShares = 152;
static_assert(kShares <= kManyShares, "the joining kernel has room for every share's part");
constexpr int kMostScaleSlots = 4;
// Tiles of tokens whose scales are kept: with rows in two tiles, and where the
// tiles of tokens are shared (narrow, below).
template <class Args>
constexpr int kScaleSlots = std::is_same<Args, TreeArgs>::value ? 4 : 3;
constexpr int kLoaderWarps = 4;
// K and V tiles in shared memory, as 16-bit values; tiles of 8-bit codes on
// their way there
constexpr int kMostSlots = 4, kRawSlots = 3;
template <int FMT>
constexpr int kSlots = FMT == kKv16Bit ? 4 : 3;
// How far (base 2) a row's reference lies below its maximum when it is set, and
// how far the maximum may then rise before it is set again.  fp16 holds 2^-24 to
// 2^16: with 9 and 6 (and 0.09 for scale_log2) a probability is off by 2^-34 of the
// largest at most, apart from its rounding to 11 bits; kSpread may take 4 bits.
// Setting it again costs, a lower reference saves bits: with 7 and 8 5 x 2048
// windowed INT8 chunks took 707 us for 710, 4096 E4M3 tokens over 32768 1893 for
// 1908, 2048 fp16 tokens over 16384 357 for 364.  bf16 has binary32's range.
// Operand M:
template <class M>
constexpr float kSlack = M::kHalf ? 6.f : 8.f;
template <class M>
constexpr float kLower = M::kHalf ? 9.f : 0.f;
// 8-bit caches: where the value scales of 32 rows, and the largest of the tile's
// four such groups, lie within a factor of 4 (a difference of scale_bits; zeros
// do not count), the largest stands for all in a row's reference, which then lies
// up to 4 too high; else it is looked for score by score (2048 new tokens over
// 16384: 526 us alike, 535 apart).  That way for every tile whose reference moves:
// 999 us for 703 (5 x 2048 windowed INT8 chunks).
constexpr uint32_t kSpread = 2u << 23;
// Halves of result rows (128 bytes) that a softmax warp has on their way out at
// a time
template <int FMT, class Args>
constexpr int kStageRows = FMT == kKv16Bit ? 16 : (std::is_same<Args, TreeArgs>::value ? 4 : 8);
template <int FMT, class Args>
constexpr int kStageBytes = 8 * 128 * kStageRows<FMT, Args>;

// Registers of a thread: the launch's 4 x 128 a warpgroup, divided anew (two
// softmax warpgroups, two of the others).
constexpr int kSoftmaxRegs = 192, kLoaderRegs = 64;

// TMEM columns
constexpr uint32_t kColS = 0, kColO = 256;  // S of row tile i at 128 i (P over it), O at 256 + 128 i

constexpr int kRing = 4;  // pieces handed on and not yet taken by all

struct Shared {
    uint64_t q_full[2], s_full[2], p_full[2], o_full[2];
    uint64_t kv_full[kMostSlots], kv_free[kMostSlots], scale_full[kMostScaleSlots];
    uint64_t raw_full[kRawSlots], raw_free[kRawSlots];
    uint64_t drained;
    uint64_t half_full[2], half_read[2];  // narrow items: a warpgroup's statistics are there, it has read both accumulators
    uint32_t tmem;
    uint32_t stop;  // a bounded wait ran out: every role leaves
    uint32_t odd;   // a row that the block wrote came out non-finite
    uint32_t prefix[kMaxBatch + 1];
    // One warp walks along the line and hands the pieces on; every other warp
    // takes a copy (softmax warps keep two, this piece and the next, here rather
    // than in registers, which hold a row of S).
    Piece ring[kRing], piece[8][2];
    uint64_t piece_full[kRing], piece_free[kRing];
    alignas(16) float k_scale[kMostScaleSlots][kTokens];
    alignas(16) float v_scale[kMostScaleSlots][kTokens];
    // the largest value scale of each warp's rows (scale_bits), its lowest bit
    // instead saying whether others of them lie far below
    alignas(16) uint32_t v_top[kMostScaleSlots][kLoaderWarps];
};

// Narrow items, behind Shared: the reference and the sum of each warpgroup's rows.
struct Halves {
    float m[2][kTileRows], l[2][kTileRows];
};
template <class Args>
constexpr size_t kHalvesBytes = std::is_same<Args, TreeArgs>::value ? sizeof(Halves) : 0;
__device__ __forceinline__ Halves& halves_of(Shared* sh) { return *reinterpret_cast<Halves*>(sh + 1); }

// ---------------------------------------------------------------- tcgen05
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
                 : "memory");
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{ .reg .pred p; setp.ne.u32 p, %4, 0; tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p; }" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{ .reg .pred p; setp.ne.u32 p, %4, 0; tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p; }" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
        : "memory");
}
#define CCCL_R4(r, i) "=r"(r[i]), "=r"(r[i + 1]), "=r"(r[i + 2]), "=r"(r[i + 3])
#define CCCL_W4(r, i) "r"(r[i]), "r"(r[i + 1]), "r"(r[i + 2]), "r"(r[i + 3])
__device__ __forceinline__ void tc_load32(uint32_t at, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
        "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : CCCL_R4(r, 0), CCCL_R4(r, 4), CCCL_R4(r, 8), CCCL_R4(r, 12), CCCL_R4(r, 16), CCCL_R4(r, 20), CCCL_R4(r, 24),
          CCCL_R4(r, 28)
        : "r"(at));
}
__device__ __forceinline__ void tc_load16(uint32_t at, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : CCCL_R4(r, 0), CCCL_R4(r, 4), CCCL_R4(r, 8), CCCL_R4(r, 12)
        : "r"(at));
}
__device__ __forceinline__ void tc_load8(uint32_t at, uint32_t* r) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : CCCL_R4(r, 0), CCCL_R4(r, 4)
                 : "r"(at));
}
__device__ __forceinline__ void tc_store32(uint32_t at, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,"
        "%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::CCCL_W4(r, 0),
        CCCL_W4(r, 4), CCCL_W4(r, 8), CCCL_W4(r, 12), CCCL_W4(r, 16), CCCL_W4(r, 20), CCCL_W4(r, 24), CCCL_W4(r, 28),
        "r"(at)
        : "memory");
}
#undef CCCL_R4
#undef CCCL_W4
__device__ __forceinline__ void tc_wait_load() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_store() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Shared-memory operands: rows of 64 values (128 bytes, 128-byte swizzle), a
// half of up to 64 channels each, 128 rows (16 KB) a half.
//   Q and K, K-major: 8-row groups 1024 bytes apart; 16 channels are 32 bytes.
//   V, MN-major (channels along a row): 8-token groups 1024 bytes apart, the
//   second 64 channels one half further; 16 tokens are 2048 bytes.
constexpr uint32_t kHalfBytes = kTileRows * 128;
__device__ __forceinline__ uint64_t operand(uint32_t addr, uint32_t leading) {
    return (uint64_t)((addr & 0x3FFFF) >> 4) | ((uint64_t)(leading >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
           (1ull << 46) | (2ull << 61);
}
// kind::f16: binary32 accumulator, M = 128, both operands of one type (bit 13
// would change A's sign).
__device__ __forceinline__ uint32_t instruction(bool half, int n, bool b_mn_major) {
    const uint32_t type = half ? 0u : 1u;
    return (1u << 4) | (type << 7) | (type << 10) | ((b_mn_major ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) |
           ((uint32_t)(kTileRows >> 4) << 24);
}
__device__ __forceinline__ uint32_t swizzled(uint32_t row, uint32_t chunk) {  // 16-byte chunk of a row
    return (chunk >> 3) * kHalfBytes + row * 128 + (((chunk & 7) ^ (row & 7)) << 4);
}

// ---------------------------------------------------------------- f32 pairs
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(reinterpret_cast<uint64_t&>(d))
        : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)), "l"(reinterpret_cast<uint64_t&>(c)));
    return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("mul.rn.f32x2 %0, %1, %2;"
        : "=l"(reinterpret_cast<uint64_t&>(d))
        : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("add.rn.f32x2 %0, %1, %2;"
        : "=l"(reinterpret_cast<uint64_t&>(d))
        : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
    return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
template <class T>
__device__ __forceinline__ uint32_t pack(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack<BfType>(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}
template <>
__device__ __forceinline__ uint32_t pack<HfType>(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}

// The products' operands: 8-bit codes are multiplied in fp16.
template <class T, int FMT>
using Operand = typename std::conditional<FMT == kKv16Bit, T, HfType>::type;

// A bounded wait of one role; false: leave (this wait or another's ran out).
// Most waits are over at the first look; the others' code is kept in one place.
__device__ __forceinline__ bool wait_long(Shared* sh, WsHeader* ws, uint64_t* bar, uint32_t parity) {
    if (mbar_wait(bar, parity)) return true;
    record_error(ws, kStatusTimeout);
    *reinterpret_cast<volatile uint32_t*>(&sh->stop) = 1;
    return false;
}
// A whole warp waits.
struct Waiter {
    Shared* sh;
    WsHeader* ws;
    __device__ __forceinline__ bool operator()(uint64_t* bar, uint32_t parity) const {
        if (__all_sync(0xFFFFFFFFu, mbar_test(bar, parity))) return true;
        return __all_sync(0xFFFFFFFFu, wait_long(sh, ws, bar, parity)) != 0;
    }
};

// The walking warp: pieces to the ring, one without tiles at the end; and, for
// the joining kernel, whether an item is cut at this share's start (said before
// anything is waited for: that kernel runs even if this one gives up).
template <class Args>
__device__ __forceinline__ void walk_role(const KvArgs& a, const Args& t, Shared* sh, Walk w) {
    const Waiter wait{sh, a.ws};
    const int lane = threadIdx.x & 31;
    Piece p{};
    for (uint32_t n = 0;; ++n) {
        const uint32_t s = n % kRing, use = n / kRing;
        const bool more = next_piece<kRows, kTokens>(a, t, sh->prefix, w, p);
        if (use > 0 && !wait(&sh->piece_free[s], (use - 1) & 1)) return;
        if (lane == 0) {
            sh->ring[s] = p;
            if (!more) sh->ring[s].count = 0;
            mbar_arrive(&sh->piece_full[s]);
        }
        if (n == 0 && !w.whole) {
            Cut cut{0, 0, 0, -1, {}};
            if (more) cut = cut_of<kRows, kTokens>(p, w.line, w.share);
            if (lane == 0) part_layout(a, gridDim.x, kRows).cuts[w.share] = cut;
        }
        if (!more) return;
    }
}
// The walking warp where `cluster` blocks share an item: one piece, this block's
// part of item blockIdx.x / cluster (count 0: none; items of fewer tiles than
// blocks leave some without).  prefix counts items.
__device__ __forceinline__ int parts_of(const Piece& p, int cluster) { return min(cluster, p.range.n); }
template <class Args>
__device__ __forceinline__ void share_role(const KvArgs& a, const Args& t, Shared* sh, int cluster) {
    const uint32_t items = sh->prefix[a.batch];
    Walk w = make_walk(items, blockIdx.x / cluster, items, 1);
    Piece p{};
    if (next_piece<kRows, 0>(a, t, sh->prefix, w, p)) p.range = tile_range<kRows, kTokens>(t, p.seq, p.rt);
    const int rank = (int)cluster_rank(), n = parts_of(p, cluster);
    p.from = p.count = 0;
    if (rank < n) {
        p.from = (int32_t)((int64_t)rank * p.range.n / n);
        p.count = (int32_t)((int64_t)(rank + 1) * p.range.n / n) - p.from;
    }
    if ((threadIdx.x & 31) == 0) {
        sh->ring[0] = p;
        mbar_arrive(&sh->piece_full[0]);
        if (p.count > 0) {
            sh->ring[1].count = 0;
            mbar_arrive(&sh->piece_full[1]);
        }
    }
}
// The other warps: piece n.  Its count is 0 after the last one; false: leave.
__device__ __forceinline__ bool take_piece(const Waiter& wait, uint32_t n, Piece* to) {
    Shared* sh = wait.sh;
    const uint32_t s = n % kRing;
    if (!wait(&sh->piece_full[s], (n / kRing) & 1)) return false;
    *to = sh->ring[s];
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&sh->piece_free[s]);
    return true;
}

// ---------------------------------------------------------------- K and V
// Tiles come through a ring, K and V in turn.  A tile that every row of the
// item's range covers is brought by TMA, a page (or 128 tokens) a box, each warp
// issuing the boxes that begin in its rows; one that the range cuts, or pages
// that TMA's boxes do not fit (`box` is 0), by 16-byte copies that put zeros where
// the range ends, so that no product meets what nobody wrote.
struct Fetch {
    const CUtensorMap *k, *v;
    int32_t box;  // tokens of a TMA box; 0: none
};
struct TileRow {
    int64_t at;
    bool real;
};
// Positions pos + 32 i of a lane: the page entries are asked for together.
template <int N>
__device__ __forceinline__ void tile_rows(const KvArgs& a, const Piece& p, int32_t pos, TileRow* r) {
    int32_t page[N];
    uint32_t slot[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        // inside the visible range, so inside the table
        const int32_t at = pos + 32 * i;
        r[i].real = at >= p.range.first && at < p.range.last;
        const uint32_t pi = div_by(a.page_tokens, r[i].real ? (uint32_t)at : 0u);
        slot[i] = (uint32_t)at - pi * a.page_tokens.d;
        page[i] = a.table[(int64_t)p.b * a.table_stride + pi];
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
        if (r[i].real && (page[i] < 0 || page[i] >= a.pages)) {
            record_error(a.ws, kStatusInvalidArg);
            r[i].real = false;
        }
        r[i].at = r[i].real ? page[i] * a.page_stride + (int64_t)slot[i] * a.token_stride +
                                  (int64_t)p.kv_head * a.head_stride
                            : 0;
    }
}
__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap* map, int32_t d, int32_t slot, int32_t head,
                                        int32_t page, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
        "[%6];" ::"r"(dst),
        "l"(map), "r"(d), "r"(slot), "r"(head), "r"(page), "r"(smem_addr(bar))
        : "memory");
}
__device__ __forceinline__ void arrive_expect(uint64_t* bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_addr(bar)), "r"(bytes) : "memory");
}

// The role of WARPS warps (this one is `warp`): every tile of the share's
// pieces to slots of slot_bytes from `slots` on; full[s] is arrived at by each
// of the warps.
template <int FMT, int WARPS, int SLOTS>
__device__ __forceinline__ void fetch_role(const KvArgs& a, const AttnArgs& t, Shared* sh, const Fetch& f, int warp,
                                           uint32_t slots, uint32_t slot_bytes, uint64_t* full, uint64_t* free_) {
    constexpr bool kWide = FMT == kKv16Bit;      // 16-bit values in the swizzled layout; else codes, row after row
    constexpr int kParts = 4 / WARPS;            // groups of 32 rows of this warp
    const int lane = threadIdx.x & 31;
    const Waiter wait{sh, a.ws};
    const int chunks = a.dim * (kWide ? 2 : 1) / 16, per_row = chunks > 8 ? 16 : 8, chunk = lane % per_row;
    // this warp's boxes: one for each lane below `issue`
    const int halves = kWide ? (a.dim > 64 ? 2 : 1) : 1, span = kTokens / WARPS;
    const int boxes = f.box == 0 || (warp * span) % f.box != 0 ? 0 : (f.box >= span ? 1 : span / f.box);
    const int issue = boxes * halves, half = boxes > 0 ? lane / boxes : 0;
    const int first_row = warp * span + (boxes > 0 ? lane % boxes : 0) * f.box;
    const uint32_t expect = (uint32_t)boxes * (uint32_t)f.box * (slot_bytes / kTokens);
    uint32_t entry = 0, handed = 0;
    auto hand_over = [&](uint32_t upto) {  // this warp's copies of entries below `upto` are done
        if (handed >= upto) return;
        if (kWide) fence_proxy_async_smem();
        __syncwarp();
        for (; handed < upto; ++handed)
            if (lane == 0) mbar_arrive(&full[handed % SLOTS]);
    };
    Piece p;
    for (uint32_t n = 0; take_piece(wait, n, &p) && p.count > 0; ++n) {
        const int32_t base = (p.range.lo + p.from) * kTokens;
        for (int32_t j = 0; j < p.count; ++j) {
            const int32_t at = base + j * kTokens;
            const bool tma = f.box > 0 && at >= p.range.first && at + kTokens <= p.range.last;
            TileRow rows[kParts];
            int32_t page = 0, slot0 = 0;
            if (tma) {
                if (lane < issue) {
                    const uint32_t pos = (uint32_t)(at + first_row), pi = div_by(a.page_tokens, pos);
                    slot0 = (int32_t)(pos - pi * a.page_tokens.d);
                    page = (int32_t)page_of(a, p.b, pi);  // -1: outside the map, zeros
                }
            } else {
                tile_rows<kParts>(a, p, at + 32 * warp * kParts + lane, rows);
            }
#pragma unroll 1
            for (int side = 0; side < 2; ++side, ++entry) {
                const uint32_t s = entry % SLOTS, use = entry / SLOTS;
                const uint32_t dst = slots + s * slot_bytes;
                if (use > 0 && !__all_sync(0xFFFFFFFFu, mbar_test(&free_[s], (use - 1) & 1))) {
                    // about to wait: hand over what has been brought so far
                    copy_wait<0>();
                    hand_over(entry);
                    if (!wait(&free_[s], (use - 1) & 1)) goto leave;
                }
                if (tma) {
                    copy_wait<0>();
                    hand_over(entry);
                    ++handed;
                    if (lane == 0) arrive_expect(&full[s], expect);
                    __syncwarp();
                    if (lane < issue)
                        tma_box(dst + (kWide ? half * kHalfBytes + first_row * 128 : first_row * a.dim),
                                side ? f.v : f.k, 64 * half, slot0, p.kv_head, page, &full[s]);
                    continue;
                }
                const uint8_t* data = side ? a.v : a.k;
#pragma unroll
                for (int part = 0; part < kParts; ++part)
#pragma unroll 4
                    for (int i = 0; i < per_row; ++i) {  // 32 / per_row rows a pass
                        const int local = i * (32 / per_row) + lane / per_row;
                        const int64_t from = __shfl_sync(0xFFFFFFFFu, rows[part].at, local);
                        const bool real = __shfl_sync(0xFFFFFFFFu, (int)rows[part].real, local) != 0;
                        const int row = 32 * (warp * kParts + part) + local;
                        const uint32_t to = dst + (kWide ? swizzled(row, chunk) : (uint32_t)(row * a.dim + 16 * chunk));
                        if (chunk < chunks) copy16(to, data + (real ? from + 16 * chunk : 0), real);
                    }
                copy_commit();
                copy_wait<1>();
                hand_over(entry);
            }
        }
    }
leave:
    // early or not: no copy of this warp may still be in flight when the block ends
    copy_wait<0>();
    hand_over(entry);
    if (f.box > 0)
        for (uint32_t k = entry > SLOTS ? entry - SLOTS : 0; k < entry; ++k)
            if (!mbar_wait(&full[k % SLOTS], (k / SLOTS) & 1, kDrainLimitNs)) break;
}

// 8-bit caches: codes to fp16, four warps of 32 rows each.  A lane takes 16
// codes of a row at a time; lanes of a row's second half store their two
// chunks the other way round, so that a row's eight lanes meet all banks.
template <int FMT>
__device__ __forceinline__ void widen_rows(uint32_t from, uint32_t to, int dim, int warp, int lane) {
    const int chunks = dim / 16, per_row = chunks > 4 ? 8 : 4, chunk = lane % per_row;
    if (chunk >= chunks) return;
#pragma unroll 4
    for (int i = 0; i < per_row; ++i) {  // 32 / per_row rows a pass
        const uint32_t row = 32 * warp + i * (32 / per_row) + lane / per_row;
        uint4 x;
        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
                     : "r"(from + row * dim + 16 * chunk));
        const uint32_t c[4] = {x.x, x.y, x.z, x.w};
        uint32_t v[8];
#pragma unroll
        for (int k = 0; k < 4; ++k) expand4_in_order<FMT>(c[k], v[2 * k], v[2 * k + 1]);
        const int second = chunk >> 2;  // which of the two goes first
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int part = k ^ second;
            asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(to + swizzled(row, 2 * chunk + part)),
                         "r"(part ? v[4] : v[0]), "r"(part ? v[5] : v[1]), "r"(part ? v[6] : v[2]),
                         "r"(part ? v[7] : v[3])
                         : "memory");
        }
    }
}
// A row's scales (zeros where the range ends: nothing is multiplied there).
struct RowScales {
    float k, v;
};
__device__ __forceinline__ RowScales row_scales(const KvArgs& a, const Piece& p, int32_t pos) {
    RowScales r{0.f, 0.f};
    int64_t ignore, at;
    if (pos >= p.range.first && pos < p.range.last && slot_of(a, p.b, (uint32_t)pos, ignore, at)) {
        at += (int64_t)p.kv_head * a.s_head;
        r.k = a.k_scale[at];
        r.v = a.v_scale[at];
    }
    return r;
}
template <int FMT, class Args>
__device__ __forceinline__ void widen_role(const KvArgs& a, const Args& t, Shared* sh, uint32_t raw,
                                           uint32_t raw_bytes, uint32_t slots, uint32_t slot_bytes) {
    constexpr int kN = kSlots<FMT>;
    const int warp = (threadIdx.x >> 5) - 8, lane = threadIdx.x & 31;
    const Waiter wait{sh, a.ws};
    uint32_t entry = 0;
    Piece p;
    for (uint32_t n = 0; take_piece(wait, n, &p) && p.count > 0; ++n) {
        const int32_t base = (p.range.lo + p.from) * kTokens + 32 * warp + lane;
        RowScales scales = row_scales(a, p, base);
        for (int32_t j = 0; j < p.count; ++j) {
            {
                // V of tile j - 1 has a slot, so K of tile j - 2 was freed, so both
                // row tiles are done with the scales of tile j - 3: three slots do
                // (narrow items: K of j - 2 meets the queries when tile j - 4 is done)
                const uint32_t n = (entry / 2) % kScaleSlots<Args>;
                sh->k_scale[n][32 * warp + lane] = scales.k;
                sh->v_scale[n][32 * warp + lane] = scales.v;
                const uint32_t bits = scale_bits(scales.v), top = __reduce_max_sync(0xFFFFFFFFu, bits);
                const bool far = __any_sync(0xFFFFFFFFu, bits != 0 && top - bits > kSpread);
                if (lane == 0) sh->v_top[n][warp] = (top & ~1u) | (far ? 1u : 0u);
            }
            if (j + 1 < p.count) scales = row_scales(a, p, base + (j + 1) * kTokens);
#pragma unroll 1
            for (int side = 0; side < 2; ++side, ++entry) {
                const uint32_t s = entry % kN, use = entry / kN, q = entry % kRawSlots, turn = entry / kRawSlots;
                if (!wait(&sh->raw_full[q], turn & 1)) return;
                if (use > 0 && !wait(&sh->kv_free[s], (use - 1) & 1)) return;
                widen_rows<FMT>(raw + q * raw_bytes, slots + s * slot_bytes, a.dim, warp, lane);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    if (side == 0) mbar_arrive(&sh->scale_full[(entry / 2) % kScaleSlots<Args>]);
                    mbar_arrive(&sh->kv_full[s]);
                    mbar_arrive(&sh->raw_free[q]);
                }
            }
        }
    }
}

// Items of drafted tokens that have no more than one tile of rows are narrow: one
// tile's softmax alone leaves the tensor core waiting most of the time, so both
// warpgroups take the same rows (each has them in its Q), the one the tiles of
// tokens of even number, the other the odd ones, and they put their accumulators
// together at the piece's end.  Without and with, 40 to 128 rows (us): 16-bit caches,
// 32 sequences of 2560 77.5 to 78.8, 72.7 to 75.2; 32 of up to 4096 95 to 101, 89 to
// 95; 16 of 20480 234 to 241, 231 to 237.  E4M3, 32 of up to 2560 123 to 129, 114;
// 40 of up to 5000 243 to 252, 235 to 246; 16 of 20480 325, 317 (128 rows: 325, 339).
// INT8 the same where items stay whole or clusters share them (122 to 128, 116; one
// of 1024 21.5 to 23.1, 19.6 to 20.9), but not where they are cut: 12 of 8192 133 to
// 136, 139 to 142; 40 of up to 5000 232 to 242, 242 to 251; 16 of 20480 313 to 316,
// 327 to 334 (two of 65536 at 128 rows: 157, 154); hence not there (launch_one).
// Then the copies bound it: without products and softmax 32 of 2560 take 61 us of 71;
// 16 of 20480 in INT8, of 332: without widening 227, without the softmax 248, with
// copies alone 194.  Items of 128 rows alone, one Q and four slots for tiles (or three,
// and five for codes): 306 (301), but 33 drafted then take 590 for 398.  Two slots for
// tiles and five for codes: 365.  Boxes asked for from the L2 a tile ahead of their
// copies: 251 for 229 (16 x 20480, 16-bit).
// ASKED: whether the call says so, else always (constants where they can be: a number
// read instead cost 16-bit caches 0.3 to 1 %).
template <bool ASKED, class Args>
__device__ __forceinline__ bool narrow(const Args& t, const Piece& p) {
    if constexpr (std::is_same<Args, TreeArgs>::value)
        return live_rows<kRows>(t, p) <= (ASKED ? t.narrow_rows : kTileRows);
    return false;
}
template <int FMT, bool CLUSTERS>
constexpr bool kNarrowAsked = FMT == kKvInt8 && !CLUSTERS;
// Tiles of tokens of warpgroup i.
template <bool ASKED, class Args>
__device__ __forceinline__ int32_t own_tiles(const Args& t, const Piece& p, int i) {
    if (narrow<ASKED>(t, p)) return (p.count - i + 1) / 2;
    return live_rows<kRows>(t, p) > i * kTileRows ? p.count : 0;
}

// ---------------------------------------------------------------- products
// Returns whether this lane is the one that issued them.
template <class M, int SLOTS, bool ASKED, class Args>
__device__ __forceinline__ bool mma_role(const KvArgs& a, const Args& t, Shared* sh, uint32_t q_base,
                                         uint32_t slots, uint32_t slot_bytes) {
    const Waiter wait{sh, a.ws};
    const uint32_t tmem = sh->tmem;
    // a negative scale: Q enters with its sign changed, the softmax takes the scale's size
    const uint32_t qk = instruction(M::kHalf, kTokens, false) | (t.scale < 0.f ? 1u << 13 : 0u);
    const uint32_t pv = instruction(M::kHalf, a.dim > 64 ? 128 : 64, true);
    const int steps = a.dim / 16;
    const uint32_t q_bytes = slot_bytes;
    uint32_t entry = 0;
    uint32_t q_phase[2] = {0, 0}, p_phase[2] = {0, 0};
    // the whole warp walks; one lane issues
    uint32_t leader;
    asm volatile("{ .reg .pred p; elect.sync _|p, 0xFFFFFFFF; selp.u32 %0, 1, 0, p; }" : "=r"(leader));
    auto product_qk = [&](int i, uint32_t slot) {
        if (leader) {
            const uint64_t qd = operand(q_base + i * q_bytes, 16), kd = operand(slots + slot * slot_bytes, 16);
            const uint32_t d = tmem + kColS + 128 * i;
#pragma unroll
            for (int ks = 0; ks < 8; ++ks) {
                constexpr uint32_t kHalf = kHalfBytes >> 4;
                const uint32_t at = (ks >> 2) * kHalf + (ks & 3) * 2;
                if (ks < steps) mma_ss(d, qd + at, kd + at, qk, ks > 0);
            }
            tc_commit(&sh->s_full[i]);
        }
        __syncwarp();
    };
    auto product_pv = [&](int i, uint32_t slot, bool add) {
        if (leader) {
            const uint64_t vd = operand(slots + slot * slot_bytes, kHalfBytes);
            const uint32_t d = tmem + kColO + 128 * i, x = tmem + kColS + 128 * i;
#pragma unroll
            for (int kt = 0; kt < kTokens / 16; ++kt) mma_ts(d, x + 8 * kt, vd + (kt * 2048 >> 4), pv, add || kt > 0);
        }
        __syncwarp();
    };
    auto commit = [&](uint64_t* bar) {
        if (leader) tc_commit(bar);
        __syncwarp();
    };
    Piece p;
    for (uint32_t n = 0; take_piece(wait, n, &p) && p.count > 0; ++n) {
        const int tiles = live_rows<kRows>(t, p) > kTileRows ? 2 : 1;
        const int32_t count = p.count;
        if (narrow<ASKED>(t, p)) {
            // whichever is ready first: scores of tile qk (K there; P of the tile before
            // in its place in TMEM read, by a product issued before), values of tile pv
            int32_t qk = 0, pv = 0;
            uint64_t since = 0;
            auto ready = [&](uint64_t* bar, uint32_t parity) {
                return __all_sync(0xFFFFFFFFu, mbar_test(bar, parity)) != 0;
            };
            while (pv < count) {
                const uint32_t k = entry + 2 * (uint32_t)qk, v = entry + 2 * (uint32_t)pv + 1;
                const int i = pv & 1;
                if (qk < count && qk < pv + 2 && ready(&sh->kv_full[k % SLOTS], (k / SLOTS) & 1) &&
                    (qk > 1 || ready(&sh->q_full[qk], q_phase[qk & 1]))) {
                    if (qk < 2) q_phase[qk] ^= 1;
                    tc_fence_after();
                    product_qk(qk & 1, k % SLOTS);
                    commit(&sh->kv_free[k % SLOTS]);
                    ++qk;
                } else if (pv < qk && ready(&sh->kv_full[v % SLOTS], (v / SLOTS) & 1) &&
                           ready(&sh->p_full[i], p_phase[i])) {
                    p_phase[i] ^= 1;
                    tc_fence_after();
                    product_pv(i, v % SLOTS, pv > 1);
                    commit(&sh->kv_free[v % SLOTS]);
                    if (pv + 2 >= count) commit(&sh->o_full[i]);
                    ++pv;
                } else {  // bounded, as every wait
                    const uint64_t now = globaltimer_ns();
                    if (since == 0) since = now;
                    if (__any_sync(0xFFFFFFFFu, kWaitLimitNs == 0 || now - since > kWaitLimitNs) != 0) {
                        record_error(a.ws, kStatusTimeout);
                        *reinterpret_cast<volatile uint32_t*>(&sh->stop) = 1;
                        return leader != 0;
                    }
                    continue;
                }
                since = 0;
            }
            entry += 2 * (uint32_t)count;
            continue;
        }
        // K of the first tile
        if (!wait(&sh->kv_full[entry % SLOTS], (entry / SLOTS) & 1)) return leader != 0;
        for (int i = 0; i < tiles; ++i) {
            if (!wait(&sh->q_full[i], q_phase[i])) return leader != 0;
            q_phase[i] ^= 1;
            tc_fence_after();
            product_qk(i, entry % SLOTS);
        }
        commit(&sh->kv_free[entry % SLOTS]);
        ++entry;
        for (int32_t j = 0; j < count; ++j) {
            const uint32_t v_entry = entry, k_entry = entry + 1;
            const bool more = j + 1 < count;
            if (!wait(&sh->kv_full[v_entry % SLOTS], (v_entry / SLOTS) & 1)) return leader != 0;
            for (int i = 0; i < tiles; ++i) {
                if (!wait(&sh->p_full[i], p_phase[i])) return leader != 0;
                p_phase[i] ^= 1;
                tc_fence_after();
                product_pv(i, v_entry % SLOTS, j > 0);
                if (more) {
                    if (i == 0 && !wait(&sh->kv_full[k_entry % SLOTS], (k_entry / SLOTS) & 1)) return leader != 0;
                    product_qk(i, k_entry % SLOTS);
                } else {
                    commit(&sh->o_full[i]);
                }
            }
            commit(&sh->kv_free[v_entry % SLOTS]);
            if (more) commit(&sh->kv_free[k_entry % SLOTS]);
            entry += more ? 2 : 1;
        }
    }
    return leader != 0;
}

// ---------------------------------------------------------------- softmax
// Rows 32 warp .. + 31 of row tile i of Q into shared memory, 16 lanes a row;
// rows that do not exist are zeros.  A row that goes as it is comes by
// asynchronous copies, which the caller waits for; bf16 rows for 8-bit caches
// pass through registers for their power of two, and what undoes that of row
// 32 warp + lane is returned.  (Code that runs once an item is fetched anew each
// time and waits behind the K and V copies in flight: it is kept short, with few
// rounds to memory.)
template <class T, int FMT>
__device__ __forceinline__ float bring_rows(const KvArgs& a, const AttnArgs& t, const Piece& p, int i, int warp,
                                            uint32_t q_tile) {
    const int lane = threadIdx.x & 31, chunk = lane & 15;
    const int row0 = i * kTileRows + 32 * warp, live = live_rows<kRows>(t, p) - row0;
    const RowPlace mine = row_place(t, p, kRows, row0 + lane);
    const int64_t from = mine.token * t.q_token + (int64_t)mine.head * t.q_head;
    const bool inside = 8 * chunk < a.dim;
    float inverse = 1.f;
    if (FMT == kKv16Bit || T::kHalf) {
#pragma unroll 4
        for (int k = 0; k < 32; k += 2) {
            const int row = k + (lane >> 4);
            const int64_t at = __shfl_sync(0xFFFFFFFFu, from, row);
            const bool real = row < live;
            if (inside) copy16(q_tile + swizzled(32 * warp + row, chunk), t.q + (real ? at + 16 * chunk : 0), real);
        }
        copy_commit();
        return inverse;
    }
    constexpr int kEach = 8;  // loads in flight
#pragma unroll 1
    for (int part = 0; part < 32; part += 2 * kEach) {
        uint4 x[kEach];
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            const int row = part + 2 * k + (lane >> 4);
            const int64_t at = __shfl_sync(0xFFFFFFFFu, from, row);
            x[k] = make_uint4(0, 0, 0, 0);
            if (row < live && inside) x[k] = *reinterpret_cast<const uint4*>(t.q + at + 16 * chunk);
        }
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            uint4 y = x[k];
            uint32_t top = vmax_u16x2(vmax_u16x2(y.x & 0x7FFF7FFFu, y.y & 0x7FFF7FFFu),
                                      vmax_u16x2(y.z & 0x7FFF7FFFu, y.w & 0x7FFF7FFFu));
#pragma unroll
            for (int o = 1; o < 16; o <<= 1) top = vmax_u16x2(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
            const float power = query_power<T>(max(top & 0xFFFFu, top >> 16));
            y = make_uint4(scaled_pair<T>(y.x, power), scaled_pair<T>(y.y, power), scaled_pair<T>(y.z, power),
                           scaled_pair<T>(y.w, power));
            const float to_owner = __shfl_sync(0xFFFFFFFFu, power, (lane & 1) * 16);
            if ((lane >> 1) == part / 2 + k) inverse = 1.f / to_owner;
            if (inside)
                asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(
                                 q_tile + swizzled(32 * warp + part + 2 * k + (lane >> 4), chunk)),
                             "r"(y.x), "r"(y.y), "r"(y.z), "r"(y.w)
                             : "memory");
        }
    }
    return inverse;
}

// 64 columns of a warp's 32 result rows (16-bit, a row a lane) to global
// memory, STEP rows at a time through shared memory, so that a store
// instruction writes 128-byte runs.  to: where this lane's row goes (null:
// nowhere); the first `bytes` of the 128 exist.  Chunk c of row r lies at chunk
// c ^ r: the writing lanes (rows) and the reading ones (chunks) meet all banks.
template <int STEP>
__device__ __forceinline__ void store_rows(uint32_t stage, const uint32_t* words, uint8_t* to, int bytes) {
    const int lane = threadIdx.x & 31, chunk = lane & 7;
#pragma unroll 1
    for (int pass = 0; pass < 32; pass += STEP) {
        __syncwarp();
        const int r = lane - pass;
        if (r >= 0 && r < STEP) {
#pragma unroll
            for (int c = 0; c < 8; ++c)
                asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(stage + r * 128 + ((c ^ (r & 7)) << 4)),
                             "r"(words[4 * c]), "r"(words[4 * c + 1]), "r"(words[4 * c + 2]), "r"(words[4 * c + 3])
                             : "memory");
        }
        __syncwarp();
#pragma unroll
        for (int k = 0; k < STEP; k += 4) {
            const int row = k + (lane >> 3);
            const uint64_t dst = __shfl_sync(0xFFFFFFFFu, reinterpret_cast<uint64_t>(to), pass + row);
            uint4 x;
            asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                         : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
                         : "r"(stage + row * 128 + ((chunk ^ (row & 7)) << 4)));
            if (dst != 0 && 16 * chunk < bytes) *reinterpret_cast<uint4*>(dst + 16 * chunk) = x;
        }
    }
}

// 32 scales (every lane the same ones), asked for together.
__device__ __forceinline__ void load_scales(uint32_t at, float2* f) {
#pragma unroll
    for (int k = 0; k < 16; k += 2)
        asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];"
                     : "=f"(f[k].x), "=f"(f[k].y), "=f"(f[k + 1].x), "=f"(f[k + 1].y)
                     : "r"(at + 8 * k));
}

// Whether a tile's value scales lie further apart than kSpread; v: its v_top.
__device__ __forceinline__ bool scales_apart(const uint4& v) {
    const uint32_t most = max(max(v.x, v.y), max(v.z, v.w));
    auto low = [&](uint32_t x) { return x != 0 && most - x > kSpread; };
    return ((v.x | v.y | v.z | v.w) & 1u) != 0 || low(v.x) || low(v.y) || low(v.z) || low(v.w);
}
// n low bits set (0 for n <= 0, all for n >= 32)
__device__ __forceinline__ uint32_t bits_below(int32_t n) {
    return n <= 0 ? 0u : (n >= 32 ? 0xFFFFFFFFu : (1u << n) - 1u);
}

template <class T, int FMT, bool ASKED, class Args>
__device__ __forceinline__ void softmax_role(const KvArgs& a, const Args& t, Shared* sh, uint32_t q_tile,
                                             uint32_t stages, float* joint) {
    using M = Operand<T, FMT>;
    constexpr bool kTree = std::is_same<Args, TreeArgs>::value;
    const int i = threadIdx.x / 128, row = threadIdx.x % 128, warp = row >> 5, lane = row & 31;
    const int me = threadIdx.x >> 5;
    const Waiter wait{sh, a.ws};
    const uint32_t tmem = sh->tmem + ((uint32_t)(32 * warp) << 16), stage = stages + me * (128 * kStageRows<FMT, Args>);
    const uint32_t at_s = tmem + kColS + 128 * i, at_o = tmem + kColO + 128 * i;
    const float scale_base2 = fabsf(t.scale) * 1.4426950408889634f;
    // hidden scores are -infinity when the scale meets them: a scale of zero (or one
    // that a row's power makes zero) is the smallest number instead, which leaves
    // nothing of any finite score
    const float least = __uint_as_float(1u);
    uint32_t s_phase = 0, o_phase = 0, taken = 0, tile = 0;  // tile: this block's tiles of tokens, whoever's
    int slot = 1;                                 // of the piece at hand
    int32_t first = 0, last = 0;                  // what this row sees
    uint32_t halves = 0;                          // narrow pieces put together so far
    float m = -INFINITY, l = 0.f;
    uint32_t skipped = 0;  // tiles of pieces without rows for this warpgroup, since the one at hand
    for (bool open = false;;) {  // open: a piece is at hand
        // the next piece that has rows for this warpgroup.  Its rows of Q may
        // come now: the last S is done, so is every product with these.
        float to_base2 = 1.f;
        bool found = true;
        Piece* const next = &sh->piece[me][slot ^ 1];
        for (;;) {
            Piece p;
            if (!take_piece(wait, taken, &p)) return;
            ++taken;
            if (p.count > 0 && own_tiles<ASKED>(t, p, i) == 0) {
                skipped += (uint32_t)p.count;
                // A shared piece is put together first: the other warpgroup, which waits
                // for that, has taken one piece more and no others, so that a run of
                // these would end where the ring is full.
                found = !(kTree && open);
                if (found) continue;
            } else {
                if (lane == 0) *next = p;
                __syncwarp();
            }
            break;
        }
        const bool more = found && next->count > 0;
        if (more)
            to_base2 = fmaxf(
                scale_base2 * bring_rows<T, FMT>(a, t, *next, narrow<ASKED>(t, *next) ? 0 : i, warp, q_tile), least);
        if (open) {  // the end of the piece at hand
            const Piece& cur = sh->piece[me][slot];
            if (!wait(&sh->o_full[i], o_phase)) return;
            o_phase ^= 1;
            tc_fence_after();
            const bool full = cur.count == cur.range.n;
            // narrow: the other warpgroup has the rest of these rows' tiles
            const bool shared = narrow<ASKED>(t, cur) && cur.count > 1;
            const int tile_row = (narrow<ASKED>(t, cur) ? 0 : i * kTileRows) + row;
            const bool is_row = tile_row < live_rows<kRows>(t, cur);
            const RowPlace at = row_place(t, cur, kRows, tile_row);
            const PartLayout parts = part_layout(a, gridDim.x, kRows);
            const int which = cur.from > 0 ? 0 : 1;
            float* const acc = joint != nullptr ? joint : parts.acc(blockIdx.x, which);
            float* const stats = joint != nullptr ? joint + kRows * a.dim : parts.stats(blockIdx.x, which);
            // a joint part takes the tiles' place: when both row tiles' products are done
            if (joint != nullptr && live_rows<kRows>(t, cur) > kTileRows && !wait(&sh->o_full[1], 0)) return;
            float mine = 1.f, theirs = 0.f;  // the accumulators' weights
            if (kTree && shared) {
                Halves& half = halves_of(sh);
                half.m[i][row] = m;
                half.l[i][row] = l;
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh->half_full[i]);
                if (!wait(&sh->half_full[i ^ 1], halves & 1)) return;
                ++halves;
                tc_fence_after();
                const float other = half.m[i ^ 1][row], to = fmaxf(m, other);
                const float base = to == -INFINITY ? 0.f : to;
                mine = exp2_fast(m - base);
                theirs = exp2_fast(other - base);
                l = l * mine + half.l[i ^ 1][row] * theirs;
                m = to;
            }
            // two warpgroups with the same rows take 64 columns of them in turn
            const int from = kTree && shared ? 64 * i : 0, step = kTree && shared ? 128 : 64;
            const bool none = kTree ? is_row && sees_none(t, cur.seq, at.token, at.pos, l) : last <= first;
            const float inv = none ? 0.f : 1.f / l;
            bool odd = false;
            if (full) {
                uint8_t* const to = t.out + at.token * t.o_token + (int64_t)at.head * t.o_head;
#pragma unroll 1
                for (int c = from; c < a.dim; c += step) {
                    uint32_t o[64], y[32];
                    tc_load32(at_o + c, o);
                    tc_load32(at_o + c + 32, o + 32);
                    tc_wait_load();
                    if (kTree && shared) {
#pragma unroll
                        for (int h = 0; h < 64; h += 16) {
                            uint32_t x[16];
                            tc_load16((i == 0 ? at_o + 128 : at_o - 128) + c + h, x);
                            tc_wait_load();
#pragma unroll
                            for (int k = 0; k < 16; ++k)
                                o[h + k] = __float_as_uint(__uint_as_float(o[h + k]) * mine +
                                                           __uint_as_float(x[k]) * theirs);
                        }
                    }
#pragma unroll
                    for (int k = 0; k < 64; k += 2) {
                        const float u = none ? 0.f : __uint_as_float(o[k]) * inv;
                        const float v = none ? 0.f : __uint_as_float(o[k + 1]) * inv;
                        odd |= c + k < a.dim && !(fabsf(u) <= 3.402823466e+38f && fabsf(v) <= 3.402823466e+38f);
                        y[k / 2] = pack<T>(u, v);
                    }
                    store_rows<kStageRows<FMT, Args>>(stage, y, is_row ? to + 2 * c : nullptr, 2 * (a.dim - c));
                }
            } else {
                float* dst = acc + tile_row;
#pragma unroll 1
                for (int c = from; c < a.dim; c += 16) {
                    if (kTree && shared && (c & 64) != from) continue;
                    uint32_t o[16];
                    tc_load16(at_o + c, o);
                    tc_wait_load();
                    if (kTree && shared) {
                        uint32_t x[16];
                        tc_load16((i == 0 ? at_o + 128 : at_o - 128) + c, x);
                        tc_wait_load();
#pragma unroll
                        for (int k = 0; k < 16; ++k)
                            o[k] = __float_as_uint(__uint_as_float(o[k]) * mine + __uint_as_float(x[k]) * theirs);
                    }
                    if (is_row) {
#pragma unroll
                        for (int k = 0; k < 16; ++k) dst[(size_t)(c + k) * kRows] = __uint_as_float(o[k]);
                    }
                }
            }
            if (!(kTree && shared && i != 0)) {
                if (full) {
                    if (is_row && t.lse != nullptr)
                        t.lse[at.token * t.q_heads + at.head] = none ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
                } else if (is_row) {
                    stats[tile_row] = m;
                    stats[kRows + tile_row] = l;
                }
            }
            if (full && odd && is_row) *reinterpret_cast<volatile uint32_t*>(&sh->odd) = 1;
            tc_fence_before();
            if (kTree && shared) {
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh->half_read[i]);
            }
        }
        open = false;
        if (kTree && !found) continue;
        if (!more) return;
        copy_wait<0>();
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh->q_full[i]);
        slot ^= 1;
        tile += skipped;
        skipped = 0;
        open = true;
        const Piece& cur = sh->piece[me][slot];
        first = last = 0;
        const bool alone = kTree && narrow<ASKED>(t, cur);  // its rows are row tile 0's
        const RowPlace own = row_place(t, cur, kRows, (alone ? 0 : i * kTileRows) + row);
        const bool is_row = (alone ? 0 : i * kTileRows) + row < live_rows<kRows>(t, cur);
        if (is_row) search_range(t, cur.seq, own.token, own.pos, first, last);
        const int32_t count = cur.count, stride = alone ? 2 : 1;
        m = -INFINITY;
        l = 0.f;
        int32_t base = (cur.range.lo + cur.from) * kTokens;
        if (alone && i != 0) {
            ++tile;
            base += kTokens;
        }
        const bool idle = kTree && __any_sync(0xFFFFFFFFu, is_row) == 0;  // a warp without rows
        // every place from here to there is seen by all of the warp's rows
        const int32_t whole_from = kTree ? __reduce_max_sync(0xFFFFFFFFu, is_row ? first : 0) : 0;
        const int32_t whole_to =
            kTree ? __reduce_min_sync(0xFFFFFFFFu, is_row ? gapless_below(t, cur.seq, last) : 0x7FFFFFFF) : 0;
        // one tile of tokens; false: a wait ran out.  MASKED: some places are hidden
        // from some rows (drafted tokens: in code of its own, since as a branch that is
        // hardly ever taken it cost every tile 10 %)
        auto one_tile = [&](bool start, auto masked) -> bool {
            constexpr bool kMasked = decltype(masked)::value;
            const uint32_t scale_slot = tile % kScaleSlots<Args>;
            if (FMT != kKv16Bit && !wait(&sh->scale_full[scale_slot], (tile / kScaleSlots<Args>) & 1)) return false;
            uint32_t s[kTokens];
#pragma unroll
            for (int c = 0; c < kTokens; c += 32) tc_load32(at_s + c, s + c);
            tc_wait_load();
            if (FMT != kKv16Bit) {
                const uint32_t at = smem_addr(&sh->k_scale[scale_slot][0]);
#pragma unroll
                for (int c = 0; c < kTokens; c += 32) {
                    float2 f[16];
                    load_scales(at + 4 * c, f);
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        const float2 x = mul2(make_float2(__uint_as_float(s[c + 2 * k]), __uint_as_float(s[c + 2 * k + 1])),
                                              f[k]);
                        s[c + 2 * k] = __float_as_uint(x.x);
                        s[c + 2 * k + 1] = __float_as_uint(x.y);
                    }
                }
            }
            if (kTree ? kMasked : base < first || base + kTokens > last) {
#pragma unroll
                for (int c = 0; c < kTokens; c += 32) {
                    uint32_t seen = bits_below(last - base - c) & ~bits_below(first - base - c);
                    if (seen != 0) seen &= seen_32(t, cur.seq, own.token, base + c);
#pragma unroll
                    for (int k = 0; k < 32; ++k) s[c + k] = (seen >> k & 1u) != 0 ? s[c + k] : 0xFF800000u;
                }
            }
            float top0 = -INFINITY, top1 = -INFINITY;
#pragma unroll
            for (int c = 0; c < kTokens; c += 4) {
                top0 = max3(top0, __uint_as_float(s[c]), __uint_as_float(s[c + 1]));
                top1 = max3(top1, __uint_as_float(s[c + 2]), __uint_as_float(s[c + 3]));
            }
            float top = fmaxf(top0, top1) * to_base2;
            uint4 v{};
            if (FMT != kKv16Bit) {
                v = *reinterpret_cast<const uint4*>(sh->v_top[scale_slot]);
                top += scale_log2(max(max(v.x, v.y), max(v.z, v.w)));
            }
            const bool move = start || __any_sync(0xFFFFFFFFu, top > m + (kSlack<M> + kLower<M>));
            // 8-bit caches: so far a bound of what the tile adds at most; what it is
            // exactly is only looked for where the reference would follow it
            if (FMT != kKv16Bit && move && scales_apart(v)) {
                top = -INFINITY;
#pragma unroll 1
                for (int c = 0; c < kTokens; c += 8) {
                    uint32_t o[8];  // S again: few registers
                    tc_load8(at_s + c, o);
                    tc_wait_load();
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const float x = __uint_as_float(o[k]) * sh->k_scale[scale_slot][c + k];
                        const float y = fmaf(x, to_base2, scale_log2(scale_bits(sh->v_scale[scale_slot][c + k])));
                        const int32_t at = base + c + k;
                        if (at >= first && at < last && (!kMasked || drafted_seen(t, cur.seq, own.token, at)))
                            top = fmaxf(top, y);
                    }
                }
            }
            if (start) {
                m = top - kLower<M>;
            } else if (move) {
                const float to = fmaxf(m, top - kLower<M>);
                const float f = to == -INFINITY ? 1.f : exp2_fast(m - to);
                m = to;
                l *= f;
#pragma unroll 1
                for (int c = 0; c < a.dim; c += 32) {  // (128 columns are its own at any dim)
                    uint32_t o[32];
                    tc_load32(at_o + c, o);
                    tc_wait_load();
#pragma unroll
                    for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                    tc_store32(at_o + c, o);
                }
            }
            const float from = m == -INFINITY ? 0.f : -m;
            const float2 scale2 = make_float2(to_base2, to_base2), from2 = make_float2(from, from);
            float2 sum0 = make_float2(0.f, 0.f), sum1 = make_float2(0.f, 0.f);
            uint32_t pr[kTokens / 2];
#pragma unroll
            for (int c = 0; c < kTokens; c += 32) {
                float2 f[16];
                if (FMT != kKv16Bit) load_scales(smem_addr(&sh->v_scale[scale_slot][0]) + 4 * c, f);
#pragma unroll
                for (int k = 0; k < 16; k += 2) {
                    const int i0 = c + 2 * k;
                    float2 x = fma2(make_float2(__uint_as_float(s[i0]), __uint_as_float(s[i0 + 1])), scale2, from2);
                    float2 y = fma2(make_float2(__uint_as_float(s[i0 + 2]), __uint_as_float(s[i0 + 3])), scale2, from2);
                    x.x = exp2_fast(x.x);
                    x.y = exp2_fast(x.y);
                    y.x = exp2_fast(y.x);
                    y.y = exp2_fast(y.y);
                    sum0 = add2(sum0, x);
                    sum1 = add2(sum1, y);
                    if (FMT != kKv16Bit) {
                        x = mul2(x, f[k]);
                        y = mul2(y, f[k + 1]);
                    }
                    pr[i0 / 2] = pack<M>(x.x, x.y);
                    pr[i0 / 2 + 1] = pack<M>(y.x, y.y);
                }
                if (c % 64 == 32) tc_store32(at_s + (c / 64) * 32, pr + (c / 64) * 32);
            }
            sum0 = add2(sum0, sum1);
            l += sum0.x + sum0.y;
            tc_wait_store();
            return true;
        };
        int32_t j = alone ? i : 0;
        bool start = true;
        for (; j < count; j += stride, tile += stride, base += stride * kTokens, start = false) {
            if (!wait(&sh->s_full[i], s_phase)) return;
            s_phase ^= 1;
            tc_fence_after();
            if constexpr (kTree) {
                if (!idle) {  // (what an idle warp's rows come to is nobody's)
                    if (base >= whole_from && base + kTokens <= whole_to) {
                        if (!one_tile(start, std::false_type{})) return;
                    } else {
                        if (!one_tile(start, std::true_type{})) return;
                    }
                }
                // the other warpgroup may still be reading this one's accumulator of the piece before
                if (start && halves > 0 && !wait(&sh->half_read[i ^ 1], (halves - 1) & 1)) return;
            } else {
                if (!one_tile(start, std::false_type{})) return;
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh->p_full[i]);
        }
        // on to the end of the piece's tiles, whoever's
        if (alone) tile -= (uint32_t)(j - count);
    }
}

// Warps 0 to 7, after the cluster's PARTS blocks have left their parts of item
// ring[0] at `joint` of their shared memory: this block joins 256 / PARTS of the
// rows, 32 rows and 16 channels a warp at a time, in the parts' order.
template <class T, int FMT, int PARTS, class Args>
__device__ __forceinline__ void join_item(const KvArgs& a, const Args& t, Shared* sh, uint32_t joint) {
    const Piece p = sh->ring[0];
    const int n = parts_of(p, PARTS);
    if (n < 2) return;  // no item, or its only block wrote the result
    constexpr int kJoinRows = kRows / PARTS;
    const int row0 = (int)cluster_rank() * kJoinRows, live = live_rows<kRows>(t, p);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll 1
    for (int u = warp; u < kJoinRows / 32 * (a.dim / 16); u += 8) {
        const int band = u % (kJoinRows / 32), d = 16 * (u / (kJoinRows / 32)), row = row0 + 32 * band + lane;
        if (row >= live) continue;
        float part_m[PARTS], part_sum[PARTS], x[PARTS][16];
#pragma unroll
        for (int k = 0; k < PARTS; ++k) {  // of fewer parts the last again, with no weight
            const int part = min(k, n - 1);
            const uint32_t from = in_block(joint + 4 * row, part);
            part_m[k] = load_cluster(from + 4 * kRows * a.dim);
            part_sum[k] = load_cluster(from + 4 * kRows * (a.dim + 1));
#pragma unroll
            for (int e = 0; e < 16; ++e) x[k][e] = load_cluster(from + 4 * kRows * (d + e));
        }
        float m = -INFINITY;
#pragma unroll
        for (int k = 0; k < PARTS; ++k) m = fmaxf(m, part_m[k]);
        const float base = m == -INFINITY ? 0.f : m;
        float sum = 0.f, v[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] = 0.f;
#pragma unroll
        for (int k = 0; k < PARTS; ++k) {
            const float f = k < n ? exp2f(part_m[k] - base) : 0.f;
            sum += f * part_sum[k];
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] += f * x[k][e];
        }
        bool odd = store_row_part<T>(t, p, kRows, row, d, v, m, sum);
        odd |= store_row_part<T>(t, p, kRows, row, d + 8, v + 8, m, sum);
        if (odd) *reinterpret_cast<volatile uint32_t*>(&sh->odd) = 1;
    }
}

// The same warps, when their part in the pipeline is over and some row came out
// non-finite: the rows that the block wrote are looked through and those worked out
// again.  (Not between two pieces: a row's keys are gone through by one warp, and
// no bounded wait may span that.)  Rows from + warp, + 8 and so on, below `to`.
template <class T, int FMT, class Args>
__device__ __forceinline__ void repair_rows(const KvArgs& a, const Args& t, const Piece& p, int from, int to) {
    constexpr uint32_t kExponent = T::kHalf ? 0x7C00u : 0x7F80u;
    const int lane = threadIdx.x & 31, end = min(to, live_rows<kRows>(t, p));
    for (int row = from + (threadIdx.x >> 5); row < end; row += 8) {
        const RowPlace at = row_place(t, p, kRows, row);
        const uint16_t* out =
            reinterpret_cast<const uint16_t*>(t.out + at.token * t.o_token + (int64_t)at.head * t.o_head);
        bool odd = false;
        for (int d = lane; d < a.dim; d += 32) odd |= (out[d] & kExponent) == kExponent;
        if (__any_sync(0xFFFFFFFFu, odd)) fix_row<T, FMT>(a, t, p, kRows, row);
    }
}
// cluster: the blocks that share an item, or 1.
template <class T, int FMT, class Args>
__device__ __noinline__ void repair_role(const KvArgs& a, const Args& t, Shared* sh, int whole, int cluster) {
    Piece p;
    if (cluster > 1) {
        p = sh->ring[0];
        const int rank = (int)cluster_rank(), rows = kRows / cluster;
        if (parts_of(p, cluster) > 1)
            repair_rows<T, FMT>(a, t, p, rank * rows, (rank + 1) * rows);
        else if (p.count > 0)
            repair_rows<T, FMT>(a, t, p, 0, kRows);
        return;
    }
    Walk w = make_walk(sh->prefix[a.batch], blockIdx.x, gridDim.x, whole);
    while (next_piece<kRows, kTokens>(a, t, sh->prefix, w, p))
        if (p.count == p.range.n) repair_rows<T, FMT>(a, t, p, 0, kRows);  // cut items: where they are joined
}

// how: whether items are left whole (0: they are cut at shares' ends); with
// CLUSTERS how many blocks, a cluster, share each item.  (Kernels of their own:
// as one with the others they cost those 1 %.)
template <class T, int FMT, class Args, bool CLUSTERS>
__global__ void __launch_bounds__(kThreads, 1)
    attend_chunk_kernel(const __grid_constant__ KvArgs a, const __grid_constant__ Args t,
                        const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map, int32_t box,
                        int how) {
    constexpr int kN = kSlots<FMT>;
    extern __shared__ uint8_t raw[];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    // tiles at 1024-byte boundaries (the swizzle's period): Q0, Q1, the K and V slots, then the rest
    const uint32_t base = (smem_addr(raw) + 1023) & ~1023u;
    const uint32_t tile_bytes = (a.dim > 64 ? 2 : 1) * kHalfBytes;
    const uint32_t raw_bytes = FMT == kKv16Bit ? 0 : kRawSlots * kTokens * a.dim;
    Shared* sh = reinterpret_cast<Shared*>(raw + (base - smem_addr(raw)) + (2 + kN) * tile_bytes + raw_bytes +
                                           kStageBytes<FMT, Args>);
    const int warp = threadIdx.x >> 5;
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(&sh->tmem))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    if (threadIdx.x == 32) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh->q_full[i], 4);
            mbar_init(&sh->s_full[i], 1);
            mbar_init(&sh->p_full[i], 4);
            mbar_init(&sh->o_full[i], 1);
        }
        for (int i = 0; i < kN; ++i) {
            mbar_init(&sh->kv_full[i], kLoaderWarps);
            mbar_init(&sh->kv_free[i], 1);
        }
        for (int i = 0; i < kRawSlots; ++i) {
            mbar_init(&sh->raw_full[i], 2);
            mbar_init(&sh->raw_free[i], kLoaderWarps);
        }
        for (int i = 0; i < kMostScaleSlots; ++i) mbar_init(&sh->scale_full[i], kLoaderWarps);
        for (int i = 0; i < kRing; ++i) {
            mbar_init(&sh->piece_full[i], 1);
            mbar_init(&sh->piece_free[i], FMT == kKv16Bit ? 13 : 15);  // the warps that take pieces
        }
        mbar_init(&sh->drained, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh->half_full[i], 4);
            mbar_init(&sh->half_read[i], 4);
        }
        sh->stop = sh->odd = 0;
        fence_mbar_init();
    }
    int cluster = 1;
    if constexpr (CLUSTERS) {
        build_prefix<kRows, 0>(a, t, sh->prefix);
        // (more items than the call's bounds allow: every block for itself)
        if (sh->prefix[a.batch] <= gridDim.x / how) cluster = how;
        __syncthreads();
    }
    if (cluster == 1) build_prefix<kRows, kTokens>(a, t, sh->prefix);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t slots = base + 2 * tile_bytes, raw_codes = slots + kN * tile_bytes;
    const Fetch fetch{&k_map, &v_map, box};
    if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
        // 256 rows of sums and two statistics: less than Q and the slots, at every dim
        float* const joint = reinterpret_cast<float*>(raw + (base - smem_addr(raw)));
        softmax_role<T, FMT, kNarrowAsked<FMT, CLUSTERS>>(a, t, sh, base + (warp / 4) * tile_bytes, raw_codes + raw_bytes,
                             CLUSTERS && cluster > 1 ? joint : nullptr);
        copy_wait<0>();  // of Q, where the role gave up
        __syncwarp();
        if (CLUSTERS && cluster > 1) {
            cluster_sync();
            if (cluster == 2)
                join_item<T, FMT, 2>(a, t, sh, base);
            else
                join_item<T, FMT, 4>(a, t, sh, base);
            __syncwarp();
        }
        asm volatile("bar.sync 1, 256;" ::: "memory");
        if (sh->odd != 0 && sh->stop == 0) repair_role<T, FMT>(a, t, sh, CLUSTERS ? 1 : how, cluster);
    } else if (warp < 12) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kLoaderRegs));
        if constexpr (FMT == kKv16Bit)
            fetch_role<FMT, 4, kN>(a, t, sh, fetch, warp - 8, slots, tile_bytes, sh->kv_full, sh->kv_free);
        else
            widen_role<FMT>(a, t, sh, raw_codes, kTokens * a.dim, slots, tile_bytes);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kLoaderRegs));
        if (warp == 12) {
            const bool issued =
                mma_role<Operand<T, FMT>, kN, kNarrowAsked<FMT, CLUSTERS>>(a, t, sh, base, slots, tile_bytes);
            __syncwarp();
            // every product is done before TMEM goes (the thread that issued them says so)
            if (issued) tc_commit(&sh->drained);
            mbar_wait(&sh->drained, 0, kDrainLimitNs);
        } else if (warp != 14 && FMT != kKv16Bit) {  // 13 and 15
            fetch_role<FMT, 2, kRawSlots>(a, t, sh, fetch, (warp - 13) / 2, raw_codes, kTokens * a.dim, sh->raw_full,
                                          sh->raw_free);
        } else if (warp == 14) {
            if (CLUSTERS && cluster > 1)
                share_role(a, t, sh, cluster);
            else
                walk_role(a, t, sh, make_walk(sh->prefix[a.batch], blockIdx.x, gridDim.x, CLUSTERS ? 1 : how));
        }
    }
    __syncwarp();
    if (CLUSTERS && cluster > 1) {
        if (warp >= 8) cluster_sync();
        cluster_sync();  // nobody's shared memory is given up before all have read it
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(sh->tmem) : "memory");
}

template <int FMT, class Args>
constexpr size_t shared_bytes(int dim) {
    return 1024 + (size_t)(2 + kSlots<FMT>) * (dim > 64 ? 2 : 1) * kHalfBytes +
           (FMT == kKv16Bit ? 0 : (size_t)kRawSlots * kTokens * dim) + kStageBytes<FMT, Args> + sizeof(Shared) +
           kHalvesBytes<Args>;
}

static_assert(1024 * (128 + 2) <= (2 + kSlots<kKvInt8>) * 2 * kHalfBytes &&
                  1024 * (64 + 2) <= (2 + kSlots<kKvInt8>) * kHalfBytes,
              "a joint part takes the place of Q and the slots");
static_assert(shared_bytes<kKv16Bit, AttnArgs>(128) <= 232448 && shared_bytes<kKvInt8, AttnArgs>(128) <= 232448 &&
                  shared_bytes<kKv16Bit, TreeArgs>(128) <= 232448 && shared_bytes<kKvInt8, TreeArgs>(128) <= 232448,
              "227 KB a block");

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeFn encode_fn() {
    static const EncodeFn fn = []() -> EncodeFn {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess) {
            cudaGetLastError();
            return nullptr;
        }
        return reinterpret_cast<EncodeFn>(p);
    }();
    return fn;
}
// K or V as (channel, slot, head, page); a box is up to 64 channels of 16-bit
// values with the products' swizzle, or all channels of codes, of `box` slots.
// False where TMA's rules do not hold (the copies then go another way).
bool make_map(CUtensorMap* map, void* data, bool wide, const KvArgs& a, int32_t box) {
    const EncodeFn encode = encode_fn();
    if (encode == nullptr) return false;
    const cuuint64_t dims[4] = {(cuuint64_t)a.dim, a.page_tokens.d, (cuuint64_t)a.kv_heads, (cuuint64_t)a.pages};
    const int64_t given[3] = {a.token_stride, a.head_stride, a.page_stride};
    cuuint64_t strides[3];
    for (int i = 0; i < 3; ++i) {
        // an axis of one entry has no step: any legal one will do
        strides[i] = dims[i + 1] == 1 ? 16 * ((cuuint64_t)a.dim) : (cuuint64_t)given[i];
        if (strides[i] == 0 || strides[i] >= (1ull << 40)) return false;
    }
    const cuuint32_t boxes[4] = {wide ? 64u : (cuuint32_t)a.dim, (cuuint32_t)box, 1, 1}, steps[4] = {1, 1, 1, 1};
    return encode(map, wide ? CU_TENSOR_MAP_DATA_TYPE_UINT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, data, dims, strides,
                  boxes, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  wide ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// Tokens of a TMA box: a page where pages of 8 tokens or more divide a tile,
// a tile where tiles divide a page, else none.
int32_t box_tokens(uint32_t page_tokens) {
    if (page_tokens % kTokens == 0) return kTokens;
    return page_tokens >= 8 && kTokens % page_tokens == 0 ? (int32_t)page_tokens : 0;
}

constexpr int join_bytes(int dim) { return (int)sizeof(float) * kJoinMany * (dim + 1); }

template <class T, int FMT, class Args>
cudaError_t launch_one(const KvArgs& a, Args t, int max_new, int max_len, cudaStream_t s) {
    static PerDeviceOnce once;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    e = once.run(dev, [] {
        const cudaError_t set = cudaFuncSetAttribute(join_columns_kernel<T, FMT, kRows, Args>,
                                                     cudaFuncAttributeMaxDynamicSharedMemorySize, join_bytes(128));
        if (set != cudaSuccess) return set;
        const cudaError_t both = cudaFuncSetAttribute(attend_chunk_kernel<T, FMT, Args, true>,
                                                      cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                      (int)shared_bytes<FMT, Args>(128));
        if (both != cudaSuccess) return both;
        return cudaFuncSetAttribute(attend_chunk_kernel<T, FMT, Args, false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    (int)shared_bytes<FMT, Args>(128));
    });
    if (e != cudaSuccess) return e;
    CUtensorMap k_map{}, v_map{};
    int32_t box = box_tokens(a.page_tokens.d);
    constexpr bool kWide = FMT == kKv16Bit;
    if (box > 0 && !(make_map(&k_map, a.k, kWide, a, box) && make_map(&v_map, a.v, kWide, a, box))) box = 0;
    // Cutting items costs a second kernel and the parts' way through memory, 8 to
    // 12 us; not cutting them costs up to one item's time at the end.  Six chunks
    // of up to 97 tokens over 1500: 32.6 us whole, 37.3 cut; three of 700 over
    // 2500: 49.9, 63.9; two of 256 over 4096: 63.9, 45.4.
    const bool whole = max_len <= 20 * kTokens;
    // Few items: each is shared by a cluster of 2 or 4 blocks.  At most 128 blocks:
    // clusters that cannot be resident together run one after the other (16 of 8
    // blocks do).  Without, with (us, 16-bit): 128 new tokens (16 items, 4 blocks)
    // over 256: 14.1, 15.7 (not taken); 512: 17.1, 15.5; 1024: 24.1, 17.1; 4096:
    // 39.0, 26.5; 8192: 48.0, 40.0; 16384: 58.0, 65.9 (not taken).  512 new (64
    // items, 2 blocks) over 512: 18.1, 20.3 (not taken); 1024: 25.1, 21.2; 2048:
    // 37.4, 27.5; 4096: 50.6, 39.7.  INT8: 128 over 1024: 34.0, 22.5; 2 x 256 over
    // 2048: 52.2, 36.4.
    const int64_t tiled = (int64_t)a.batch * a.kv_heads * (((int64_t)t.group.d * max_new + kRows - 1) / kRows);
    const int cluster = 4 * tiled <= 128 ? 4 : 2 * tiled <= 128 ? 2 : 1;
    const bool clusters = cluster > 1 && max_len > (cluster == 4 ? 3 : 7) * kTokens && max_len <= 16 * cluster * kTokens;
    if constexpr (std::is_same<Args, TreeArgs>::value)
        t.narrow_rows = kNarrowAsked<FMT, false> && !whole ? 0 : kTileRows;
    if (clusters)
        return launch_clusters(attend_chunk_kernel<T, FMT, Args, true>, (int)tiled * cluster, cluster, kThreads,
                               shared_bytes<FMT, Args>(a.dim), s, a, t, k_map, v_map, box, cluster);
    int shares = shares_for(a, t, max_new, max_len, kRows, kTokens, kShares);
    // One tree with several row tiles a head: with as many shares for each item its
    // row tiles are walked in step, and all but the first find their tokens in the L2.
    // Not where that leaves more than a tenth of the SMs without a share.  152 shares,
    // and so many an item, over 131072 tokens in 16 bits, groups of 8 (us): 8 heads of 2
    // row tiles (144) 223, 206; 9 of 2 (144) 247, 232; 7 of 2 (140) 200, 190; 5 of 3
    // (150) 213, 191; 2 of 9 (144) 247, 225; 4 of 4 (144) 206, 202; 1 of 10 (150) 147,
    // 143; 1 of 13 (143) 177, 178; 1 of 17 (136, not taken) 217, 227.  Over 32768: 89,
    // 80; 94, 87; 80, 76; 83, 75; 92, 81; 80, 77; 67, 63; 74, 70; 84, 82.
    if (std::is_same<Args, TreeArgs>::value && a.batch == 1 && tiled > a.kv_heads && shares == kShares &&
        8 * tiled <= kShares && 10 * (kShares % tiled) <= kShares)
        shares = (int)(kShares / tiled * tiled);
    attend_chunk_kernel<T, FMT, Args, false>
        <<<shares, kThreads, shared_bytes<FMT, Args>(a.dim), s>>>(a, t, k_map, v_map, box, whole ? 1 : 0);
    e = cudaGetLastError();
    if (e != cudaSuccess || whole) return e;
    return launch_join(join_columns_kernel<T, FMT, kRows, Args>, a, t, shares, kRows / kJoinMany, kJoinManyThreads,
                       (size_t)join_bytes(a.dim), s);
}

template <class Args>
cudaError_t launch_any(int dtype, int format, const KvArgs& a, const Args& t, int max_new, int max_len,
                       cudaStream_t s) {
    if (dtype == (int)Bf16::kCode) {
        if (format == kKv16Bit) return launch_one<BfType, kKv16Bit>(a, t, max_new, max_len, s);
        return format == kKvInt8 ? launch_one<BfType, kKvInt8>(a, t, max_new, max_len, s)
                                 : launch_one<BfType, kKvE4m3>(a, t, max_new, max_len, s);
    }
    if (format == kKv16Bit) return launch_one<HfType, kKv16Bit>(a, t, max_new, max_len, s);
    return format == kKvInt8 ? launch_one<HfType, kKvInt8>(a, t, max_new, max_len, s)
                             : launch_one<HfType, kKvE4m3>(a, t, max_new, max_len, s);
}

}  // namespace

}  // namespace cccl
