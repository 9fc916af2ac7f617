// cccl_kv_chunk.cu -- attention of many rows a kv head (chunks of prompts) on
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
// rows of Q and write the result), 8-11 bring K and V in, 12 issues the
// products.  One block an SM: 512 columns of TMEM (S0, S1, O0, O1).
//
// The running maximum is only moved when a score exceeds it by more than 2^8
// (the accumulator is then rescaled in TMEM); any fixed reference gives the
// same quotient, and binary32 sums and 16-bit probabilities hold a factor of
// 256.  The products of one thread execute in order, so a full S also means
// that the previous O is done, and S may be written over the P that the
// product before it reads.
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
constexpr int kSlots = 4;        // K and V tiles in shared memory
constexpr int kScaleSlots = 4;   // tiles of tokens whose scales are kept
constexpr int kLoaderWarps = 4;
constexpr float kSlack = 8.f;    // base 2

// Registers of a thread: the launch's 4 x 128 a warpgroup, divided anew (two
// softmax warpgroups, the loaders, and 64 for the issuing warp's).
template <int FMT>
constexpr int kSoftmaxRegs = FMT == kKv16Bit ? 192 : 176;
template <int FMT>
constexpr int kLoaderRegs = FMT == kKv16Bit ? 64 : 96;

// TMEM columns
constexpr uint32_t kColS = 0, kColO = 256;  // S of row tile i at 128 i (P over it), O at 256 + 128 i

struct Shared {
    uint64_t q_full[2], s_full[2], p_full[2], o_full[2];
    uint64_t kv_full[kSlots], kv_free[kSlots], scale_full[kScaleSlots];
    uint64_t drained;
    uint32_t tmem;
    uint32_t stop;  // a bounded wait ran out: every role leaves
    uint64_t prefix[kMaxBatch + 1];
    alignas(16) float k_scale[kScaleSlots][kTokens];
    alignas(16) float v_scale[kScaleSlots][kTokens];
    alignas(16) uint32_t v_top[kScaleSlots][kLoaderWarps];  // the largest value scale of each warp's rows
};

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
__device__ __forceinline__ void tc_store32(uint32_t at, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,"
        "%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::CCCL_W4(r, 0),
        CCCL_W4(r, 4), CCCL_W4(r, 8), CCCL_W4(r, 12), CCCL_W4(r, 16), CCCL_W4(r, 20), CCCL_W4(r, 24), CCCL_W4(r, 28),
        "r"(at)
        : "memory");
}
__device__ __forceinline__ void tc_store16(uint32_t at, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::CCCL_W4(
            r, 0),
        CCCL_W4(r, 4), CCCL_W4(r, 8), CCCL_W4(r, 12), "r"(at)
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
// kind::f16: binary32 accumulator, M = 128, both operands of one type.
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

// A share's pieces, one after the other (every role walks them by itself).
struct Walk {
    uint64_t x, x0, x1, T;
    uint32_t share, shares;
    int32_t whole;
};
__device__ __forceinline__ bool next_piece(const KvArgs& a, const AttnArgs& t, const uint64_t* prefix, Walk& w,
                                           Piece& p) {
    while (w.x < w.x1) {
        find_item<kRows, kTokens>(a, t, prefix, w.x, p);
        const uint64_t end = p.item + (uint64_t)p.range.n;
        if (w.whole) {
            const bool before = p.item < w.x;
            w.x = end;
            if (before) continue;  // the share before does all of it
            p.from = 0;
            p.count = p.range.n;
        } else {
            p.from = (int32_t)(w.x - p.item);
            p.count = (int32_t)(min(end, w.x1) - w.x);
            w.x += (uint64_t)p.count;
        }
        return true;
    }
    return false;
}
__device__ __forceinline__ int live_rows(const AttnArgs& t, const Piece& p) {
    return (int)min((int64_t)kRows, (int64_t)p.seq.n * t.group - (int64_t)p.rt * kRows);
}

// A bounded wait of one role; false: leave (this wait or another's ran out).
struct Waiter {
    Shared* sh;
    WsHeader* ws;
    __device__ __forceinline__ bool operator()(uint64_t* bar, uint32_t parity) const {
        if (mbar_wait(bar, parity)) return true;
        record_error(ws, kStatusTimeout);
        *reinterpret_cast<volatile uint32_t*>(&sh->stop) = 1;
        return false;
    }
};

// ---------------------------------------------------------------- K and V
// Loader warp w brings rows 32 w .. 32 w + 31 of every tile.
struct TileRow {
    int64_t at, scale_at;
    bool real;
};
__device__ __forceinline__ TileRow tile_row(const KvArgs& a, const Piece& p, int32_t pos) {
    TileRow r{0, 0, false};
    if (pos >= p.range.first && pos < p.range.last) {
        r.real = slot_of(a, p.b, (uint32_t)pos, r.at, r.scale_at);
        if (!r.real) r.at = r.scale_at = 0;
    }
    r.at += (int64_t)p.kv_head * a.head_stride;
    r.scale_at += (int64_t)p.kv_head * a.s_head;
    return r;
}
// 16-bit values go straight to shared memory.
__device__ __forceinline__ void copy_tile(const KvArgs& a, const uint8_t* data, uint32_t slot, const TileRow& r,
                                          int warp, int lane, int chunks) {
    // chunks (16 bytes each) of a row: up to 16; lanes beyond them idle
    const int per_row = chunks > 8 ? 16 : 8, rows_per_pass = 32 / per_row;
    const int chunk = lane % per_row;
#pragma unroll 8
    for (int i = 0; i < 32 / rows_per_pass; ++i) {
        const int local = i * rows_per_pass + lane / per_row;
        const int64_t at = __shfl_sync(0xFFFFFFFFu, r.at, local);
        const bool real = __shfl_sync(0xFFFFFFFFu, (int)r.real, local) != 0;
        if (chunk < chunks) copy16(slot + swizzled(32 * warp + local, chunk), data + (real ? at + 16 * chunk : 0), real);
    }
}

// 8-bit codes pass through registers: a lane takes 16 codes of a row at a time
// and stores them as 16-bit values.  Lanes of a row's second half store their
// two chunks the other way round, so that a row's eight lanes meet all banks.
constexpr int kCodePasses = 8;  // 32 rows, at least 4 a pass
struct Codes {
    uint4 w[kCodePasses];
};
__device__ __forceinline__ void fetch_codes(const uint8_t* data, const TileRow& r, int lane, int chunks, Codes& c) {
    const int per_row = chunks > 4 ? 8 : 4, rows_per_pass = 32 / per_row, chunk = lane % per_row;
#pragma unroll
    for (int i = 0; i < kCodePasses; ++i) {
        c.w[i] = make_uint4(0, 0, 0, 0);
        if (i < per_row) {
            const int local = i * rows_per_pass + lane / per_row;
            const int64_t at = __shfl_sync(0xFFFFFFFFu, r.at, local);
            const bool real = __shfl_sync(0xFFFFFFFFu, (int)r.real, local) != 0;
            if (real && chunk < chunks) c.w[i] = *reinterpret_cast<const uint4*>(data + at + 16 * chunk);
        }
    }
}
template <int FMT>
__device__ __forceinline__ void store_codes(const Codes& c, uint32_t slot, int warp, int lane, int chunks) {
    const int per_row = chunks > 4 ? 8 : 4, rows_per_pass = 32 / per_row, chunk = lane % per_row;
#pragma unroll
    for (int i = 0; i < kCodePasses; ++i) {
        if (i < per_row && chunk < chunks) {
            const uint32_t row = 32 * warp + i * rows_per_pass + lane / per_row;
            const uint32_t w[4] = {c.w[i].x, c.w[i].y, c.w[i].z, c.w[i].w};
            uint32_t v[8];
#pragma unroll
            for (int k = 0; k < 4; ++k)  // in the row's order
                expand4<FMT>(FMT == kKvInt8 ? __byte_perm(w[k], 0, 0x3120) : w[k], v[2 * k], v[2 * k + 1]);
            const int second = chunk >> 2;  // which of the two goes first
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int part = k ^ second;
                const uint32_t at = slot + swizzled(row, 2 * chunk + part);
                asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(part ? v[4] : v[0]),
                             "r"(part ? v[5] : v[1]), "r"(part ? v[6] : v[2]), "r"(part ? v[7] : v[3])
                             : "memory");
            }
        }
    }
}

template <class T, int FMT>
__device__ __forceinline__ void load_role(const KvArgs& a, const AttnArgs& t, Shared* sh, uint32_t slots,
                                          uint32_t slot_bytes, Walk w) {
    const int warp = (threadIdx.x >> 5) - 8, lane = threadIdx.x & 31;
    const Waiter wait{sh, a.ws};
    const int chunks = a.dim * (FMT == kKv16Bit ? 2 : 1) / 16;
    uint32_t entry = 0, published = 0;  // K and V tiles, alternating
    Piece p;
    auto publish_to = [&](uint32_t upto) {
        fence_proxy_async_smem();
        __syncwarp();
        for (; published < upto; ++published)
            if (lane == 0) mbar_arrive(&sh->kv_full[published % kSlots]);
    };
    while (next_piece(a, t, sh->prefix, w, p)) {
        const int32_t base = (p.range.lo + p.from) * kTokens + 32 * warp + lane;
        TileRow r = tile_row(a, p, base);
        Codes codes;
        float ks = 0.f, vs = 0.f;
        if (FMT != kKv16Bit) {
            fetch_codes(a.k, r, lane, chunks, codes);
            if (r.real) ks = a.k_scale[r.scale_at], vs = a.v_scale[r.scale_at];
        }
        for (int32_t j = 0; j < p.count; ++j) {
            const TileRow here = r;
            if (j + 1 < p.count) r = tile_row(a, p, base + (j + 1) * kTokens);
#pragma unroll
            for (int side = 0; side < 2; ++side, ++entry) {
                const uint32_t s = entry % kSlots, use = entry / kSlots;
                const uint32_t slot = slots + s * slot_bytes;
                if (use > 0 && !__all_sync(0xFFFFFFFFu, mbar_test(&sh->kv_free[s], (use - 1) & 1))) {
                    // about to wait: hand over what has been brought so far
                    if (FMT == kKv16Bit) {
                        copy_wait<0>();
                        publish_to(entry);
                    }
                    if (!__all_sync(0xFFFFFFFFu, wait(&sh->kv_free[s], (use - 1) & 1))) return;
                }
                if (FMT == kKv16Bit) {
                    copy_tile(a, side ? a.v : a.k, slot, here, warp, lane, chunks);
                    copy_commit();
                    copy_wait<2>();
                    if (entry >= 2) publish_to(entry - 1);
                    continue;
                }
                // this side's codes are here; the next side's are asked for before they are worked on
                const Codes now = codes;
                if (side == 0) {
                    fetch_codes(a.v, here, lane, chunks, codes);
                    const uint32_t n = (entry / 2) % kScaleSlots;
                    sh->k_scale[n][32 * warp + lane] = ks;
                    sh->v_scale[n][32 * warp + lane] = vs;
                    const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(vs));
                    if (lane == 0) sh->v_top[n][warp] = top;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sh->scale_full[n]);
                    store_codes<FMT>(now, slot, warp, lane, chunks);
                } else {
                    ks = vs = 0.f;
                    if (j + 1 < p.count) {
                        fetch_codes(a.k, r, lane, chunks, codes);
                        if (r.real) ks = a.k_scale[r.scale_at], vs = a.v_scale[r.scale_at];
                    }
                    store_codes<FMT>(now, slot, warp, lane, chunks);
                }
                publish_to(entry + 1);
            }
        }
    }
    if (FMT == kKv16Bit) {
        copy_wait<0>();
        publish_to(entry);
    }
}

// ---------------------------------------------------------------- products
template <class M>
__device__ __forceinline__ void mma_role(const KvArgs& a, const AttnArgs& t, Shared* sh, uint32_t q_base,
                                         uint32_t slots, uint32_t slot_bytes, Walk w) {
    const Waiter wait{sh, a.ws};
    const uint32_t tmem = sh->tmem;
    const uint32_t qk = instruction(M::kHalf, kTokens, false), pv = instruction(M::kHalf, a.dim > 64 ? 128 : 64, true);
    const int steps = a.dim / 16;
    const uint32_t q_bytes = slot_bytes;
    uint32_t entry = 0;
    uint32_t q_phase[2] = {0, 0}, p_phase[2] = {0, 0};
    auto product_qk = [&](int i, uint32_t slot) {
        const uint64_t qd = operand(q_base + i * q_bytes, 16), kd = operand(slots + slot * slot_bytes, 16);
#pragma unroll 8
        for (int ks = 0; ks < steps; ++ks) {
            const uint32_t off = ((uint32_t)(ks >> 2) * kHalfBytes + (uint32_t)(ks & 3) * 32) >> 4;
            mma_ss(tmem + kColS + 128 * i, qd + off, kd + off, qk, ks > 0);
        }
        tc_commit(&sh->s_full[i]);
    };
    auto product_pv = [&](int i, uint32_t slot, bool add) {
        const uint64_t vd = operand(slots + slot * slot_bytes, kHalfBytes);
#pragma unroll
        for (int kt = 0; kt < kTokens / 16; ++kt)
            mma_ts(tmem + kColO + 128 * i, tmem + kColS + 128 * i + 8 * kt, vd + (uint32_t)(kt * 2048 >> 4), pv,
                   add || kt > 0);
    };
    Piece p;
    while (next_piece(a, t, sh->prefix, w, p)) {
        const int tiles = live_rows(t, p) > kTileRows ? 2 : 1;
        // K of the first tile
        if (!wait(&sh->kv_full[entry % kSlots], (entry / kSlots) & 1)) return;
        for (int i = 0; i < tiles; ++i) {
            if (!wait(&sh->q_full[i], q_phase[i])) return;
            q_phase[i] ^= 1;
            tc_fence_after();
            product_qk(i, entry % kSlots);
        }
        tc_commit(&sh->kv_free[entry % kSlots]);
        ++entry;
        for (int32_t j = 0; j < p.count; ++j) {
            const uint32_t v_entry = entry, k_entry = entry + 1;
            const bool more = j + 1 < p.count;
            if (!wait(&sh->kv_full[v_entry % kSlots], (v_entry / kSlots) & 1)) return;
            if (more && !wait(&sh->kv_full[k_entry % kSlots], (k_entry / kSlots) & 1)) return;
            for (int i = 0; i < tiles; ++i) {
                if (!wait(&sh->p_full[i], p_phase[i])) return;
                p_phase[i] ^= 1;
                tc_fence_after();
                product_pv(i, v_entry % kSlots, j > 0);
                if (more)
                    product_qk(i, k_entry % kSlots);
                else
                    tc_commit(&sh->o_full[i]);
            }
            tc_commit(&sh->kv_free[v_entry % kSlots]);
            if (more) tc_commit(&sh->kv_free[k_entry % kSlots]);
            entry += more ? 2 : 1;
        }
    }
}

// ---------------------------------------------------------------- softmax
// Row `row` (0..127) of row tile i of Q into shared memory; rows that do not
// exist are zeros.  flip: the sign bit when the scale is negative; zero: the
// scale is zero (every score is then 0 times the products, so are zeros').
// Returns what undoes the row's power of two (8-bit caches).
template <class T, int FMT>
__device__ __forceinline__ float bring_row(const KvArgs& a, const AttnArgs& t, const Piece& p, int i, int row,
                                           uint32_t q_tile, bool flip, bool zero) {
    const bool real = i * kTileRows + row < live_rows(t, p) && !zero;
    const RowPlace at = row_place(t, p, kRows, i * kTileRows + row);
    const uint4* src = reinterpret_cast<const uint4*>(t.q + at.token * t.q_token + (int64_t)at.head * t.q_head);
    const uint32_t sign = flip ? 0x80008000u : 0u;
    float power = 1.f;
    if (FMT != kKv16Bit && real) {
        uint32_t top = 0;
#pragma unroll 4
        for (int c = 0; c < a.dim / 8; ++c) {
            const uint4 x = src[c];
            top = vmax_u16x2(vmax_u16x2(top, x.x & 0x7FFF7FFFu), vmax_u16x2(x.y & 0x7FFF7FFFu, x.z & 0x7FFF7FFFu));
            top = vmax_u16x2(top, x.w & 0x7FFF7FFFu);
        }
        power = query_power<T>(max(top & 0xFFFFu, top >> 16));
    }
#pragma unroll 4
    for (int c = 0; c < a.dim / 8; ++c) {
        uint4 x = make_uint4(0, 0, 0, 0);
        if (real) {
            x = src[c];
            x.x ^= sign;
            x.y ^= sign;
            x.z ^= sign;
            x.w ^= sign;
            if (FMT != kKv16Bit)
                x = make_uint4(scaled_pair<T>(x.x, power), scaled_pair<T>(x.y, power), scaled_pair<T>(x.z, power),
                               scaled_pair<T>(x.w, power));
        }
        asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(q_tile + swizzled(row, c)), "r"(x.x), "r"(x.y),
                     "r"(x.z), "r"(x.w)
                     : "memory");
    }
    fence_proxy_async_smem();
    return 1.f / power;
}

template <class T, int FMT>
__device__ __forceinline__ void softmax_role(const KvArgs& a, const AttnArgs& t, Shared* sh, uint32_t q_tile, Walk w) {
    const int i = threadIdx.x / 128, row = threadIdx.x % 128, warp = row >> 5, lane = row & 31;
    const Waiter wait{sh, a.ws};
    const uint32_t tmem = sh->tmem + ((uint32_t)(32 * warp) << 16);
    const uint32_t at_s = tmem + kColS + 128 * i, at_o = tmem + kColO + 128 * i;
    const bool flip = t.scale < 0.f, zero = t.scale == 0.f;
    const float scale_base2 = (zero ? 1.f : fabsf(t.scale)) * 1.4426950408889634f;
    float next_base2 = scale_base2;
    const PartLayout parts = part_layout(a, gridDim.x, kRows);
    uint32_t s_phase = 0, o_phase = 0, tile = 0;  // tile: this block's tiles of tokens, whoever's
    const uint64_t x0 = w.x;
    bool first_piece = true;

    // the next piece that has rows for this warpgroup, with its rows of Q on their way
    Piece p;
    uint32_t skipped = 0;  // tiles of pieces without
    auto take = [&]() -> bool {
        for (;;) {
            if (!next_piece(a, t, sh->prefix, w, p)) return false;
            if (first_piece && !w.whole && threadIdx.x == 0) {
                parts.cuts[w.share] = cut_of<kRows, kTokens>(p, x0, w.T, w.share, w.shares);
            }
            first_piece = false;
            if (live_rows(t, p) > i * kTileRows) break;
            skipped += (uint32_t)p.count;
        }
        next_base2 = scale_base2 * bring_row<T, FMT>(a, t, p, i, row, q_tile, flip, zero);
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh->q_full[i]);
        return true;
    };
    bool have = take();
    if (first_piece && !w.whole && threadIdx.x == 0) parts.cuts[w.share].last = -1;
    while (have) {
        const Piece cur = p;
        const float to_base2 = next_base2;
        const bool is_row = i * kTileRows + row < live_rows(t, cur);
        const RowPlace at = row_place(t, cur, kRows, i * kTileRows + row);
        int32_t first = 0, last = 0;
        if (is_row) visible_range(t, cur.seq.len, at.pos, first, last);
        float m = -INFINITY, l = 0.f;
        int32_t base = (cur.range.lo + cur.from) * kTokens;
        tile += skipped;
        skipped = 0;
        for (int32_t j = 0; j < cur.count; ++j, ++tile, base += kTokens) {
            if (!__all_sync(0xFFFFFFFFu, wait(&sh->s_full[i], s_phase))) return;
            s_phase ^= 1;
            tc_fence_after();
            uint32_t s[kTokens];
#pragma unroll
            for (int c = 0; c < kTokens; c += 32) tc_load32(at_s + c, s + c);
            tc_wait_load();
            const uint32_t scale_slot = tile % kScaleSlots;
            if (FMT != kKv16Bit) {
                if (!__all_sync(0xFFFFFFFFu, wait(&sh->scale_full[scale_slot], (tile / kScaleSlots) & 1))) return;
#pragma unroll
                for (int c = 0; c < kTokens; c += 4) {
                    const float4 f = *reinterpret_cast<const float4*>(&sh->k_scale[scale_slot][c]);
                    const float2 x = mul2(make_float2(__uint_as_float(s[c]), __uint_as_float(s[c + 1])),
                                          make_float2(f.x, f.y));
                    const float2 y = mul2(make_float2(__uint_as_float(s[c + 2]), __uint_as_float(s[c + 3])),
                                          make_float2(f.z, f.w));
                    s[c] = __float_as_uint(x.x);
                    s[c + 1] = __float_as_uint(x.y);
                    s[c + 2] = __float_as_uint(y.x);
                    s[c + 3] = __float_as_uint(y.y);
                }
            }
            if (base < first || base + kTokens > last) {
                const int32_t lo = first - base, hi = last - base;  // visible columns lo .. hi - 1
#pragma unroll
                for (int c = 0; c < kTokens; ++c)
                    if (c < lo || c >= hi) s[c] = 0xFF800000u;
            }
            float top0 = -INFINITY, top1 = -INFINITY;
#pragma unroll
            for (int c = 0; c < kTokens; c += 4) {
                top0 = max3(top0, __uint_as_float(s[c]), __uint_as_float(s[c + 1]));
                top1 = max3(top1, __uint_as_float(s[c + 2]), __uint_as_float(s[c + 3]));
            }
            float top = fmaxf(top0, top1) * to_base2;
            if (FMT != kKv16Bit) {
                const uint4 v = *reinterpret_cast<const uint4*>(sh->v_top[scale_slot]);
                top += scale_exponent(max(max(v.x, v.y), max(v.z, v.w)));
            }
            if (j == 0) {
                m = top;
            } else if (__any_sync(0xFFFFFFFFu, top > m + kSlack)) {
                const float to = fmaxf(m, top);
                const float f = to == -INFINITY ? 1.f : exp2_fast(m - to);
                m = to;
                l *= f;
                for (int c = 0; c < a.dim; c += 16) {
                    uint32_t o[16];
                    tc_load16(at_o + c, o);
                    tc_wait_load();
#pragma unroll
                    for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                    tc_store16(at_o + c, o);
                }
            }
            const float from = m == -INFINITY ? 0.f : -m;
            const float2 scale2 = make_float2(to_base2, to_base2), from2 = make_float2(from, from);
            float2 sum0 = make_float2(0.f, 0.f), sum1 = make_float2(0.f, 0.f);
            uint32_t pr[kTokens / 2];
#pragma unroll
            for (int c = 0; c < kTokens; c += 4) {
                float2 x = fma2(make_float2(__uint_as_float(s[c]), __uint_as_float(s[c + 1])), scale2, from2);
                float2 y = fma2(make_float2(__uint_as_float(s[c + 2]), __uint_as_float(s[c + 3])), scale2, from2);
                x.x = exp2_fast(x.x);
                x.y = exp2_fast(x.y);
                y.x = exp2_fast(y.x);
                y.y = exp2_fast(y.y);
                sum0 = add2(sum0, x);
                sum1 = add2(sum1, y);
                if (FMT != kKv16Bit) {
                    const float4 f = *reinterpret_cast<const float4*>(&sh->v_scale[scale_slot][c]);
                    x = mul2(x, make_float2(f.x, f.y));
                    y = mul2(y, make_float2(f.z, f.w));
                }
                pr[c / 2] = pack<Operand<T, FMT>>(x.x, x.y);
                pr[c / 2 + 1] = pack<Operand<T, FMT>>(y.x, y.y);
                if (c % 64 == 60) tc_store32(at_s + (c / 64) * 32, pr + (c / 64) * 32);
            }
            sum0 = add2(sum0, sum1);
            l += sum0.x + sum0.y;
            tc_wait_store();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh->p_full[i]);
        }
        // the next item's rows of Q may come now: the last S is done, so is every product with these
        have = take();
        if (!__all_sync(0xFFFFFFFFu, wait(&sh->o_full[i], o_phase))) return;
        o_phase ^= 1;
        tc_fence_after();
        const bool full = cur.count == cur.range.n;
        const int tile_row = i * kTileRows + row;
        bool odd = false;
        if (full) {
            const bool none = last <= first;
            const float inv = none ? 0.f : 1.f / l;
            uint8_t* dst = t.out + at.token * t.o_token + (int64_t)at.head * t.o_head;
            for (int c = 0; c < a.dim; c += 16) {
                uint32_t o[16];
                tc_load16(at_o + c, o);
                tc_wait_load();
                uint32_t y[8];
#pragma unroll
                for (int k = 0; k < 16; k += 2) {
                    const float u = none ? 0.f : __uint_as_float(o[k]) * inv;
                    const float v = none ? 0.f : __uint_as_float(o[k + 1]) * inv;
                    odd |= !(fabsf(u) <= 3.402823466e+38f) || !(fabsf(v) <= 3.402823466e+38f);
                    y[k / 2] = pack<T>(u, v);
                }
                if (is_row) {
                    *reinterpret_cast<uint4*>(dst + 2 * c) = make_uint4(y[0], y[1], y[2], y[3]);
                    *reinterpret_cast<uint4*>(dst + 2 * c + 16) = make_uint4(y[4], y[5], y[6], y[7]);
                }
            }
            if (is_row && t.lse != nullptr)
                t.lse[at.token * t.q_heads + at.head] = none ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
            for (uint32_t todo = __ballot_sync(0xFFFFFFFFu, odd && is_row); todo != 0; todo &= todo - 1) {
                __syncwarp();
                fix_row<T, FMT>(a, t, cur, kRows, i * kTileRows + 32 * warp + __ffs(todo) - 1);
            }
        } else {
            const int which = cur.from > 0 ? 0 : 1;
            float* dst = parts.acc(w.share, which) + (size_t)tile_row * a.dim;
            for (int c = 0; c < a.dim; c += 16) {
                uint32_t o[16];
                tc_load16(at_o + c, o);
                tc_wait_load();
                if (is_row) {
#pragma unroll
                    for (int k = 0; k < 16; k += 4)
                        *reinterpret_cast<uint4*>(dst + c + k) = make_uint4(o[k], o[k + 1], o[k + 2], o[k + 3]);
                }
            }
            if (is_row) {
                parts.stats(w.share, which)[tile_row] = m;
                parts.stats(w.share, which)[kRows + tile_row] = l;
            }
        }
        tc_fence_before();
    }
}

template <class T, int FMT>
__global__ void __launch_bounds__(kThreads, 1)
    attend_chunk_kernel(const __grid_constant__ KvArgs a, const __grid_constant__ AttnArgs t, uint32_t min_tiles,
                        int whole_items) {
    extern __shared__ uint8_t raw[];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    // tiles at 1024-byte boundaries (the swizzle's period): Q0, Q1, the K and V slots, then the rest
    const uint32_t base = (smem_addr(raw) + 1023) & ~1023u;
    const uint32_t tile_bytes = (a.dim > 64 ? 2 : 1) * kHalfBytes;
    Shared* sh = reinterpret_cast<Shared*>(raw + (base - smem_addr(raw)) + (2 + kSlots) * tile_bytes);
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
        for (int i = 0; i < kSlots; ++i) {
            mbar_init(&sh->kv_full[i], kLoaderWarps);
            mbar_init(&sh->kv_free[i], 1);
        }
        for (int i = 0; i < kScaleSlots; ++i) mbar_init(&sh->scale_full[i], kLoaderWarps);
        mbar_init(&sh->drained, 1);
        sh->stop = 0;
        fence_mbar_init();
    }
    build_prefix<kRows, kTokens>(a, t, sh->prefix);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint64_t all = sh->prefix[a.batch];
    Walk w;
    w.T = all;
    w.shares = (uint32_t)min((uint64_t)gridDim.x, max((all + min_tiles - 1) / min_tiles, (uint64_t)1));
    w.share = blockIdx.x;
    w.x0 = w.x = w.share < w.shares ? share_start(all, w.share, w.shares) : all;
    w.x1 = w.share < w.shares ? share_start(all, w.share + 1, w.shares) : all;
    w.whole = whole_items;
    const uint32_t slots = base + 2 * tile_bytes;
    if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs<FMT>));
        softmax_role<T, FMT>(a, t, sh, base + (warp / 4) * tile_bytes, w);
    } else if (warp < 12) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kLoaderRegs<FMT>));
        load_role<T, FMT>(a, t, sh, slots, tile_bytes, w);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
        if (threadIdx.x == 12 * 32) {
            mma_role<Operand<T, FMT>>(a, t, sh, base, slots, tile_bytes, w);
            tc_commit(&sh->drained);
            if (!mbar_wait(&sh->drained, 0)) record_error(a.ws, kStatusTimeout);
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(sh->tmem) : "memory");
}

size_t shared_bytes(int dim) { return 1024 + (size_t)(2 + kSlots) * (dim > 64 ? 2 : 1) * kHalfBytes + sizeof(Shared); }

template <class T, int FMT>
cudaError_t launch_one(const KvArgs& a, const AttnArgs& t, bool whole, uint32_t min_tiles, cudaStream_t s) {
    static PerDeviceOnce once;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    e = once.run(dev, [] {
        return cudaFuncSetAttribute(attend_chunk_kernel<T, FMT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    (int)shared_bytes(128));
    });
    if (e != cudaSuccess) return e;
    attend_chunk_kernel<T, FMT><<<kShares, kThreads, shared_bytes(a.dim), s>>>(a, t, min_tiles, whole ? 1 : 0);
    e = cudaGetLastError();
    if (e != cudaSuccess || whole) return e;
    return launch_join<T, FMT, kRows>(a, t, kShares, s);
}

}  // namespace

size_t kv_chunk_scratch(int dim) { return part_bytes(kShares, kRows, dim); }

cudaError_t launch_kv_chunk(int dtype, int format, const KvArgs& a, const AttnArgs& t, int max_len, cudaStream_t s) {
    const bool whole = max_len <= kTokens;
    const uint32_t min_tiles = 1;
    if (dtype == (int)Bf16::kCode) {
        if (format == kKv16Bit) return launch_one<BfType, kKv16Bit>(a, t, whole, min_tiles, s);
        return format == kKvInt8 ? launch_one<BfType, kKvInt8>(a, t, whole, min_tiles, s)
                                 : launch_one<BfType, kKvE4m3>(a, t, whole, min_tiles, s);
    }
    if (format == kKv16Bit) return launch_one<HfType, kKv16Bit>(a, t, whole, min_tiles, s);
    return format == kKvInt8 ? launch_one<HfType, kKvInt8>(a, t, whole, min_tiles, s)
                             : launch_one<HfType, kKvE4m3>(a, t, whole, min_tiles, s);
}

}  // namespace cccl
