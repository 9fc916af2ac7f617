// cccl_kv_tokens.cuh -- attention of few rows a kv head (single tokens, short
// drafts): the cache is read once and everything else is small, so the kernel
// is built around the loads.
//
// An item is up to 8 or 16 rows (new tokens x the query heads that share a kv
// head).  Each of a block's four warps takes TS consecutive cached tokens of
// every tile and runs on its own: its ring of stages filled by its own 16-byte
// asynchronous copies (page lookups one stage ahead of the copies), products by
// mma.sync, its own running maximum, sum and accumulator in registers.  The
// four meet once, at the end of an item: with m the largest of their maxima,
//   out = sum_i 2^(m_i - m) acc_i / sum_i 2^(m_i - m) sum_i .
// The same joins the parts of an item that several blocks share, by a cluster's
// shared memory (few, short items) or by a second kernel (any).
//
// What bounds it: the loads.  32 tokens over 32 x 4096 cached (8 kv heads of
// 128, groups of 4, 16-bit): 88 to 93 us, 5.8 to 6.1 TB/s, DRAM 75 % busy under the
// profiler; INT8, 16 x 16384: 106 to 112 us, 4.9 to 5.2 TB/s, DRAM 65 % and 56 % of
// the issue slots taken, by the codes' way to fp16; one token over 131077 of E4M3, whose codes take fewer
// instructions: 57 us under the profiler, DRAM 62 %, 44 % of the issue slots, and
// 11 more for joining 57 parts.  Three blocks an SM, each with 64 KB of rings; four
// spill (INT8: 299 us against 264).  Short calls are bound by the launch, the first
// page lookups and the joining: one token over 517: 7.1 us.
//
// Both products are taken transposed, S' = K Q' and O' = V' P', so that tokens
// and channels fill the instruction's 16 and the rows its 8: a tile with the
// rows as the 16 would be mostly padding, twice the instructions and twice the
// registers.  tcgen05 is not used here: its M of 128 could be the tokens, but
// the softmax would then run across threads and every tile would pay the way
// through TMEM; the tensor work is a small part of the time.
//
// Precision: products of 16-bit values are exact and summed in binary32.  A
// probability enters the second product as the sum of two 16-bit values (high
// part and remainder): 16 bits of it with bf16, 22 with fp16 (see kLower), far
// more than the result keeps.  8-bit codes
// are exact in fp16; the key's scale multiplies the score and the value's scale
// the probability, both in binary32.
#pragma once

#include <algorithm>
#include <type_traits>

#include "cccl_kv.cuh"
#include "cccl_kv_launch.h"
#include "cccl_kv_schedule.cuh"
#include "cccl_launch.h"

namespace cccl {

namespace {

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kSms = 152;

__device__ __forceinline__ void ldsm4(uint32_t a, uint32_t* r) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a));
}
__device__ __forceinline__ void ldsm4_trans(uint32_t a, uint32_t* r) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a));
}
__device__ __forceinline__ uint4 lds16(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}
__device__ __forceinline__ float lds4(uint32_t a) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a));
    return v;
}
__device__ __forceinline__ uint2 lds8(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
    return v;
}
template <class T>
__device__ __forceinline__ void mma16816(float* d, const uint32_t* a, uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma16816<BfType>(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma16816<HfType>(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// (hi, lo) with x ~ hi + lo in two 16-bit values each: two probabilities at a time
template <class T>
__device__ __forceinline__ void split_pair(float x, float y, uint32_t& hi, uint32_t& lo) {
    hi = round_pair<T>(x, y);
    lo = round_pair<T>(x - T::load((uint16_t)(hi & 0xFFFFu)), y - T::load((uint16_t)(hi >> 16)));
}

// [8][8] 16-bit values across the warp, two a lane: transposed.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// Sizes of the instance for values of T in format FMT, heads of up to DP and
// items of 8 NR rows.
template <class T_, int FMT_, int DP_, int NR_, class Args_>
struct Shape {
    using T = T_;
    using Args = Args_;  // which rows see which keys
    using M = typename std::conditional<FMT_ == kKv16Bit, T_, HfType>::type;  // the products' operands
    static constexpr int FMT = FMT_, DP = DP_, NR = NR_;
    static constexpr int kRows = 8 * NR;
    // The reference lies this much (base 2) below the row's maximum.  fp16 ends at
    // 2^-24: the largest probability is made 2^14 (times a value's scale, at most
    // 2^15), so that those down to 2^-28 of it keep 22 bits in their two parts and
    // none is off by more than 2^-39 of it.  bf16 has binary32's range.
    static constexpr float kLower = M::kHalf ? 14.f : 0.f;
    static constexpr int kElem = FMT == kKv16Bit ? 2 : 1;
    static constexpr int kRowBytes = DP * kElem;                      // 64, 128 or 256
    static constexpr int kTokens = kRowBytes == 256 ? 16 : 32;        // tokens of a warp's stage
    static constexpr int kTile = kWarps * kTokens;                    // tokens of a block's tile
    static constexpr int kSide = kTokens * kRowBytes;                 // bytes of K (or V) in a stage
    static constexpr int kScaleBytes = FMT == kKv16Bit ? 0 : 8 * kTokens;
    static constexpr int kStage = 2 * kSide + kScaleBytes;
    static constexpr int kStages = kStage > 4096 + 512 ? 2 : 4;
    static constexpr int kRing = kStages * kStage;                    // bytes of a warp's ring
    static constexpr int kMerge = kWarps * kRows * (DP + 4) * 4;      // accumulators at the end of an item
    static constexpr int kBlocksPerSm = 3;
    static constexpr int kShares = kSms * kBlocksPerSm;
    static constexpr int kGather = kRows * (DP + 4) * 4;              // a block's own, for its cluster
    static constexpr int kSmem = kWarps * kRing > kMerge + kGather ? kWarps * kRing : kMerge + kGather;
};

// Where 16-byte chunk c of row r lies in a stage's K or V.  The swizzles spread
// what one quarter-warp reads together over all banks: eight rows of one chunk
// (ldmatrix), or rows r, r + 1 of four chunks (K codes), or rows 0, 2, 4, 6 of
// two chunks (V codes; two-way conflicts remain at 64-byte rows).
template <class S, bool V>
__device__ __forceinline__ uint32_t chunk_at(uint32_t r, uint32_t c) {
    if (S::FMT == kKv16Bit) return r * S::kRowBytes + ((c ^ (r & 7)) << 4);
    if (V) return r * S::kRowBytes + ((c ^ (((r >> 1) << 1) & (S::kRowBytes / 16 - 1))) << 4);
    if (S::kRowBytes == 128) return r * S::kRowBytes + ((c ^ ((r & 1) << 2)) << 4);
    return r * S::kRowBytes + (c << 4);
}

// Where row r of a stage lies in the cache (lane r knows).
struct RowAt {
    int64_t at, scale_at;
    bool real;  // false: outside what the item sees, or in no page of the cache
};
template <class S>
__device__ __forceinline__ RowAt look_up(const KvArgs& a, const Piece& p, int32_t base) {
    const int32_t pos = base + (int)(threadIdx.x & 31);
    RowAt r{0, 0, false};
    if ((int)(threadIdx.x & 31) < S::kTokens && pos >= p.range.first && pos < p.range.last) {
        r.real = slot_of(a, p.b, (uint32_t)pos, r.at, r.scale_at);
        if (!r.real) r.at = r.scale_at = 0;
    }
    r.at += (int64_t)p.kv_head * a.head_stride;
    r.scale_at += (int64_t)p.kv_head * a.s_head;
    return r;
}
// This warp's copies of one stage; rows that are not real become zeros.
template <class S>
__device__ __forceinline__ void issue_stage(const KvArgs& a, uint32_t stage, const RowAt& r) {
    const int lane = threadIdx.x & 31;
    constexpr int kChunks = S::kRowBytes / 16, kPerPass = 32 / kChunks;
    const int chunk = lane % kChunks;
    const bool inside = chunk * 16 < a.dim * S::kElem;
#pragma unroll
    for (int i = 0; i < S::kTokens / kPerPass; ++i) {
        const int row = i * kPerPass + lane / kChunks;
        const int64_t at = __shfl_sync(0xFFFFFFFFu, r.at, row);
        const bool real = __shfl_sync(0xFFFFFFFFu, (int)r.real, row) != 0 && inside;
        const int64_t off = real ? at + chunk * 16 : 0;
        copy16(stage + chunk_at<S, false>(row, chunk), a.k + off, real);
        copy16(stage + S::kSide + chunk_at<S, true>(row, chunk), a.v + off, real);
    }
    if (S::FMT != kKv16Bit && lane < S::kTokens) {
        copy4(stage + 2 * S::kSide + 4 * lane, a.k_scale + r.scale_at, r.real);
        copy4(stage + 2 * S::kSide + 4 * S::kTokens + 4 * lane, a.v_scale + r.scale_at, r.real);
    }
}

// The query fragments: lane (g, c) holds channels of row 8 nr + g (zeros where
// there is no such row), 16-bit caches 16 ks + 2 c, + 1 and + 8, + 9; 8-bit
// caches, whose lanes read 16 codes in a row, 64 (ks / 4) + 16 c + 4 (ks % 4)
// .. + 3.  inverse[nr]: what undoes the row's power of two.
template <class S>
__device__ __forceinline__ void load_queries(const KvArgs& a, const AttnArgs& t, const Piece& p,
                                             uint32_t (*q)[S::DP / 16][2], float* inverse) {
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const int live = live_rows<S::kRows>(t, p);
#pragma unroll
    for (int nr = 0; nr < S::NR; ++nr) {
        const bool real = g + 8 * nr < live;
        const RowPlace at = row_place(t, p, S::kRows, real ? g + 8 * nr : 0);
        const uint8_t* src = t.q + at.token * t.q_token + (int64_t)at.head * t.q_head;
#pragma unroll
        for (int ks = 0; ks < S::DP / 16; ++ks) {
            uint32_t lo = 0, hi = 0;
            if (S::FMT == kKv16Bit) {
                if (real && 16 * ks < a.dim) {
                    lo = *reinterpret_cast<const uint32_t*>(src + 2 * (16 * ks + 2 * c));
                    hi = *reinterpret_cast<const uint32_t*>(src + 2 * (16 * ks + 2 * c + 8));
                }
            } else {
                const int d = 64 * (ks / 4) + 16 * c + 4 * (ks % 4);
                uint2 w = make_uint2(0, 0);
                if (real && d < a.dim) w = *reinterpret_cast<const uint2*>(src + 2 * d);
                lo = w.x;
                hi = w.y;
            }
            q[nr][ks][0] = lo;
            q[nr][ks][1] = hi;
        }
        inverse[nr] = 1.f;
        if (S::FMT != kKv16Bit) {
            uint32_t top = 0;
#pragma unroll
            for (int ks = 0; ks < S::DP / 16; ++ks) {
                top = vmax_u16x2(top, q[nr][ks][0] & 0x7FFF7FFFu);
                top = vmax_u16x2(top, q[nr][ks][1] & 0x7FFF7FFFu);
            }
            top = max(top & 0xFFFFu, top >> 16);
            top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
            top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
            const float power = query_power<typename S::T>(top);
            inverse[nr] = 1.f / power;
#pragma unroll
            for (int ks = 0; ks < S::DP / 16; ++ks) {
                const uint32_t x = scaled_pair<typename S::T>(q[nr][ks][0], power);
                const uint32_t y = scaled_pair<typename S::T>(q[nr][ks][1], power);
                q[nr][ks][0] = S::FMT == kKvE4m3 ? x : __byte_perm(x, y, 0x5410);
                q[nr][ks][1] = S::FMT == kKvE4m3 ? y : __byte_perm(x, y, 0x7632);
            }
        }
    }
}

// Scores of the stage's tokens before any scale: lane (g, c) holds tokens
// 16 mt + g and + 8, rows 8 nr + 2 c and + 1.
template <class S>
__device__ __forceinline__ void scores(uint32_t stage, const uint32_t (*q)[S::DP / 16][2], float (*s)[S::NR][4]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int mt = 0; mt < S::kTokens / 16; ++mt) {
#pragma unroll
        for (int nr = 0; nr < S::NR; ++nr)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[mt][nr][i] = 0.f;
        if (S::FMT == kKv16Bit) {
#pragma unroll
            for (int ks = 0; ks < S::DP / 16; ++ks) {
                uint32_t k[4];
                ldsm4(stage + chunk_at<S, false>(16 * mt + (lane & 15), 2 * ks + (lane >> 4)), k);
#pragma unroll
                for (int nr = 0; nr < S::NR; ++nr) mma16816<typename S::M>(s[mt][nr], k, q[nr][ks][0], q[nr][ks][1]);
            }
        } else {
#pragma unroll
            for (int h = 0; h < S::DP / 64; ++h) {
                const uint4 x = lds16(stage + chunk_at<S, false>(16 * mt + (lane >> 2), 4 * h + (lane & 3)));
                const uint4 y = lds16(stage + chunk_at<S, false>(16 * mt + 8 + (lane >> 2), 4 * h + (lane & 3)));
                const uint32_t w[4] = {x.x, x.y, x.z, x.w}, u[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint32_t k[4];
                    expand4<S::FMT>(w[j], k[0], k[2]);
                    expand4<S::FMT>(u[j], k[1], k[3]);
#pragma unroll
                    for (int nr = 0; nr < S::NR; ++nr)
                        mma16816<typename S::M>(s[mt][nr], k, q[nr][4 * h + j][0], q[nr][4 * h + j][1]);
                }
            }
        }
    }
}

// acc += V' P' over the stage's tokens; p as the fragments of its two parts.
template <class S>
__device__ __forceinline__ void values(uint32_t stage, const uint32_t (*hi)[S::NR][2], const uint32_t (*lo)[S::NR][2],
                                       float (*acc)[S::NR][4]) {
    const int lane = threadIdx.x & 31;
    const uint32_t v = stage + S::kSide;
#pragma unroll
    for (int kt = 0; kt < S::kTokens / 16; ++kt) {
        if (S::FMT == kKv16Bit) {
#pragma unroll
            for (int j = 0; j < S::DP / 16; ++j) {
                uint32_t x[4];
                ldsm4_trans(v + chunk_at<S, true>(16 * kt + (lane & 7) + ((lane >> 4) << 3), 2 * j + ((lane >> 3) & 1)),
                            x);
#pragma unroll
                for (int nr = 0; nr < S::NR; ++nr) {
                    mma16816<typename S::M>(acc[j][nr], x, hi[kt][nr][0], hi[kt][nr][1]);
                    mma16816<typename S::M>(acc[j][nr], x, lo[kt][nr][0], lo[kt][nr][1]);
                }
            }
        } else {
            // lane (g, c): tokens 2c, 2c + 1, 2c + 8, 2c + 9, DP / 8 values from g DP / 8 on
            const int g = lane >> 2, c = lane & 3;
            uint32_t w[4][S::DP / 32];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t row = 16 * kt + 2 * c + (i & 1) + 8 * (i >> 1);
                if (S::DP == 128) {
                    const uint4 x = lds16(v + chunk_at<S, true>(row, g));
                    w[i][0] = x.x;
                    w[i][1] = x.y;
                    w[i][S::DP / 32 - 2] = x.z;
                    w[i][S::DP / 32 - 1] = x.w;
                } else {
                    const uint2 x = lds8(v + chunk_at<S, true>(row, g >> 1) + 8 * (g & 1));
                    w[i][0] = x.x;
                    w[i][1] = x.y;
                }
            }
            // pairs of tokens at one channel: the byte order that expand4 pairs up
            constexpr uint32_t kFirst = S::FMT == kKvE4m3 ? 0x5140 : 0x5410;
            constexpr uint32_t kSecond = S::FMT == kKvE4m3 ? 0x7362 : 0x7632;
#pragma unroll
            for (int j = 0; j < S::DP / 32; ++j) {
                uint32_t x[2][4];
                expand4<S::FMT>(__byte_perm(w[0][j], w[1][j], kFirst), x[0][0], x[0][1]);
                expand4<S::FMT>(__byte_perm(w[2][j], w[3][j], kFirst), x[0][2], x[0][3]);
                expand4<S::FMT>(__byte_perm(w[0][j], w[1][j], kSecond), x[1][0], x[1][1]);
                expand4<S::FMT>(__byte_perm(w[2][j], w[3][j], kSecond), x[1][2], x[1][3]);
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int nr = 0; nr < S::NR; ++nr) {
                        mma16816<typename S::M>(acc[2 * j + i][nr], x[i], hi[kt][nr][0], hi[kt][nr][1]);
                        mma16816<typename S::M>(acc[2 * j + i][nr], x[i], lo[kt][nr][0], lo[kt][nr][1]);
                    }
            }
        }
    }
}
// Channel of accumulator tile j, lane group g, half h (element pairs 0, 1 or 2, 3).
template <class S>
__device__ __forceinline__ int channel(int j, int g, int h) {
    return S::FMT == kKv16Bit ? 16 * j + g + 8 * h : g * (S::DP / 8) + 2 * j + h;
}

// What a lane carries through an item: rows 8 nr + 2 c + i.
template <class S>
struct Running {
    float m[S::NR][2], l[S::NR][2];  // reference (base 2) of the row; this lane's part of the sum
    float acc[S::DP / 16][S::NR][4];
};

// One stage: scores, the softmax's step, values.  base: the stage's first
// token.  to_base2: the factor of each row's products.
template <class S>
__device__ __forceinline__ void step(const typename S::Args& t, const Piece& p, uint32_t stage, int32_t base,
                                     const uint32_t (*q)[S::DP / 16][2], const int32_t (*first)[2],
                                     const int32_t (*last)[2], bool whole_stage, const float (*to_base2)[2],
                                     Running<S>& st) {
    const int lane = threadIdx.x & 31, g = lane >> 2;
    constexpr int MT = S::kTokens / 16;
    float s[MT][S::NR][4];
    scores<S>(stage, q, s);
    float vscale[MT][2], vlog[MT][2];
    if (S::FMT != kKv16Bit) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t at = stage + 2 * S::kSide + 4 * (16 * mt + 8 * h + g);
                const float ks = lds4(at);
                vscale[mt][h] = lds4(at + 4 * S::kTokens);
                vlog[mt][h] = scale_log2(scale_bits(vscale[mt][h]), S::kLower);
#pragma unroll
                for (int nr = 0; nr < S::NR; ++nr) {
                    s[mt][nr][2 * h] *= ks;
                    s[mt][nr][2 * h + 1] *= ks;
                }
            }
    }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int nr = 0; nr < S::NR; ++nr)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[mt][nr][i] *= to_base2[nr][i & 1];
    if (!whole_stage) {  // some row of the item does not see all of it
#pragma unroll
        for (int nr = 0; nr < S::NR; ++nr)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                // rows that see nothing may have no place in the packed tensors
                uint32_t seen = ~0u;
                if (first[nr][r] < last[nr][r])
                    seen = seen_32(t, p.seq, row_place(t, p, S::kRows, 8 * nr + 2 * (lane & 3) + r).token, base);
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int32_t at = 16 * mt + 8 * h + g, j = base + at;
                        if (j < first[nr][r] || j >= last[nr][r] || (seen >> at & 1u) == 0)
                            s[mt][nr][2 * h + r] = -INFINITY;
                    }
            }
    }
    uint32_t hi[MT][S::NR][2], lo[MT][S::NR][2];
    float keep[S::NR][2];
    bool moved = false;
#pragma unroll
    for (int nr = 0; nr < S::NR; ++nr)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float m = -INFINITY;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    m = fmaxf(m, s[mt][nr][2 * h + i] + (S::FMT != kKv16Bit ? vlog[mt][h] : 0.f));
            m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 4));
            m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 8));
            m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 16));
            m = fmaxf(st.m[nr][i], S::FMT != kKv16Bit ? m : m - S::kLower);
            moved |= m != st.m[nr][i];
            const float from = m == -INFINITY ? 0.f : m;  // nothing seen so far: every term is 0
            keep[nr][i] = exp2_fast(st.m[nr][i] - from);
            st.m[nr][i] = m;
            float sum = 0.f;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float x = exp2_fast(s[mt][nr][2 * h + i] - from);
                    sum += x;
                    if (S::FMT != kKv16Bit) x *= vscale[mt][h];
                    s[mt][nr][2 * h + i] = x;
                }
            st.l[nr][i] = st.l[nr][i] * keep[nr][i] + sum;
        }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int nr = 0; nr < S::NR; ++nr)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t x, y;
                split_pair<typename S::M>(s[mt][nr][2 * h], s[mt][nr][2 * h + 1], x, y);
                hi[mt][nr][h] = transpose8x8(x);
                lo[mt][nr][h] = transpose8x8(y);
            }
    if (__any_sync(0xFFFFFFFFu, moved)) {
#pragma unroll
        for (int j = 0; j < S::DP / 16; ++j)
#pragma unroll
            for (int nr = 0; nr < S::NR; ++nr)
#pragma unroll
                for (int i = 0; i < 4; ++i) st.acc[j][nr][i] *= keep[nr][i & 1];
    }
    values<S>(stage, hi, lo, st.acc);
}

constexpr int kCluster = 8;  // at most

// how: whether items are left whole; with CLUSTERS (whole, then) the number of
// blocks that share every item of their cluster's share: each takes that part of
// its tiles, and they put the parts together through each other's shared memory,
// in the blocks' order.  (Kernels of their own: as one with the others they cost
// those 2 %.)
template <class S, bool CLUSTERS>
__global__ void __launch_bounds__(kThreads, S::kBlocksPerSm)
    attend_tokens_kernel(const __grid_constant__ KvArgs a, const __grid_constant__ typename S::Args t, int how) {
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint32_t prefix[kMaxBatch + 1];
    __shared__ float stats[2][kWarps][S::kRows];
    __shared__ float gathered[2][S::kRows];
    __shared__ uint32_t odd_rows;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    build_prefix<S::kRows, S::kTile>(a, t, prefix);
    const int whole_items = CLUSTERS ? 1 : how, cluster = CLUSTERS ? how : 1;
    const uint32_t rank = CLUSTERS ? cluster_rank() : 0;
    Walk w = make_walk(prefix[a.batch], blockIdx.x / cluster, gridDim.x / cluster, whole_items);
    const PartLayout parts = part_layout(a, (int)gridDim.x, S::kRows);
    if (!whole_items && w.x >= w.x1 && threadIdx.x == 0) parts.cuts[w.share].last = -1;
    const float to_base2 = t.scale * 1.4426950408889634f;
    const uint32_t ring = smem_addr(smem) + warp * S::kRing;
    Piece p;
    for (bool begin = true; next_piece<S::kRows, S::kTile>(a, t, prefix, w, p); begin = false) {
        if (begin && !whole_items && threadIdx.x == 0)
            parts.cuts[w.share] = cut_of<S::kRows, S::kTile>(p, w.line, w.share);
        const bool full = p.count == p.range.n;
        const int which = p.from > 0 ? 0 : 1;
        const int32_t from = CLUSTERS ? p.from + (int32_t)rank * p.count / cluster : p.from;
        const int32_t count = CLUSTERS ? p.from + (int32_t)(rank + 1) * p.count / cluster - from : p.count;
        const int32_t live = live_rows<S::kRows>(t, p);
        int32_t first[S::NR][2], last[S::NR][2], all_from = 0, all_to = 0x7FFFFFFF;
#pragma unroll
        for (int nr = 0; nr < S::NR; ++nr)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                first[nr][i] = last[nr][i] = 0;
                if (8 * nr + 2 * c + i < live) {
                    const RowPlace at = row_place(t, p, S::kRows, 8 * nr + 2 * c + i);
                    search_range(t, p.seq, at.token, at.pos, first[nr][i], last[nr][i]);
                    all_from = max(all_from, first[nr][i]);
                    all_to = min(all_to, gapless_below(t, p.seq, last[nr][i]));
                }
            }
        // tokens that every row sees: all_from .. all_to - 1
        all_from = __reduce_max_sync(0xFFFFFFFFu, all_from);
        all_to = __reduce_min_sync(0xFFFFFFFFu, all_to);
        uint32_t q[S::NR][S::DP / 16][2];
        float inverse[S::NR], factor[S::NR][2];
        load_queries<S>(a, t, p, q, inverse);
#pragma unroll
        for (int nr = 0; nr < S::NR; ++nr)
#pragma unroll
            for (int i = 0; i < 2; ++i)
                factor[nr][i] = to_base2 * __shfl_sync(0xFFFFFFFFu, inverse[nr], 4 * (2 * c + i));
        Running<S> st;
#pragma unroll
        for (int nr = 0; nr < S::NR; ++nr) {
#pragma unroll
            for (int i = 0; i < 2; ++i) st.m[nr][i] = -INFINITY, st.l[nr][i] = 0.f;
#pragma unroll
            for (int j = 0; j < S::DP / 16; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) st.acc[j][nr][i] = 0.f;
        }

        const int32_t base0 = (p.range.lo + from) * S::kTile + warp * S::kTokens;
#pragma unroll
        for (int i = 0; i < S::kStages - 1; ++i) {
            if (i < count) issue_stage<S>(a, ring + i * S::kStage, look_up<S>(a, p, base0 + i * S::kTile));
            copy_commit();
        }
        RowAt ahead = look_up<S>(a, p, base0 + (S::kStages - 1) * S::kTile);
        int slot = 0, fill = S::kStages - 1;
        for (int32_t i = 0; i < count; ++i) {
            if (i + S::kStages - 1 < count) issue_stage<S>(a, ring + fill * S::kStage, ahead);
            copy_commit();
            fill = fill + 1 == S::kStages ? 0 : fill + 1;
            ahead = look_up<S>(a, p, base0 + (i + S::kStages) * S::kTile);
            copy_wait<S::kStages - 1>();
            __syncwarp();
            const int32_t base = base0 + i * S::kTile;
            if (base < p.range.last && base + S::kTokens > p.range.first)
                step<S>(t, p, ring + slot * S::kStage, base, q, first, last,
                        base >= all_from && base + S::kTokens <= all_to, factor, st);
            slot = slot + 1 == S::kStages ? 0 : slot + 1;
            __syncwarp();
        }
        copy_wait<0>();
        // the four warps' parts meet in shared memory, over the rings
        __syncthreads();
        if (threadIdx.x == 0) odd_rows = 0;
        float* merge = reinterpret_cast<float*>(smem);
#pragma unroll
        for (int nr = 0; nr < S::NR; ++nr)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float l = st.l[nr][i];
                l += __shfl_xor_sync(0xFFFFFFFFu, l, 4);
                l += __shfl_xor_sync(0xFFFFFFFFu, l, 8);
                l += __shfl_xor_sync(0xFFFFFFFFu, l, 16);
                const int row = 8 * nr + 2 * c + i;
                if (row < live) {
                    if (g == 0) {
                        stats[0][warp][row] = st.m[nr][i];
                        stats[1][warp][row] = l;
                    }
#pragma unroll
                    for (int j = 0; j < S::DP / 16; ++j)
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            merge[(warp * S::kRows + row) * (S::DP + 4) + channel<S>(j, g, h)] = st.acc[j][nr][2 * h + i];
                }
            }
        __syncthreads();
        const int groups = a.dim / 8;
        for (int k = threadIdx.x; k < live * groups; k += kThreads) {
            const int row = k / groups, d = 8 * (k - row * groups);
            float m = stats[0][0][row];
#pragma unroll
            for (int i = 1; i < kWarps; ++i) m = fmaxf(m, stats[0][i][row]);
            const float from = m == -INFINITY ? 0.f : m;
            float sum = 0.f, v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < kWarps; ++i) {
                const float f = exp2_fast(stats[0][i][row] - from);
                sum += f * stats[1][i][row];
                const float4* src = reinterpret_cast<const float4*>(&merge[(i * S::kRows + row) * (S::DP + 4) + d]);
                const float4 lo = src[0], hi = src[1];
                v[0] += f * lo.x;
                v[1] += f * lo.y;
                v[2] += f * lo.z;
                v[3] += f * lo.w;
                v[4] += f * hi.x;
                v[5] += f * hi.y;
                v[6] += f * hi.z;
                v[7] += f * hi.w;
            }
            if constexpr (CLUSTERS) {
                float4* dst = reinterpret_cast<float4*>(smem + S::kMerge) + (row * (S::DP + 4) + d) / 4;
                dst[0] = make_float4(v[0], v[1], v[2], v[3]);
                dst[1] = make_float4(v[4], v[5], v[6], v[7]);
                if (d == 0) {
                    gathered[0][row] = m;
                    gathered[1][row] = sum;
                }
                continue;
            }
            if (!full) {
                float4* dst = reinterpret_cast<float4*>(parts.acc(w.share, which) + row * a.dim + d);
                dst[0] = make_float4(v[0], v[1], v[2], v[3]);
                dst[1] = make_float4(v[4], v[5], v[6], v[7]);
                if (d == 0) {
                    parts.stats(w.share, which)[row] = m;
                    parts.stats(w.share, which)[S::kRows + row] = sum;
                }
                continue;
            }
            if (store_row_part<typename S::T>(t, p, S::kRows, row, d, v, m, sum)) atomicOr(&odd_rows, 1u << row);
        }
        if constexpr (CLUSTERS) {
            __syncwarp();
            cluster_sync();
            // this block finishes rows rank, rank + cluster, ...: a warp each
            const int row = (int)rank + cluster * warp;
            if (row < live) {
                // loads of kCluster parts at once: of fewer, the last again, with no weight
                float m = -INFINITY, part_m[kCluster], part_sum[kCluster];
                float4 x[kCluster];
                const uint32_t at = smem_addr(smem) + S::kMerge + 4 * (row * (S::DP + 4) + min(4 * lane, S::DP));
#pragma unroll
                for (int k = 0; k < kCluster; ++k) {
                    const int from_block = min(k, cluster - 1);
                    part_m[k] = load_cluster(in_block(smem_addr(&gathered[0][row]), from_block));
                    part_sum[k] = load_cluster(in_block(smem_addr(&gathered[1][row]), from_block));
                    x[k] = load_cluster4(in_block(at, from_block));
                }
#pragma unroll
                for (int k = 0; k < kCluster; ++k) m = fmaxf(m, part_m[k]);
                const float base = m == -INFINITY ? 0.f : m;
                float sum = 0.f, v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
                for (int k = 0; k < kCluster; ++k) {
                    const float f = k < cluster ? exp2_fast(part_m[k] - base) : 0.f;
                    sum += f * part_sum[k];
                    v[0] += f * x[k].x;
                    v[1] += f * x[k].y;
                    v[2] += f * x[k].z;
                    v[3] += f * x[k].w;
                }
                // pairs of lanes hold 8 values together: the even one stores them
#pragma unroll
                for (int k = 0; k < 4; ++k) v[4 + k] = __shfl_down_sync(0xFFFFFFFFu, v[k], 1);
                bool odd = false;
                if ((lane & 1) == 0 && 4 * lane < a.dim)
                    odd = store_row_part<typename S::T>(t, p, S::kRows, row, 4 * lane, v, m, sum);
                if (__any_sync(0xFFFFFFFFu, odd)) fix_row<typename S::T, S::FMT>(a, t, p, S::kRows, row);
            }
            __syncwarp();
            cluster_sync();  // nobody's shared memory is written again, or given up, before all have read it
            continue;
        }
        __syncthreads();
        if (full) {
            for (uint32_t odd = odd_rows; odd != 0; odd &= odd - 1) {
                const int row = __ffs(odd) - 1;
                if (row % kWarps == warp) fix_row<typename S::T, S::FMT>(a, t, p, S::kRows, row);
            }
            __syncthreads();
        }
    }
}

template <class S>
cudaError_t launch_tokens(const KvArgs& a, const typename S::Args& t, int max_new, int max_len, cudaStream_t s) {
    static PerDeviceOnce once;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    e = once.run(dev, [] {
        const cudaError_t e = cudaFuncSetAttribute(attend_tokens_kernel<S, false>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
        if (e != cudaSuccess) return e;
        return cudaFuncSetAttribute(attend_tokens_kernel<S, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    S::kSmem);
    });
    if (e != cudaSuccess) return e;
    // Cutting items costs a second kernel, about 3.5 us; not cutting them costs up
    // to one item's time at the end.  64 tokens over 512 (8 tiles, 512 items): 28.0
    // us whole, 31.4 cut; over 1024: 47.6, 44.4; 8 over 256 (4 tiles): 9.1, 9.7.
    const int64_t items = (int64_t)a.batch * a.kv_heads;
    const bool whole = max_len <= (items >= S::kShares ? 8 : 4) * S::kTile;
    // Few items: each is shared by a cluster of 4 or 8 blocks, which join their
    // parts through shared memory.  Without, with (us; 8 kv heads of 128, 16-bit,
    // tiles of 64 tokens): one token over 120: 6.4, 6.7 (not taken); 250: 8.0, 6.5;
    // 517: 9.8, 7.1; 2048: 12.0, 9.2; 4096: 15.9, 12.4.  Two: 250: 8.4, 7.3; 1024:
    // 10.5, 9.1; 2048: 12.5, 10.3; 4096: 15.2, 15.8 (not taken).  Four: 1024: 11.3,
    // 11.8 (not taken).  Blocks a cluster, 4 and 8: one over 250: 7.0, 7.5; two
    // over 517: 9.0, 9.8; one over 2048: 12.8, 10.1.  A share does the items that
    // begin in it, and lengths differ: with one share an item some do two (two
    // tokens over 2048: 14.1 against 11.2), with up to four few do.
    const int64_t tiled = items * (((int64_t)t.group.d * max_new + S::kRows - 1) / S::kRows);
    const bool alone = tiled * kCluster * 2 <= kSms;
    if (tiled * kCluster * 2 <= S::kShares && max_len > 2 * S::kTile && max_len <= (alone ? 64 : 32) * S::kTile) {
        const int cluster = max_len <= 8 * S::kTile ? kCluster / 2 : kCluster;
        const bool equal = a.batch == 1 && tiled == items;
        const int64_t clusters = equal ? items : std::min<int64_t>(4 * tiled, S::kShares / cluster);
        return launch_clusters(attend_tokens_kernel<S, true>, (int)clusters * cluster, cluster, kThreads, S::kSmem, s,
                               a, t, cluster);
    }
    const int shares = shares_for(a, t, max_new, max_len, S::kRows, S::kTile, S::kShares);
    attend_tokens_kernel<S, false><<<shares, kThreads, S::kSmem, s>>>(a, t, whole ? 1 : 0);
    e = cudaGetLastError();
    if (e != cudaSuccess || whole) return e;
    return launch_join(join_rows_kernel<typename S::T, S::FMT, S::kRows, typename S::Args>, a, t, shares,
                       S::kRows / kJoinFew, kJoinFewThreads, 0, s);
}

template <class T, int FMT, int DP, class Args>
cudaError_t launch_rows(const KvArgs& a, const Args& t, int max_new, int max_len, cudaStream_t s) {
    return (int64_t)t.group.d * max_new <= 8 ? launch_tokens<Shape<T, FMT, DP, 1, Args>>(a, t, max_new, max_len, s)
                                             : launch_tokens<Shape<T, FMT, DP, 2, Args>>(a, t, max_new, max_len, s);
}
template <class T, int FMT, class Args>
cudaError_t launch_dim(const KvArgs& a, const Args& t, int max_new, int max_len, cudaStream_t s) {
    return a.dim <= 64 ? launch_rows<T, FMT, 64>(a, t, max_new, max_len, s)
                       : launch_rows<T, FMT, 128>(a, t, max_new, max_len, s);
}

template <class Args>
cudaError_t launch_any(int dtype, int format, const KvArgs& a, const Args& t, int max_new, int max_len,
                       cudaStream_t s) {
    if (dtype == (int)Bf16::kCode) {
        if (format == kKv16Bit) return launch_dim<BfType, kKv16Bit>(a, t, max_new, max_len, s);
        return format == kKvInt8 ? launch_dim<BfType, kKvInt8>(a, t, max_new, max_len, s)
                                 : launch_dim<BfType, kKvE4m3>(a, t, max_new, max_len, s);
    }
    if (format == kKv16Bit) return launch_dim<HfType, kKv16Bit>(a, t, max_new, max_len, s);
    return format == kKvInt8 ? launch_dim<HfType, kKvInt8>(a, t, max_new, max_len, s)
                             : launch_dim<HfType, kKvE4m3>(a, t, max_new, max_len, s);
}

}  // namespace

}  // namespace cccl
