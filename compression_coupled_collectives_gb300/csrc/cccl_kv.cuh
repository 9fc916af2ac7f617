// cccl_kv.cuh -- what the paged key/value cache kernels share (sm_103a): the
// launch arguments, the way from a position to its place in the cache, 8-bit
// codes, and the row-at-a-time form of attention.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "cccl_device.cuh"

namespace cccl {

constexpr int kKv16Bit = 0, kKvInt8 = 1, kKvE4m3 = 2;  // CCCL_KV_*

// Division of 0 <= n < 2^31 by d >= 1 as a multiplication: with
// 2^(s-1) < d <= 2^s and m = ceil(2^(31+s) / d) the error m d - 2^(31+s) is
// below d <= 2^s, so floor(n m / 2^(31+s)) = floor(n / d) for n < 2^31.
struct FastDiv {
    uint32_t d, m, s;
};
inline FastDiv fast_div(uint32_t d) {
    uint32_t s = 0;
    while ((1ull << s) < d) ++s;
    const uint64_t p = 1ull << (31 + s);
    return FastDiv{d, (uint32_t)((p + d - 1) / d), s};
}
__device__ __forceinline__ uint32_t div_by(const FastDiv& f, uint32_t n) {
    return (uint32_t)(((uint64_t)n * f.m) >> (31 + f.s));
}

// One call on one cache and batch.  Strides of k and v in bytes, of the
// scales in floats, of the packed tensors (x, y) in bytes.
struct KvArgs {
    uint8_t *k, *v;
    float *k_scale, *v_scale;
    int64_t page_stride, token_stride, head_stride;
    int64_t s_page, s_token, s_head;
    int64_t pages;
    const int32_t *table, *cu, *lens;
    int64_t table_stride, n_tokens;
    WsHeader* ws;
    FastDiv page_tokens;
    int32_t kv_heads, dim, batch, table_pages;
};
// The packed K and V of a write or a read.
struct KvPacked {
    uint8_t *k, *v;
    int64_t k_token, k_head, v_token, v_head;
};
// What attention adds.
struct AttnArgs {
    const uint8_t* q;
    uint8_t* out;
    float* lse;
    int64_t q_token, q_head, o_token, o_head;
    float scale;
    int32_t window;  // 0: none
    int32_t causal, q_heads;
    FastDiv group;  // query heads that share a kv head
};
// Attention of drafted tokens: token i of a sequence's n new ones sees what was
// cached before them and those of them whose bit is set in its row of `mask`
// (bit k in word k / 32; bits from 32 words on are clear).  The kernels are
// written for either kind of arguments, Args.
struct TreeArgs : AttnArgs {
    const uint32_t* mask;
    int64_t mask_stride;  // words from one row to the next
    int32_t words;        // of a row
    int32_t narrow_rows;  // items of so many rows at most are shared by two warpgroups (many rows)
};

// Sequence b's rows and length, with everything that does not fit clamped
// (and reported): 0 <= row, row + n <= n_tokens, 0 <= len <= table capacity.
struct Sequence {
    int64_t row;  // first row of its new tokens
    int32_t n;    // new tokens
    int32_t len;  // cached tokens, the new ones included
};
__device__ __forceinline__ Sequence load_sequence(const KvArgs& a, int b) {
    const int64_t lo = a.cu[b], hi = a.cu[b + 1];
    const int64_t len = a.lens[b];
    const int64_t cap = min((int64_t)a.table_pages * a.page_tokens.d, (int64_t)0x7FFF0000);
    Sequence s;
    s.row = min(max(lo, (int64_t)0), a.n_tokens);
    const int64_t end = min(max(hi, s.row), a.n_tokens);
    s.n = (int32_t)(end - s.row);
    s.len = (int32_t)min(max(len, (int64_t)0), cap);
    if (s.row != lo || end != hi || s.len != len) record_error(a.ws, kStatusInvalidArg);
    return s;
}

// Page of position p of sequence b (p inside the table), or -1 (reported).
__device__ __forceinline__ int64_t page_of(const KvArgs& a, int b, uint32_t page_index) {
    const int64_t e = a.table[(int64_t)b * a.table_stride + page_index];
    if (e < 0 || e >= a.pages) {
        record_error(a.ws, kStatusInvalidArg);
        return -1;
    }
    return e;
}
// Where position p's vectors lie: byte offset of head 0 in k and v, float
// offset of its scales.  Returns false for a page outside the cache.
__device__ __forceinline__ bool slot_of(const KvArgs& a, int b, uint32_t p, int64_t& at, int64_t& scale_at) {
    const uint32_t pi = div_by(a.page_tokens, p), slot = p - pi * a.page_tokens.d;
    const int64_t page = page_of(a, b, pi);
    at = page * a.page_stride + (int64_t)slot * a.token_stride;
    scale_at = page * a.s_page + (int64_t)slot * a.s_token;
    return page >= 0;
}

// The keys that a row at position `pos` of a sequence sees: first .. last - 1
// (none when last <= first).  row: its place in the packed tensors.
__device__ __forceinline__ void visible_range(const AttnArgs& t, const Sequence& s, int64_t, int32_t pos, int32_t& first,
                                              int32_t& last) {
    last = max(t.causal ? min(s.len, pos + 1) : s.len, 0);
    first = t.window > 0 && pos >= t.window ? min(pos - t.window + 1, last) : 0;
}
// Drafted tokens: the tokens before the draft lie at positions below this.
__device__ __forceinline__ int32_t before_draft(const Sequence& s) { return s.len - s.n; }
__device__ __forceinline__ const uint32_t* draft_bits(const TreeArgs& t, int64_t row) {
    return t.mask + row * t.mask_stride;
}
// Word w of a row's mask without the bits of tokens at negative positions and of
// those from n on.
__device__ __forceinline__ uint32_t draft_word(const uint32_t* bits, int32_t w, int32_t before, int32_t n) {
    const int32_t lo = max(-before, 0) - 32 * w, hi = n - 32 * w;  // bits lo .. hi - 1
    if (hi <= 0 || lo >= 32) return 0;
    uint32_t x = bits[w];
    if (lo > 0) x &= ~0u << lo;
    if (hi < 32) x &= ~(~0u << hi);
    return x;
}
// Here what lies between first and last is visible where it is not drafted or
// its bit is set (drafted_seen).  A window leaves the last `window` of what the
// row sees without it: tokens before the draft, then drafted ones by their place.
// last is one past the last of them, so a row sees something exactly when
// first < last.  (A tree of n tokens has few words: n / 32.)
static __device__ __noinline__ int2 draft_range(const uint32_t* bits, int32_t words, int32_t before, int32_t n,
                                                int32_t window) {
    words = min(words, (n + 31) / 32);
    int32_t highest = -1, count = 0;
    for (int32_t w = 0; w < words; ++w) {
        const uint32_t x = draft_word(bits, w, before, n);
        count += __popc(x);
        if (x != 0) highest = 32 * w + 31 - __clz(x);
    }
    const int32_t last = highest >= 0 ? before + highest + 1 : max(before, 0);
    if (window <= 0) return make_int2(0, last);
    if (count <= window) return make_int2((int32_t)max((int64_t)before + count - window, (int64_t)0), last);
    // the window ends among the drafted tokens: skip the first count - window of them
    int32_t skip = count - window;
    for (int32_t w = 0; w < words; ++w) {
        uint32_t x = draft_word(bits, w, before, n);
        if (__popc(x) <= skip) {
            skip -= __popc(x);
            continue;
        }
        for (; skip > 0; --skip) x &= x - 1;
        return make_int2(before + 32 * w + __ffs(x) - 1, last);
    }
    return make_int2(last, last);  // (not reached)
}
__device__ __forceinline__ void visible_range(const TreeArgs& t, const Sequence& s, int64_t row, int32_t, int32_t& first,
                                              int32_t& last) {
    const int2 r = draft_range(draft_bits(t, row), t.words, before_draft(s), s.n, t.window);
    first = r.x;
    last = r.y;
}
// Where a row's keys are to be looked for: its range, or without a window's
// need of it all of the sequence, so that nothing waits for the mask (which is
// asked for, for the tiles that need it).
__device__ __forceinline__ void search_range(const AttnArgs& t, const Sequence& s, int64_t row, int32_t pos,
                                             int32_t& first, int32_t& last) {
    visible_range(t, s, row, pos, first, last);
}
__device__ __forceinline__ void search_range(const TreeArgs& t, const Sequence& s, int64_t row, int32_t pos,
                                             int32_t& first, int32_t& last) {
    if (t.window > 0) {
        visible_range(t, s, row, pos, first, last);
        return;
    }
    first = 0;
    last = s.len;
    asm volatile("prefetch.global.L1 [%0];" ::"l"(draft_bits(t, row)));
}
// Whether a row whose weights add up to `sum` sees no key.
__device__ __forceinline__ bool sees_none(const AttnArgs& t, const Sequence& s, int64_t row, int32_t pos, float) {
    int32_t first, last;
    visible_range(t, s, row, pos, first, last);
    return last <= first;
}
__device__ __forceinline__ bool sees_none(const TreeArgs& t, const Sequence& s, int64_t row, int32_t pos, float sum) {
    if (sum > 0.f) return false;
    int32_t first, last;
    visible_range(t, s, row, pos, first, last);
    return last <= first;
}
// Whether a row sees position j, which lies between its first and last.
__device__ __forceinline__ bool drafted_seen(const AttnArgs&, const Sequence&, int64_t, int32_t) { return true; }
__device__ __forceinline__ bool drafted_seen(const TreeArgs& t, const Sequence& s, int64_t row, int32_t j) {
    const int32_t k = j - before_draft(s);
    return k < 0 || (k < 32 * (int64_t)t.words && (draft_bits(t, row)[k >> 5] >> (k & 31) & 1u) != 0);
}
// The positions below which every one between a row's first and last is seen.
__device__ __forceinline__ int32_t gapless_below(const AttnArgs&, const Sequence&, int32_t last) { return last; }
__device__ __forceinline__ int32_t gapless_below(const TreeArgs&, const Sequence& s, int32_t last) {
    return min(last, max(before_draft(s), 0));
}
// Bit i: whether a row sees position j + i, where that lies between its first and last.
__device__ __forceinline__ uint32_t seen_32(const AttnArgs&, const Sequence&, int64_t, int32_t) { return ~0u; }
__device__ __forceinline__ uint32_t seen_32(const TreeArgs& t, const Sequence& s, int64_t row, int32_t j) {
    const int32_t k = j - before_draft(s);
    if (k <= -32) return ~0u;
    const uint32_t* bits = draft_bits(t, row);
    const int32_t w = k >> 5;  // rounded down
    const uint32_t x = w >= 0 && w < t.words ? bits[w] : 0u, y = w + 1 < t.words ? bits[w + 1] : 0u;
    const uint32_t z = __funnelshift_r(x, y, (uint32_t)k & 31u);
    return k < 0 ? z | ~(~0u << -k) : z;
}

// ---------------------------------------------------------------- values
// The two 16-bit types: bf16 and fp16 as the packed values' type.
struct BfType {
    static constexpr bool kHalf = false;
    static __device__ __forceinline__ float load(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }
    static __device__ __forceinline__ uint16_t round(float x) { return __bfloat16_as_ushort(__float2bfloat16_rn(x)); }
};
struct HfType {
    static constexpr bool kHalf = true;
    static __device__ __forceinline__ float load(uint16_t b) { return __half2float(__ushort_as_half(b)); }
    static __device__ __forceinline__ uint16_t round(float x) { return __half_as_ushort(__float2half_rn(x)); }
};
template <class T>
__device__ __forceinline__ uint32_t round_pair(float lo, float hi) {
    return (uint32_t)T::round(lo) | ((uint32_t)T::round(hi) << 16);
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
    return x;
}

// 4 codes -> fp16 values, exactly, as two pairs: E4M3 in the order (0, 1),
// (2, 3), INT8 in the order (0, 2), (1, 3) (the cheaper one for each; callers
// arrange the other operand or the bytes to suit).  INT8: with u = code + 128
// (the code's sign bit flipped), 0x6400 | u is 1024 + u; taking off 1152 leaves
// the code.
template <int FMT>
__device__ __forceinline__ void expand4(uint32_t w, uint32_t& a, uint32_t& b) {
    if (FMT == kKvE4m3) {
        asm("{ .reg .b16 l, h; mov.b32 {l, h}, %2; cvt.rn.f16x2.e4m3x2 %0, l; cvt.rn.f16x2.e4m3x2 %1, h; }"
            : "=r"(a), "=r"(b)
            : "r"(w));
    } else {
        const uint32_t x = (w & 0x00FF00FFu) ^ 0x64806480u, y = ((w >> 8) & 0x00FF00FFu) ^ 0x64806480u;
        const __half2 bias = __half2half2(__ushort_as_half(0x6480));  // 1152
        const __half2 p = __hsub2(*reinterpret_cast<const __half2*>(&x), bias);
        const __half2 q = __hsub2(*reinterpret_cast<const __half2*>(&y), bias);
        a = *reinterpret_cast<const uint32_t*>(&p);
        b = *reinterpret_cast<const uint32_t*>(&q);
    }
}

// The same, in the order (0, 1), (2, 3) for both.
template <int FMT>
__device__ __forceinline__ void expand4_in_order(uint32_t w, uint32_t& a, uint32_t& b) {
    if (FMT == kKvE4m3) {
        expand4<FMT>(w, a, b);
    } else {
        const uint32_t u = w ^ 0x80808080u;
        const uint32_t x = __byte_perm(u, 0x64646464u, 0x4140), y = __byte_perm(u, 0x64646464u, 0x4342);
        const __half2 bias = __half2half2(__ushort_as_half(0x6480));  // 1152
        const __half2 p = __hsub2(*reinterpret_cast<const __half2*>(&x), bias);
        const __half2 q = __hsub2(*reinterpret_cast<const __half2*>(&y), bias);
        a = *reinterpret_cast<const uint32_t*>(&p);
        b = *reinterpret_cast<const uint32_t*>(&q);
    }
}

// 8-bit caches are multiplied in fp16, which holds every code exactly.
//
// Queries: a bf16 row is first multiplied by a power of two that brings its
// largest value to 2^14..2^15.  Every value down to 2^-29 of the largest is
// then exact in fp16, and smaller ones are off by 2^-40 of the largest, far
// below the binary32 sum's own rounding.  fp16 rows stay as they are.
// amax: the row's largest pattern without its sign.
template <class T>
__device__ __forceinline__ float query_power(uint32_t amax) {
    if (T::kHalf || amax == 0 || amax >= 0x7F80u) return 1.f;
    const int e = max((int)(amax >> 7) - 127, -100);
    return __uint_as_float((uint32_t)(127 + 14 - e) << 23);
}
template <class T>
__device__ __forceinline__ uint32_t scaled_pair(uint32_t w, float power) {
    if (T::kHalf) return w;
    const __half2 h = __floats2half2_rn(T::load((uint16_t)(w & 0xFFFFu)) * power, T::load((uint16_t)(w >> 16)) * power);
    return *reinterpret_cast<const uint32_t*>(&h);
}
// Probabilities meet their value's scale before they go to fp16, so a row's
// reference follows the largest of 2^s_j |scale_j| over the keys that it sees,
// whatever other keys' scales are: the largest product is then near the top of
// fp16's range.  The quotient does not depend on the reference.  This is
// log2 |scale_j| but for 0.09 (the fraction's bits taken for its logarithm);
// limited, so that the sum of 2^(s_j - reference) stays in binary32's range, to
// -90 (smaller scales may lose bits, zeros do not matter) and 100 (products of
// larger ones can overflow fp16: such rows come out non-finite and are worked out
// by attend_row).  lower: taken off.
__device__ __forceinline__ uint32_t scale_bits(float scale) { return __float_as_uint(scale) & 0x7FFFFFFFu; }
__device__ __forceinline__ float scale_log2(uint32_t bits, float lower = 0.f) {
    return fminf(fmaxf(fmaf((float)bits, 0x1p-23f, -127.f - lower), -90.f - lower), 100.f - lower);
}

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool real) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(real ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src, bool real) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(real ? 4 : 0) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// 4 stored values (8 or 4 bytes) as binary32, without their scale.
template <int FMT>
__device__ __forceinline__ uint2 load_stored4(const uint8_t* p) {
    if (FMT == kKv16Bit) return *reinterpret_cast<const uint2*>(p);
    return make_uint2(*reinterpret_cast<const uint32_t*>(p), 0);
}
template <class T, int FMT>
__device__ __forceinline__ float4 stored4_values(uint2 x) {
    if (FMT == kKv16Bit)
        return make_float4(T::load((uint16_t)(x.x & 0xFFFFu)), T::load((uint16_t)(x.x >> 16)),
                           T::load((uint16_t)(x.y & 0xFFFFu)), T::load((uint16_t)(x.y >> 16)));
    uint32_t lo, hi;
    expand4_in_order<FMT>(x.x, lo, hi);
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&lo));
    const float2 g = __half22float2(*reinterpret_cast<const __half2*>(&hi));
    return make_float4(f.x, f.y, g.x, g.y);
}
// One row of attention by one warp, straight from the definition: a pass for
// the maximum and the sum of the exponentials, one for the values with their
// normalised weights (so that no sum passes the values' own size), visible keys
// only, IEEE arithmetic throughout (a NaN or an infinity among the visible
// values goes where the formula takes it, one in a hidden place goes nowhere).
// The tensor-core kernels compute hidden places as products with zero, which is
// not the same when such a place holds a NaN or an infinity; they send the rows
// whose sums come out non-finite through here, where nothing waits for them.
// 32 keys at a time: every lane looks one up and owns its score.  A key's
// channels lie across the warp, 4 a lane; the loads of 2 keys are in flight, and
// waiting for them is most of its time: one NaN in one of 8 heads makes 4096 new
// tokens over 32768 take 1.77 s for 1.3 ms, one token over 32768 21 ms for 0.07.
// Registers are few here, since the kernels' own count must not grow by this: 4
// keys in flight took 1.27 s, 16 and 8 lanes a key less still, but through the
// joining kernels' spills single tokens 0.5 to 2.5 % more.
template <class T, int FMT, class Args>
__device__ __noinline__ void attend_row(const KvArgs& a, const Args& t, int b, const Sequence& sequence, int64_t row,
                                        int32_t pos, int head) {
    constexpr uint32_t kAll = 0xFFFFFFFFu;
    constexpr int kFlight = 2;
    const int lane = threadIdx.x & 31;
    const int kv_head = (int)div_by(t.group, (uint32_t)head);
    const bool inside = 4 * lane < a.dim;
    const uint32_t column = (FMT == kKv16Bit ? 8 : 4) * lane;
    float4 q = make_float4(0.f, 0.f, 0.f, 0.f), acc = q;
    if (inside)
        q = stored4_values<T, kKv16Bit>(
            load_stored4<kKv16Bit>(t.q + row * t.q_token + (int64_t)head * t.q_head + 8 * lane));
    int32_t first, last;
    visible_range(t, sequence, row, pos, first, last);
    float m = -INFINITY, sum = 0.f;  // of this lane's keys; then of all
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass) {
#pragma unroll 1
        for (int32_t base = first; base < last; base += 32) {
            const bool seen = lane < last - base && drafted_seen(t, sequence, row, base + lane);
            int64_t at = 0, scale_at = 0;
            const bool there = seen && slot_of(a, b, (uint32_t)(base + lane), at, scale_at);
            at += (int64_t)kv_head * a.head_stride;
            float kscale = 1.f, vscale = 1.f, s = 0.f;
            if (FMT != kKv16Bit && there) {
                kscale = a.k_scale[scale_at + (int64_t)kv_head * a.s_head];
                vscale = a.v_scale[scale_at + (int64_t)kv_head * a.s_head];
            }
            const uint32_t real = __ballot_sync(kAll, there);
#pragma unroll 1
            for (int i = 0; i < 32; i += kFlight) {
                uint2 x[kFlight];
#pragma unroll
                for (int k = 0; k < kFlight; ++k) {
                    const int64_t from = __shfl_sync(kAll, at, i + k);
                    x[k] = make_uint2(0, 0);
                    if (inside && (real >> (i + k) & 1u) != 0) x[k] = load_stored4<FMT>(a.k + from + column);
                }
#pragma unroll
                for (int k = 0; k < kFlight; ++k) {
                    const float4 y = stored4_values<T, FMT>(x[k]);
                    float dot = q.x * y.x;
                    dot += q.y * y.y;
                    dot += q.z * y.z;
                    dot += q.w * y.w;
                    dot = warp_sum(dot);
                    if (lane == i + k && there) s = dot;  // (else 0, also where the query is infinite)
                }
            }
            s = s * kscale * t.scale;  // (in this order: the scales' product may leave binary32's range)
            if (pass == 0) {
                if (seen) {
                    const float to = (s > m || s != s) ? s : m;  // keeps a NaN: no later s compares above it
                    const float from = to == -INFINITY ? 0.f : to;
                    sum = sum * expf(m - from) + expf(s - from);
                    m = to;
                }
                continue;
            }
            const float p = seen ? expf(s - m) / sum : 0.f;
#pragma unroll 1
            for (int i = 0; i < 32; i += kFlight) {
                uint2 x[kFlight];
#pragma unroll
                for (int k = 0; k < kFlight; ++k) {
                    const int64_t from = __shfl_sync(kAll, at, i + k);
                    x[k] = make_uint2(0, 0);
                    if (inside && (real >> (i + k) & 1u) != 0) x[k] = load_stored4<FMT>(a.v + from + column);
                }
#pragma unroll
                for (int k = 0; k < kFlight; ++k) {
                    const float weight = __shfl_sync(kAll, p, i + k), scale = __shfl_sync(kAll, vscale, i + k);
                    if ((real >> (i + k) & 1u) != 0) {
                        const float4 y = stored4_values<T, FMT>(x[k]);
                        acc.x += weight * (y.x * scale);
                        acc.y += weight * (y.y * scale);
                        acc.z += weight * (y.z * scale);
                        acc.w += weight * (y.w * scale);
                    }
                }
            }
        }
        if (pass == 0) {  // all lanes' keys together
            const float own = m;
            const bool odd = __any_sync(kAll, own != own) != 0;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, o));
            sum = warp_sum(sum * expf(own - (m == -INFINITY ? 0.f : m)));
            // scores of -infinity alone are 0 / 0, as in the formula
            if (odd || sum != sum || (m == -INFINITY && last > first)) {  // no weight is a number
                m = sum = __uint_as_float(0x7FC00000u);
                acc = make_float4(m, m, m, m);
                break;
            }
        }
    }
    if (inside)
        *reinterpret_cast<uint2*>(t.out + row * t.o_token + (int64_t)head * t.o_head + 8 * lane) =
            make_uint2(round_pair<T>(acc.x, acc.y), round_pair<T>(acc.z, acc.w));
    if (t.lse != nullptr && lane == 0) t.lse[row * t.q_heads + head] = last > first ? m + logf(sum) : -INFINITY;
}

}  // namespace cccl
