// cccl_step_write.cu -- rotary positions for a step's queries and keys, and its
// keys and values into the cache's pages, in one pass over the data.
//
// Bound by HBM: queries are read and written, keys and values read and stored:
// 12572 tokens of 32 + 2 x 8 heads of 128 in 53.4 us, 5.8 TB/s, 0.85 of the measured
// copy; 91 tokens in 3.6.
// The angles' sines and cosines are worked out once a token and shared by its
// heads: a block brings up to 8 tokens and fills a table in shared memory first.
//
// Angles: a pair turns by turns / 2^64 of a full turn a position, so position p
// stands at p * turns modulo 2^64 of one: whole turns fall out of the 64-bit
// product exactly, at any position, and nothing else is rounded there.  Its top 32
// bits, as a number of half turns in -1..1, go to sincospi, which takes nothing off
// a large argument.  The table itself, where it comes from binary64, is off by up
// to 2^-55.5 of a turn a position (bases of 10^4 and 5 10^5): 2^-36 radians at
// position 2^17.
//
// A vector (token, head, Q, K or V) belongs to G lanes of 16 values each, two
// pieces of 8.  Interleaved pairs lie in one piece; with pairs half the rotary
// part apart a lane takes piece j and the one rot_dim / 16 pieces on, so that it
// holds both of every pair.
#include <algorithm>

#include "cccl_kv_copy.cuh"
#include "cccl_kv_launch.h"
#include "cccl_step.cuh"

namespace cccl {

namespace {

// Tokens of a block: up to 8, so that a large call has two blocks' worth for every
// place on an SM, and one's search and angles run beside another's loads: 12572
// tokens of 32 + 2 x 8 heads of 128 in 59.6 us at 16, 53.4 at 8, 53.7 at 4, 54.4 at 2.
constexpr int kTokens = 8;

// cos and sin of pairs 8 j + 2 i and + 1 of a block's tokens: a piece's 8 pairs
// are 4 entries, those of a vector's lanes side by side (no bank met twice).
template <int G>
struct Angles {
    float4 of[kTokens][4][G];
};
template <int G>
__device__ __forceinline__ void fill_angles(const RotaryArgs& r, const TokenSlots& slots, int64_t t0, int count,
                                            Angles<G>& s) {
    const int halves = r.rot_dim / 4;  // entries of a token: two pairs each
    for (int i = threadIdx.x; i < count * halves; i += kCopyThreads) {
        const int tok = i / halves, e = i - tok * halves;
        if (slots.state[tok] == 0) continue;
        const int64_t pos = r.positions != nullptr ? r.positions[t0 + tok] : slots.pos[tok];
        float c[2], d[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const uint64_t turn = (uint64_t)pos * r.turns[2 * e + k];
            sincospif((float)(int32_t)(uint32_t)(turn >> 32) * 0x1p-31f, &d[k], &c[k]);
        }
        s.of[tok][e & 3][e >> 2] = make_float4(c[0] * r.magnitude, d[0] * r.magnitude, c[1] * r.magnitude,
                                               d[1] * r.magnitude);
    }
}

template <class T>
__device__ __forceinline__ void widen(const uint4& x, float* y) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        y[2 * i] = T::load((uint16_t)(w[i] & 0xFFFFu));
        y[2 * i + 1] = T::load((uint16_t)(w[i] >> 16));
    }
}
template <class T>
__device__ __forceinline__ uint4 narrow(const float* y) {
    return make_uint4(round_pair<T>(y[0], y[1]), round_pair<T>(y[2], y[3]), round_pair<T>(y[4], y[5]),
                      round_pair<T>(y[6], y[7]));
}
// 8 values as codes.  INT8: adding 1.5 * 2^23 rounds a value below 2^22 to an
// integer, ties to even, and leaves it in the sum's low bits.
template <int FMT>
__device__ __forceinline__ uint2 encode8(const float* x, float inv) {
    uint32_t c[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = x[4 * h + i] * inv;
        if (FMT == kKvInt8) {
            uint32_t r[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) r[i] = __float_as_uint(__fadd_rn(y[i], 12582912.f));
            c[h] = __byte_perm(__byte_perm(r[0], r[1], 0x0040), __byte_perm(r[2], r[3], 0x0040), 0x5410);
        } else {
            const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(y[0], y[1]), __NV_SATFINITE, __NV_E4M3);
            const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(y[2], y[3]), __NV_SATFINITE, __NV_E4M3);
            c[h] = lo | (hi << 16);
        }
    }
    return make_uint2(c[0], c[1]);
}

// The 16 values of a lane turned by its 8 pairs.
template <int G, bool INTER>
__device__ __forceinline__ void turn16(const Angles<G>& s, int tok, int part, float* y) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float4 f = s.of[tok][i][part];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int pair = 2 * i + k, at = INTER ? 2 * pair : pair, to = INTER ? at + 1 : at + 8;
            const float c = k ? f.z : f.x, d = k ? f.w : f.y, a = y[at], b = y[to];
            y[at] = a * c - b * d;
            y[to] = b * c + a * d;
        }
    }
}

template <class T, int FMT, int G, bool INTER>
__global__ void __launch_bounds__(kCopyThreads)
    step_write_kernel(const __grid_constant__ KvArgs a, const __grid_constant__ KvPacked x,
                      const __grid_constant__ RotaryArgs r, FastDiv heads, FastDiv q_heads, int tokens) {
    __shared__ TokenSlots slots;
    __shared__ Angles<G> angles;
    const int64_t t0 = (int64_t)blockIdx.x * tokens;
    const int count = (int)min((int64_t)tokens, a.n_tokens - t0);
    find_slots(a, t0, count, slots);
    __syncthreads();
    fill_angles<G>(r, slots, t0, count, angles);
    __syncthreads();
    const int part = threadIdx.x % G;
    const bool inside = 16 * part < a.dim, turned = 16 * part < r.rot_dim;
    // the lane's two pieces of 8 values, as bytes of 16-bit values
    const int at0 = 16 * (!INTER && turned ? part : 2 * part);
    const int at1 = 16 * (!INTER && turned ? part + r.rot_dim / 16 : 2 * part + 1);
    const int of_q = count * r.q_heads, of_k = count * (int)heads.d;
    const int total = of_q + 2 * of_k;
    for (int base = 0; base < total; base += kCopyThreads / G) {
        const int vec = base + (int)threadIdx.x / G;
        const bool is_q = vec < of_q, is_v = vec >= of_q + of_k;
        const FastDiv& by = is_q ? q_heads : heads;
        const int v = is_q ? vec : vec - of_q - (is_v ? of_k : 0);
        const int tok = vec < total ? (int)div_by(by, (uint32_t)v) : 0, head = v - tok * (int)by.d;
        const int state = slots.state[tok];
        const bool live = vec < total && (is_q ? state != 0 : state == 1);
        float y[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) y[i] = 0.f;
        uint4 raw0 = make_uint4(0, 0, 0, 0), raw1 = raw0;
        if (live && inside) {
            const uint8_t* src = is_q ? r.q + (t0 + tok) * r.q_token + head * r.q_head
                                      : (is_v ? x.v + (t0 + tok) * x.v_token + head * x.v_head
                                              : x.k + (t0 + tok) * x.k_token + head * x.k_head);
            raw0 = load_stream(src + at0);
            raw1 = load_stream(src + at1);
            widen<T>(raw0, y);
            widen<T>(raw1, y + 8);
            if (!is_v && turned) {
                turn16<G, INTER>(angles, tok, part, y);
                raw0 = narrow<T>(y);
                raw1 = narrow<T>(y + 8);
            }
        }
        if (is_q && live && inside) {
            uint8_t* dst = r.q_out + (t0 + tok) * r.o_token + head * r.o_head;
            *reinterpret_cast<uint4*>(dst + at0) = raw0;
            *reinterpret_cast<uint4*>(dst + at1) = raw1;
        }
        uint8_t* const row = (is_v ? a.v : a.k) + slots.at[live ? tok : 0] + head * a.head_stride;
        if (FMT == kKv16Bit) {
            if (!is_q && live && inside) {
                *reinterpret_cast<uint4*>(row + at0) = raw0;
                *reinterpret_cast<uint4*>(row + at1) = raw1;
            }
            continue;
        }
        // the largest pattern of |y|: for numbers their order, a NaN's above infinity's
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 16; ++i) m = max(m, __float_as_uint(y[i]) & 0x7FFFFFFFu);
#pragma unroll
        for (int o = G / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        const float amax = __uint_as_float(m);
        constexpr float kLimit = FMT == kKvInt8 ? 127.f : 448.f;
        // inv is limited to the largest finite number, so that a subnormal
        // maximum does not turn zeros into NaN
        const float inv = amax == 0.f ? 0.f : fminf(kLimit / amax, 3.402823466e+38f);
        if (!is_q && live) {
            if (inside) {
                *reinterpret_cast<uint2*>(row + at0 / 2) = encode8<FMT>(y, inv);
                *reinterpret_cast<uint2*>(row + at1 / 2) = encode8<FMT>(y + 8, inv);
            }
            if (part == 0)
                (is_v ? a.v_scale : a.k_scale)[slots.scale_at[tok] + head * a.s_head] =
                    amax <= 3.402823466e+38f ? amax / kLimit : __uint_as_float(0x7FC00000u);
        }
    }
}

template <class T, int FMT>
cudaError_t launch_one(const KvArgs& a, const KvPacked& x, const RotaryArgs& r, bool interleaved, cudaStream_t s) {
    const int tpb = std::min(tokens_per_block(a.n_tokens), kTokens);
    const FastDiv heads = fast_div((uint32_t)a.kv_heads), q_heads = fast_div((uint32_t)(r.q_heads > 0 ? r.q_heads : 1));
    const dim3 grid((unsigned)((a.n_tokens + tpb - 1) / tpb));
    if (a.dim <= 64) {
        if (interleaved)
            step_write_kernel<T, FMT, 4, true><<<grid, kCopyThreads, 0, s>>>(a, x, r, heads, q_heads, tpb);
        else
            step_write_kernel<T, FMT, 4, false><<<grid, kCopyThreads, 0, s>>>(a, x, r, heads, q_heads, tpb);
    } else {
        if (interleaved)
            step_write_kernel<T, FMT, 8, true><<<grid, kCopyThreads, 0, s>>>(a, x, r, heads, q_heads, tpb);
        else
            step_write_kernel<T, FMT, 8, false><<<grid, kCopyThreads, 0, s>>>(a, x, r, heads, q_heads, tpb);
    }
    return cudaGetLastError();
}
template <class T>
cudaError_t launch_format(int format, const KvArgs& a, const KvPacked& x, const RotaryArgs& r, bool interleaved,
                          cudaStream_t s) {
    if (format == kKv16Bit) return launch_one<T, kKv16Bit>(a, x, r, interleaved, s);
    return format == kKvInt8 ? launch_one<T, kKvInt8>(a, x, r, interleaved, s)
                             : launch_one<T, kKvE4m3>(a, x, r, interleaved, s);
}

}  // namespace

cudaError_t launch_step_write(int dtype, int format, const KvArgs& a, const KvPacked& x, const RotaryArgs& r,
                              bool interleaved, cudaStream_t s) {
    return dtype == (int)Bf16::kCode ? launch_format<BfType>(format, a, x, r, interleaved, s)
                                     : launch_format<HfType>(format, a, x, r, interleaved, s);
}

}  // namespace cccl
