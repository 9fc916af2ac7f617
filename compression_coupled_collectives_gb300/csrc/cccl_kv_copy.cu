// cccl_kv_copy.cu -- storing tokens in the paged cache and taking them out
// again.  Both are one pass over the data and bound by HBM: a token and head
// moves 2 D bytes on the packed side and D or 2 D (and a 4-byte scale) on the
// cache's.  GB300: 131072 tokens x 8 heads x 128, INT8 to bf16, in 126.5 us
// (6.43 TB/s, 0.95 of the measured copy); small calls are bound by the launch and
// the four loads in a row that find a token's page (2.6 us for 333 tokens).
//
// A vector (token, head, K or V) belongs to a group of G lanes, 16 values a lane
// (32 bytes of values, 16 of codes).
// The maximum is taken over the patterns of |x| as integers, two values per
// instruction: for non-negative 16-bit floats the order of the patterns is the
// order of the values, and a NaN's pattern lies above infinity's, so a NaN
// stays the maximum.  A vector whose maximum is not finite gets a NaN as its
// scale, whatever its codes.
#include "cccl_kv.cuh"
#include "cccl_kv_copy.cuh"
#include "cccl_kv_launch.h"

namespace cccl {

namespace {

__device__ __forceinline__ uint32_t pair_abs_max(uint32_t x, uint32_t y) { return vmax_u16x2(x & 0x7FFF7FFFu, y); }

// 16 values as codes.  INT8: adding 1.5 * 2^23 rounds a value below 2^22 to an
// integer, ties to even, and leaves it in the sum's low bits.
template <class T, int FMT>
__device__ __forceinline__ uint4 encode16(const uint4* x, float inv) {
    const uint32_t w[8] = {x[0].x, x[0].y, x[0].z, x[0].w, x[1].x, x[1].y, x[1].z, x[1].w};
    uint32_t c[4];
#pragma unroll
    for (int h = 0; h < 4; ++h) {
        float y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t word = w[2 * h + i / 2];
            y[i] = T::load((uint16_t)((i & 1) ? word >> 16 : word & 0xFFFFu)) * inv;
        }
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
    return make_uint4(c[0], c[1], c[2], c[3]);
}

// Vector `vec` of a block's tokens: K of all of them, then V, token by token and
// head by head, so that what a block touches at a time lies together.
struct VecPlace {
    int tok, head;
    bool is_v;
};
__device__ __forceinline__ VecPlace vec_place(const FastDiv& heads, int count, int vec) {
    const int half = count * (int)heads.d;
    const bool is_v = vec >= half;
    const int r = is_v ? vec - half : vec, tok = (int)div_by(heads, (uint32_t)r);
    return VecPlace{tok, r - tok * (int)heads.d, is_v};
}

// (One vector a lane group at a time: with two or four in flight the read fell
// from 6.1 to 5.7 and 4.2 TB/s, 131072 tokens of 8 heads of 128, INT8.)
template <class T, int FMT, int G>
__global__ void __launch_bounds__(kCopyThreads) kv_write_kernel(const __grid_constant__ KvArgs a,
                                                                const __grid_constant__ KvPacked x, FastDiv heads,
                                                                int tokens) {
    __shared__ TokenSlots slots;
    const int64_t t0 = (int64_t)blockIdx.x * tokens;
    const int count = (int)min((int64_t)tokens, a.n_tokens - t0);
    find_slots(a, t0, count, slots);
    const int part = threadIdx.x % G;
    const bool inside = 16 * part < a.dim;
    const int total = 2 * count * (int)heads.d;
    __syncthreads();
    for (int base = 0; base < total; base += kCopyThreads / G) {
        const int vec = base + threadIdx.x / G;
        const VecPlace p = vec_place(heads, count, vec);
        const bool live = vec < total && slots.state[p.tok] == 1;
        uint4 val[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
        if (live && inside) {
            const uint8_t* src = p.is_v ? x.v + (t0 + p.tok) * x.v_token + p.head * x.v_head
                                        : x.k + (t0 + p.tok) * x.k_token + p.head * x.k_head;
            val[0] = load_stream(src + 32 * part);
            val[1] = load_stream(src + 32 * part + 16);
        }
        uint8_t* const row = (p.is_v ? a.v : a.k) + slots.at[live ? p.tok : 0] + p.head * a.head_stride;
        if (FMT == kKv16Bit) {
            if (live && inside) {
                *reinterpret_cast<uint4*>(row + 32 * part) = val[0];
                *reinterpret_cast<uint4*>(row + 32 * part + 16) = val[1];
            }
            continue;
        }
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            m = pair_abs_max(val[i].x, m);
            m = pair_abs_max(val[i].y, m);
            m = pair_abs_max(val[i].z, m);
            m = pair_abs_max(val[i].w, m);
        }
#pragma unroll
        for (int o = G / 2; o > 0; o >>= 1) m = vmax_u16x2(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        const float amax = T::load((uint16_t)max(m & 0xFFFFu, m >> 16));
        constexpr float kLimit = FMT == kKvInt8 ? 127.f : 448.f;
        // inv is limited to the largest finite number, so that a subnormal
        // maximum does not turn zeros into NaN
        const float inv = amax == 0.f ? 0.f : fminf(kLimit / amax, 3.402823466e+38f);
        if (live) {
            if (inside) *reinterpret_cast<uint4*>(row + 16 * part) = encode16<T, FMT>(val, inv);
            if (part == 0)
                (p.is_v ? a.v_scale : a.k_scale)[slots.scale_at[p.tok] + p.head * a.s_head] =
                    amax <= 3.402823466e+38f ? amax / kLimit : __uint_as_float(0x7FC00000u);
        }
    }
}

// 16 codes -> 16 values of 16 bits: to fp16 exactly, then code * scale rounded once.
template <class T, int FMT>
__device__ __forceinline__ void decode16(const uint4& c, float scale, uint4* y) {
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
    uint32_t v[8];
#pragma unroll
    for (int h = 0; h < 4; ++h) {
        uint32_t p[2];
        expand4_in_order<FMT>(w[h], p[0], p[1]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&p[i]));
            v[2 * h + i] = round_pair<T>(f.x * scale, f.y * scale);
        }
    }
    y[0] = make_uint4(v[0], v[1], v[2], v[3]);
    y[1] = make_uint4(v[4], v[5], v[6], v[7]);
}

template <class T, int FMT, int G>
__global__ void __launch_bounds__(kCopyThreads) kv_read_kernel(const __grid_constant__ KvArgs a,
                                                               const __grid_constant__ KvPacked x, FastDiv heads,
                                                               int tokens) {
    __shared__ TokenSlots slots;
    const int64_t t0 = (int64_t)blockIdx.x * tokens;
    const int count = (int)min((int64_t)tokens, a.n_tokens - t0);
    find_slots(a, t0, count, slots);
    const int part = threadIdx.x % G;
    const bool inside = 16 * part < a.dim;
    const int total = 2 * count * (int)heads.d;
    __syncthreads();
    for (int vec = threadIdx.x / G; vec < total; vec += kCopyThreads / G) {
        const VecPlace p = vec_place(heads, count, vec);
        const int state = slots.state[p.tok];
        if (state == 0 || !inside) continue;
        uint4 y[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
        if (state == 1) {
            const uint8_t* src = (p.is_v ? a.v : a.k) + slots.at[p.tok] + p.head * a.head_stride;
            if (FMT == kKv16Bit) {
                y[0] = load_stream(src + 32 * part);
                y[1] = load_stream(src + 32 * part + 16);
            } else {
                const uint4 c = load_stream(src + 16 * part);
                decode16<T, FMT>(c, (p.is_v ? a.v_scale : a.k_scale)[slots.scale_at[p.tok] + p.head * a.s_head], y);
            }
        }
        uint8_t* dst = p.is_v ? x.v + (t0 + p.tok) * x.v_token + p.head * x.v_head
                              : x.k + (t0 + p.tok) * x.k_token + p.head * x.k_head;
        __stcs(reinterpret_cast<uint4*>(dst + 32 * part), y[0]);
        __stcs(reinterpret_cast<uint4*>(dst + 32 * part + 16), y[1]);
    }
}

template <class T, int FMT>
cudaError_t write_one(const KvArgs& a, const KvPacked& x, cudaStream_t s) {
    const int tpb = tokens_per_block(a.n_tokens);
    const FastDiv heads = fast_div((uint32_t)a.kv_heads);
    const dim3 grid((unsigned)((a.n_tokens + tpb - 1) / tpb));
    if (a.dim <= 64)
        kv_write_kernel<T, FMT, 4><<<grid, kCopyThreads, 0, s>>>(a, x, heads, tpb);
    else
        kv_write_kernel<T, FMT, 8><<<grid, kCopyThreads, 0, s>>>(a, x, heads, tpb);
    return cudaGetLastError();
}
template <class T, int FMT>
cudaError_t read_one(const KvArgs& a, const KvPacked& x, cudaStream_t s) {
    const int tpb = tokens_per_block(a.n_tokens);
    const FastDiv heads = fast_div((uint32_t)a.kv_heads);
    const dim3 grid((unsigned)((a.n_tokens + tpb - 1) / tpb));
    if (a.dim <= 64)
        kv_read_kernel<T, FMT, 4><<<grid, kCopyThreads, 0, s>>>(a, x, heads, tpb);
    else
        kv_read_kernel<T, FMT, 8><<<grid, kCopyThreads, 0, s>>>(a, x, heads, tpb);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv_write(int dtype, int format, const KvArgs& a, const KvPacked& x, cudaStream_t s) {
    if (format == kKv16Bit) return write_one<BfType, kKv16Bit>(a, x, s);  // a copy: the type does not matter
    if (dtype == (int)Bf16::kCode)
        return format == kKvInt8 ? write_one<BfType, kKvInt8>(a, x, s) : write_one<BfType, kKvE4m3>(a, x, s);
    return format == kKvInt8 ? write_one<HfType, kKvInt8>(a, x, s) : write_one<HfType, kKvE4m3>(a, x, s);
}
cudaError_t launch_kv_read(int dtype, int format, const KvArgs& a, const KvPacked& x, cudaStream_t s) {
    if (format == kKv16Bit) return read_one<BfType, kKv16Bit>(a, x, s);
    if (dtype == (int)Bf16::kCode)
        return format == kKvInt8 ? read_one<BfType, kKvInt8>(a, x, s) : read_one<BfType, kKvE4m3>(a, x, s);
    return format == kKvInt8 ? read_one<HfType, kKvInt8>(a, x, s) : read_one<HfType, kKvE4m3>(a, x, s);
}

}  // namespace cccl
