// cccl_kv_copy.cu -- storing tokens in the paged cache and taking them out
// again.  Both are one pass over the data and bound by HBM: a token and head
// moves 2 D bytes on the packed side and D or 2 D (and a 4-byte scale) on the
// cache's.
//
// A vector (token, head, K or V) belongs to a group of G lanes, 8 values a
// lane on a write and on a 16-bit read (16-byte accesses on the packed side).
// The maximum is taken over the patterns of |x| as integers, two values per
// instruction: for non-negative 16-bit floats the order of the patterns is the
// order of the values, and a NaN's pattern lies above infinity's, so a NaN
// stays the maximum.
#include "cccl_kv.cuh"
#include "cccl_kv_launch.h"

namespace cccl {

namespace {

constexpr int kCopyThreads = 256;
constexpr int kMaxTokensPerBlock = 16;
constexpr int kUnroll = 4;  // vectors a lane group keeps in flight

// Tokens t0 .. t0 + count - 1 of a block: where each lies in the cache, and
// whether it lies there at all.
struct TokenSlots {
    int64_t at[kMaxTokensPerBlock], scale_at[kMaxTokensPerBlock];
    int8_t state[kMaxTokensPerBlock];  // 0 no sequence's row, 1 in the cache, 2 not in the cache
};
__device__ __forceinline__ void find_slots(const KvArgs& a, int64_t t0, int count, TokenSlots& s) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int i = warp; i < count; i += kCopyThreads / 32) {
        const int64_t t = t0 + i;
        // the last sequence that starts at or before t: 32 candidates a step
        int lo = 0, hi = a.batch;  // starts at lo, or no sequence does
        while (hi - lo > 1) {
            const int step = (hi - lo + 31) / 32;
            const int c = lo + lane * step;
            const uint32_t le = __ballot_sync(0xFFFFFFFFu, c < hi && (lane == 0 || a.cu[c] <= t));
            const int at = 31 - __clz(le);
            lo += at * step;
            hi = min(hi, lo + step);
        }
        if (lane == 0) {
            const Sequence q = load_sequence(a, lo);
            int state = 0;
            int64_t at = 0, sat = 0;
            if (t >= q.row && t < q.row + q.n) {
                const int64_t pos = (int64_t)q.len - q.n + (t - q.row);
                state = pos >= 0 && slot_of(a, lo, (uint32_t)pos, at, sat) ? 1 : 2;
            }
            s.at[i] = at;
            s.scale_at[i] = sat;
            s.state[i] = (int8_t)state;
        }
    }
}

__device__ __forceinline__ uint4 load_stream(const void* p) {
    return __ldcs(reinterpret_cast<const uint4*>(p));
}
__device__ __forceinline__ uint32_t pair_abs_max(uint32_t x, uint32_t y) { return vmax_u16x2(x & 0x7FFF7FFFu, y); }

template <class T, int FMT>
__device__ __forceinline__ uint2 encode8(const uint4& x, float inv) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    uint32_t c[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t word = w[2 * h + i / 2];
            y[i] = T::load((uint16_t)((i & 1) ? word >> 16 : word & 0xFFFFu)) * inv;
        }
        if (FMT == kKvInt8) {
            uint32_t r = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int v = __float2int_rn(y[i]);  // 0 for a NaN
                r |= ((uint32_t)min(max(v, -127), 127) & 0xFFu) << (8 * i);
            }
            c[h] = r;
        } else {
            const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(y[0], y[1]), __NV_SATFINITE, __NV_E4M3);
            const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(y[2], y[3]), __NV_SATFINITE, __NV_E4M3);
            c[h] = lo | (hi << 16);
        }
    }
    return make_uint2(c[0], c[1]);
}

// G lanes hold one vector, 8 values each.
template <class T, int FMT, int G>
__global__ void __launch_bounds__(kCopyThreads) kv_write_kernel(const __grid_constant__ KvArgs a,
                                                                const __grid_constant__ KvPacked x, int tokens) {
    __shared__ TokenSlots slots;
    const int64_t t0 = (int64_t)blockIdx.x * tokens;
    const int count = (int)min((int64_t)tokens, a.n_tokens - t0);
    find_slots(a, t0, count, slots);
    __syncthreads();
    const int part = threadIdx.x % G;
    const bool inside = 8 * part < a.dim;
    const int per_token = 2 * a.kv_heads;  // K of every head, then V of every head
    const int total = count * per_token;
    constexpr int kGroups = kCopyThreads / G;
    for (int base = threadIdx.x / G; base - (int)(threadIdx.x / G) < total; base += kGroups * kUnroll) {
        uint4 val[kUnroll];
        int tok[kUnroll], head[kUnroll];
        bool live[kUnroll], is_v[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int vec = base + u * kGroups;
            tok[u] = vec / per_token;
            const int r = vec - tok[u] * per_token;
            is_v[u] = r >= a.kv_heads;
            head[u] = is_v[u] ? r - a.kv_heads : r;
            live[u] = vec < total && slots.state[tok[u]] == 1;
            val[u] = make_uint4(0, 0, 0, 0);
            if (live[u] && inside) {
                const uint8_t* src = is_v[u] ? x.v + (t0 + tok[u]) * x.v_token + head[u] * x.v_head
                                             : x.k + (t0 + tok[u]) * x.k_token + head[u] * x.k_head;
                val[u] = load_stream(src + 16 * part);
            }
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            if (FMT == kKv16Bit) {
                if (live[u] && inside)
                    *reinterpret_cast<uint4*>((is_v[u] ? a.v : a.k) + slots.at[tok[u]] + head[u] * a.head_stride +
                                              16 * part) = val[u];
                continue;
            }
            uint32_t m = pair_abs_max(val[u].x, 0);
            m = pair_abs_max(val[u].y, m);
            m = pair_abs_max(val[u].z, m);
            m = pair_abs_max(val[u].w, m);
#pragma unroll
            for (int o = G / 2; o > 0; o >>= 1) m = vmax_u16x2(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
            const float amax = T::load((uint16_t)max(m & 0xFFFFu, m >> 16));
            constexpr float kLimit = FMT == kKvInt8 ? 127.f : 448.f;
            // inv is limited to the largest finite number, so that a
            // subnormal maximum does not turn zeros into NaN
            const float inv = amax == 0.f ? 0.f : fminf(kLimit / amax, 3.402823466e+38f);
            if (live[u]) {
                if (inside)
                    *reinterpret_cast<uint2*>((is_v[u] ? a.v : a.k) + slots.at[tok[u]] + head[u] * a.head_stride +
                                              8 * part) = encode8<T, FMT>(val[u], inv);
                if (part == 0)
                    (is_v[u] ? a.v_scale : a.k_scale)[slots.scale_at[tok[u]] + head[u] * a.s_head] = amax / kLimit;
            }
        }
    }
}

// 8 codes -> 8 values of 16 bits
template <class T, int FMT>
__device__ __forceinline__ uint4 decode8(uint32_t lo, uint32_t hi, float scale) {
    uint32_t w[4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t c = h ? hi : lo;
        float y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = code_value<FMT>((uint8_t)(c >> (8 * i))) * scale;
        w[2 * h] = round_pair<T>(y[0], y[1]);
        w[2 * h + 1] = round_pair<T>(y[2], y[3]);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

template <class T, int FMT, int G>
__global__ void __launch_bounds__(kCopyThreads) kv_read_kernel(const __grid_constant__ KvArgs a,
                                                               const __grid_constant__ KvPacked x, int tokens) {
    __shared__ TokenSlots slots;
    const int64_t t0 = (int64_t)blockIdx.x * tokens;
    const int count = (int)min((int64_t)tokens, a.n_tokens - t0);
    find_slots(a, t0, count, slots);
    __syncthreads();
    const int part = threadIdx.x % G;
    const bool inside = 8 * part < a.dim;
    const int per_token = 2 * a.kv_heads;
    const int total = count * per_token;
    constexpr int kGroups = kCopyThreads / G;
    for (int base = threadIdx.x / G; base - (int)(threadIdx.x / G) < total; base += kGroups * kUnroll) {
        uint4 val[kUnroll];
        float scale[kUnroll];
        int tok[kUnroll], head[kUnroll];
        bool live[kUnroll], is_v[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int vec = base + u * kGroups;
            tok[u] = vec / per_token;
            const int r = vec - tok[u] * per_token;
            is_v[u] = r >= a.kv_heads;
            head[u] = is_v[u] ? r - a.kv_heads : r;
            const int state = vec < total ? slots.state[tok[u]] : 0;
            live[u] = state != 0 && inside;
            val[u] = make_uint4(0, 0, 0, 0);
            scale[u] = 1.f;
            if (state == 1 && inside) {
                const uint8_t* src = (is_v[u] ? a.v : a.k) + slots.at[tok[u]] + head[u] * a.head_stride;
                if (FMT == kKv16Bit) {
                    val[u] = load_stream(src + 16 * part);
                } else {
                    const uint2 c = __ldcs(reinterpret_cast<const uint2*>(src + 8 * part));
                    val[u].x = c.x;
                    val[u].y = c.y;
                    scale[u] = (is_v[u] ? a.v_scale : a.k_scale)[slots.scale_at[tok[u]] + head[u] * a.s_head];
                }
            }
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            if (!live[u]) continue;
            uint8_t* dst = is_v[u] ? x.v + (t0 + tok[u]) * x.v_token + head[u] * x.v_head
                                   : x.k + (t0 + tok[u]) * x.k_token + head[u] * x.k_head;
            const uint4 y = FMT == kKv16Bit ? val[u] : decode8<T, FMT>(val[u].x, val[u].y, scale[u]);
            __stcs(reinterpret_cast<uint4*>(dst + 16 * part), y);
        }
    }
}

// Tokens of one block: 1 while that fills the GPU's 152 SMs with 8 blocks
// each, more (fewer searches of the batch per byte) beyond.
int tokens_per_block(int64_t n) {
    const int64_t t = n / (152 * 8);
    return (int)(t < 1 ? 1 : (t > kMaxTokensPerBlock ? kMaxTokensPerBlock : t));
}

template <class T, int FMT>
cudaError_t write_one(const KvArgs& a, const KvPacked& x, cudaStream_t s) {
    const int tpb = tokens_per_block(a.n_tokens);
    const dim3 grid((unsigned)((a.n_tokens + tpb - 1) / tpb));
    if (a.dim <= 64)
        kv_write_kernel<T, FMT, 8><<<grid, kCopyThreads, 0, s>>>(a, x, tpb);
    else
        kv_write_kernel<T, FMT, 16><<<grid, kCopyThreads, 0, s>>>(a, x, tpb);
    return cudaGetLastError();
}
template <class T, int FMT>
cudaError_t read_one(const KvArgs& a, const KvPacked& x, cudaStream_t s) {
    const int tpb = tokens_per_block(a.n_tokens);
    const dim3 grid((unsigned)((a.n_tokens + tpb - 1) / tpb));
    if (a.dim <= 64)
        kv_read_kernel<T, FMT, 8><<<grid, kCopyThreads, 0, s>>>(a, x, tpb);
    else
        kv_read_kernel<T, FMT, 16><<<grid, kCopyThreads, 0, s>>>(a, x, tpb);
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
