// cccl_step_keep.cu -- kept tokens' keys and values moved together, in place.
//
// The k-th kept token moves from place path[k] >= k to place k of the sequence's
// new ones.  A place k is never a later token's source (path[j] >= j > k), so a
// thread that loads some tokens' 16 bytes, stores them, and goes on to the next
// ones never reads what it has overwritten; every thread has 16 bytes of a head
// of its own.  A few hundred bytes a sequence: the launch and the chain of loads
// (rows, path, page, value) are the time: 3.2 us for 64 sequences' paths of up to 7,
// 5.3 for 512 of up to 16 (8 heads of 128 in E4M3; floor 2.4).
#include "cccl_kv_launch.h"
#include "cccl_step.cuh"

namespace cccl {

namespace {

constexpr int kThreads = 128, kGroup = 32;  // tokens looked up at a time
constexpr int kFlight = 8;                  // loads in flight

__global__ void __launch_bounds__(kThreads) keep_kernel(const __grid_constant__ KvArgs a,
                                                        const __grid_constant__ KeepArgs x, int elem, int scales) {
    __shared__ int64_t from[kGroup], to[kGroup], scale_from[kGroup], scale_to[kGroup];
    const int b = blockIdx.x;
    const Sequence s = load_sequence(a, b);
    const int32_t before = s.len - s.n;
    int32_t n = x.n_kept[b];
    if (n < 0 || n > s.n) {
        if (threadIdx.x == 0) record_error(a.ws, kStatusInvalidArg);
        n = min(max(n, 0), s.n);
    }
    if (blockIdx.y == 0 && threadIdx.x == 0 && x.lens != nullptr) x.lens[b] = max(before + n, 0);
    // 16-byte pieces of a token: K of all heads, then V, then the scales (4 bytes each)
    const int chunks = a.dim * elem / 16, vectors = 2 * a.kv_heads, units = vectors * chunks + (scales ? vectors : 0);
    const int u = (int)blockIdx.y * kThreads + (int)threadIdx.x;
    const bool scale = u >= vectors * chunks;
    const int vec = scale ? u - vectors * chunks : u / chunks;
    const bool is_v = vec >= a.kv_heads;
    const int head = is_v ? vec - a.kv_heads : vec;
    uint8_t* const data = (is_v ? a.v : a.k) + head * a.head_stride + 16 * (u - vec * chunks);
    float* const table = (is_v ? a.v_scale : a.k_scale) + head * a.s_head;
    for (int32_t base = 0; base < n; base += kGroup) {
        const int count = min(kGroup, n - base);
        if ((int)threadIdx.x < count) {
            const int32_t k = base + (int32_t)threadIdx.x, i = x.path[s.row + k];
            bool ok = i >= k && i < s.n;
            if (!ok) record_error(a.ws, kStatusInvalidArg);
            ok = ok && i != k && before + k >= 0;
            int64_t f = 0, fs = 0, t = 0, ts = 0;
            if (ok) {
                ok = slot_of(a, b, (uint32_t)(before + i), f, fs);
                ok = slot_of(a, b, (uint32_t)(before + k), t, ts) && ok;
            }
            from[threadIdx.x] = f;
            to[threadIdx.x] = ok ? t : -1;
            scale_from[threadIdx.x] = fs;
            scale_to[threadIdx.x] = ts;
        }
        __syncthreads();
        if (u < units) {
            for (int k = 0; k < count; k += kFlight) {
                if (scale) {
                    float v[kFlight];
#pragma unroll
                    for (int j = 0; j < kFlight; ++j)
                        if (k + j < count && to[k + j] >= 0) v[j] = table[scale_from[k + j]];
#pragma unroll
                    for (int j = 0; j < kFlight; ++j)
                        if (k + j < count && to[k + j] >= 0) table[scale_to[k + j]] = v[j];
                } else {
                    uint4 v[kFlight];
#pragma unroll
                    for (int j = 0; j < kFlight; ++j)
                        if (k + j < count && to[k + j] >= 0) v[j] = *reinterpret_cast<const uint4*>(data + from[k + j]);
#pragma unroll
                    for (int j = 0; j < kFlight; ++j)
                        if (k + j < count && to[k + j] >= 0) *reinterpret_cast<uint4*>(data + to[k + j]) = v[j];
                }
            }
        }
        __syncthreads();
    }
}

}  // namespace

cudaError_t launch_step_keep(int format, const KvArgs& a, const KeepArgs& x, cudaStream_t s) {
    const int elem = format == kKv16Bit ? 2 : 1, scales = format == kKv16Bit ? 0 : 1;
    const int units = 2 * a.kv_heads * (a.dim * elem / 16 + scales);
    keep_kernel<<<dim3((unsigned)a.batch, (unsigned)((units + kThreads - 1) / kThreads)), kThreads, 0, s>>>(a, x, elem,
                                                                                                         scales);
    return cudaGetLastError();
}

}  // namespace cccl
