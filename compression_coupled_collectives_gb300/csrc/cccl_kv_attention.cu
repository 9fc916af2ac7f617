// cccl_kv_attention.cu -- attention over the paged cache: one warp a row and
// query head.
#include "cccl_kv.cuh"
#include "cccl_kv_launch.h"

namespace cccl {

namespace {

constexpr int kRowThreads = 128;

template <class T, int FMT>
__global__ void __launch_bounds__(kRowThreads) attend_rows_kernel(const __grid_constant__ KvArgs a,
                                                                  const __grid_constant__ AttnArgs t) {
    const int b = blockIdx.y;
    const Sequence s = load_sequence(a, b);
    const int64_t rows = (int64_t)s.n * t.q_heads, step = (int64_t)gridDim.x * (kRowThreads / 32);
    for (int64_t r = (int64_t)blockIdx.x * (kRowThreads / 32) + threadIdx.x / 32; r < rows; r += step) {
        const int64_t i = r / t.q_heads;
        attend_row<T, FMT>(a, t, b, s.len, s.row + i, (int64_t)s.len - s.n + i, (int)(r - i * t.q_heads));
    }
}

template <class T, int FMT>
cudaError_t rows_one(const KvArgs& a, const AttnArgs& t, cudaStream_t s) {
    attend_rows_kernel<T, FMT><<<dim3(256, (unsigned)a.batch), kRowThreads, 0, s>>>(a, t);
    return cudaGetLastError();
}

}  // namespace

size_t kv_attention_scratch(int dim, int group, int max_new, int) {
    return (int64_t)group * max_new <= 16 ? kv_tokens_scratch(dim) : kv_chunk_scratch(dim);
}

cudaError_t launch_kv_attention(int dtype, int format, const KvArgs& a, const AttnArgs& t, int max_new, int max_len,
                                cudaStream_t s) {
    if ((int64_t)t.group * max_new <= 16) return launch_kv_tokens(dtype, format, a, t, max_len, s);
    if (format == kKv16Bit) return launch_kv_chunk(dtype, format, a, t, max_len, s);
    if (dtype == (int)Bf16::kCode) {
        if (format == kKv16Bit) return rows_one<BfType, kKv16Bit>(a, t, s);
        return format == kKvInt8 ? rows_one<BfType, kKvInt8>(a, t, s) : rows_one<BfType, kKvE4m3>(a, t, s);
    }
    if (format == kKv16Bit) return rows_one<HfType, kKv16Bit>(a, t, s);
    return format == kKvInt8 ? rows_one<HfType, kKvInt8>(a, t, s) : rows_one<HfType, kKvE4m3>(a, t, s);
}

}  // namespace cccl
