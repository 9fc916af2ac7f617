// cccl_kv_chunk.cu -- the kernels of cccl_kv_chunk.cuh for causal attention.
#include "cccl_kv_chunk.cuh"

namespace cccl {

size_t kv_chunk_scratch(int dim) { return part_bytes(kShares, kRows, dim); }

cudaError_t launch_kv_chunk(int dtype, int format, const KvArgs& a, const AttnArgs& t, int max_new, int max_len,
                            cudaStream_t s) {
    return launch_any(dtype, format, a, t, max_new, max_len, s);
}

}  // namespace cccl
