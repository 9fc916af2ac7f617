// cccl_kv_tokens.cu -- the kernels of cccl_kv_tokens.cuh for causal attention.
#include "cccl_kv_tokens.cuh"

namespace cccl {

size_t kv_tokens_scratch(int dim) { return part_bytes(kMaxShares, 16, dim); }

cudaError_t launch_kv_tokens(int dtype, int format, const KvArgs& a, const AttnArgs& t, int max_new, int max_len,
                             cudaStream_t s) {
    return launch_any(dtype, format, a, t, max_new, max_len, s);
}

}  // namespace cccl
