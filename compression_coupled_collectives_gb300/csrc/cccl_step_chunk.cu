// cccl_step_chunk.cu -- the kernels of cccl_kv_chunk.cuh for drafted tokens, whose
// masks say which of them see which.
#include "cccl_kv_chunk.cuh"

namespace cccl {

cudaError_t launch_step_chunk(int dtype, int format, const KvArgs& a, const TreeArgs& t, int max_new, int max_len,
                              cudaStream_t s) {
    return launch_any(dtype, format, a, t, max_new, max_len, s);
}

}  // namespace cccl
