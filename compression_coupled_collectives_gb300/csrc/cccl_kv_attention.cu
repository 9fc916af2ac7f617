// cccl_kv_attention.cu -- which attention kernel a call takes.
#include "cccl_kv.cuh"
#include "cccl_kv_launch.h"

namespace cccl {

// Few rows a kv head: one read of the cache, whose rate mma.sync keeps up with.
// More rows: the tensor cores.
static bool few_rows(int group, int max_new) { return (int64_t)group * max_new <= 16; }

size_t kv_attention_scratch(int dim, int group, int max_new, int) {
    return few_rows(group, max_new) ? kv_tokens_scratch(dim) : kv_chunk_scratch(dim);
}

cudaError_t launch_kv_attention(int dtype, int format, const KvArgs& a, const AttnArgs& t, int max_new, int max_len,
                                cudaStream_t s) {
    return few_rows((int)t.group.d, max_new) ? launch_kv_tokens(dtype, format, a, t, max_new, max_len, s)
                                      : launch_kv_chunk(dtype, format, a, t, max_new, max_len, s);
}

}  // namespace cccl
