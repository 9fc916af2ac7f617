// cccl_kv_attention.cu -- which attention kernel a call takes.
#include "cccl_kv.cuh"
#include "cccl_kv_launch.h"

namespace cccl {

// Few rows a kv head (query heads that share it x new tokens): the token kernel
// reads the cache once for every 16 of them and keeps up with HBM.  More: the
// chunk kernel reads it once for 256, but brings 128 or 256 rows to the tensor
// cores however many are real, and widens 8-bit codes on the way.  32 sequences
// of up to 4096 tokens, 8 kv heads of 128, in us (token kernel, chunk kernel):
//   16-bit cache  20 rows 85, 98;  32 rows 100, 93;  64 rows 158, 93
//   INT8 cache    32 rows 111, 152;  64 rows 175, 153
// Drafted trees go by the same rule, since one workspace serves both kinds of call.
// Their chunk kernel is the faster one from fewer rows on (token kernel, chunk kernel):
//   16-bit, 32 of up to 4096   16 rows 80, 86;  20 rows 87, 85;  24 rows 96, 83
//   16-bit, 4 of up to 2000    8 rows 15.9, 17.4;  16 rows 23.3, 17.5;  24 rows 25.9, 17.7
//   16-bit, one of 517         16 rows 10.6, 14.6;  24 rows 12.1, 14.3
//   INT8, 32 of up to 4096     32 rows 127, 181;  48 rows 149, 179;  64 rows 195, 187
//   INT8, 8 of up to 20480     28 rows 135, 144;  32 rows 154, 150;  40 rows 185, 151
//   INT8, one of 517           32 rows 15.5, 19.9
static bool few_rows(int format, int group, int max_new) {
    return (int64_t)group * max_new <= (format == kKv16Bit ? 24 : 32);
}

size_t kv_attention_scratch(int format, int dim, int group, int max_new) {
    return few_rows(format, group, max_new) ? kv_tokens_scratch(dim) : kv_chunk_scratch(dim);
}

cudaError_t launch_kv_attention(int dtype, int format, const KvArgs& a, const AttnArgs& t, int max_new, int max_len,
                                cudaStream_t s) {
    return few_rows(format, (int)t.group.d, max_new) ? launch_kv_tokens(dtype, format, a, t, max_new, max_len, s)
                                                     : launch_kv_chunk(dtype, format, a, t, max_new, max_len, s);
}

cudaError_t launch_step_attention(int dtype, int format, const KvArgs& a, const TreeArgs& t, int max_new, int max_len,
                                  cudaStream_t s) {
    return few_rows(format, (int)t.group.d, max_new) ? launch_step_tokens(dtype, format, a, t, max_new, max_len, s)
                                                     : launch_step_chunk(dtype, format, a, t, max_new, max_len, s);
}

}  // namespace cccl
