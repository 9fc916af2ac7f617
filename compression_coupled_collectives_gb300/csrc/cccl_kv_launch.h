// cccl_kv_launch.h -- launchers of the paged cache kernels (host side, internal).
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

namespace cccl {

struct KvArgs;
struct KvPacked;
struct AttnArgs;

// dtype: 1 bf16, 2 fp16; format: CCCL_KV_*.  All arguments are checked.
cudaError_t launch_kv_write(int dtype, int format, const KvArgs& a, const KvPacked& x, cudaStream_t stream);
cudaError_t launch_kv_read(int dtype, int format, const KvArgs& a, const KvPacked& x, cudaStream_t stream);
cudaError_t launch_kv_attention(int dtype, int format, const KvArgs& a, const AttnArgs& t, int max_new, int max_len,
                                cudaStream_t stream);
// The kernel for few rows a kv head, and its workspace bytes after the header.
cudaError_t launch_kv_tokens(int dtype, int format, const KvArgs& a, const AttnArgs& t, int max_new, int max_len,
                             cudaStream_t stream);
size_t kv_tokens_scratch(int dim);
// The kernel for chunks of rows, and its workspace bytes after the header.
cudaError_t launch_kv_chunk(int dtype, int format, const KvArgs& a, const AttnArgs& t, int max_new, int max_len,
                            cudaStream_t stream);
size_t kv_chunk_scratch(int dim);
// Workspace bytes of an attention call after the 16-byte header.
size_t kv_attention_scratch(int format, int dim, int group, int max_new);

}  // namespace cccl
