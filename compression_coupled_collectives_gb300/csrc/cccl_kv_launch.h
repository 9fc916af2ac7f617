// cccl_kv_launch.h -- launchers of the paged cache kernels (host side, internal).
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

namespace cccl {

struct KvArgs;
struct KvPacked;
struct AttnArgs;
struct TreeArgs;
struct PlanArgs;
struct RotaryArgs;
struct VerifyArgs;
struct KeepArgs;

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
// Attention of drafted tokens: the same kernels with masks.
cudaError_t launch_step_attention(int dtype, int format, const KvArgs& a, const TreeArgs& t, int max_new, int max_len,
                                  cudaStream_t stream);
cudaError_t launch_step_tokens(int dtype, int format, const KvArgs& a, const TreeArgs& t, int max_new, int max_len,
                               cudaStream_t stream);
cudaError_t launch_step_chunk(int dtype, int format, const KvArgs& a, const TreeArgs& t, int max_new, int max_len,
                              cudaStream_t stream);
// Workspace bytes of an attention call after the 16-byte header.
size_t kv_attention_scratch(int format, int dim, int group, int max_new);

// A step with drafted tokens.
cudaError_t launch_step_plan(const PlanArgs& a, cudaStream_t stream);
cudaError_t launch_step_write(int dtype, int format, const KvArgs& a, const KvPacked& x, const RotaryArgs& r,
                              bool interleaved, cudaStream_t stream);
cudaError_t launch_step_verify(const VerifyArgs& a, cudaStream_t stream);
cudaError_t launch_step_keep(int format, const KvArgs& a, const KeepArgs& x, cudaStream_t stream);

}  // namespace cccl
