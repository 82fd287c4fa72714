// Internal declarations of the attention-side calls (kv_*).
#pragma once
#include "common.cuh"

namespace ssd {
cudaError_t kv_tables_launch(const kv_tables_args &a, cudaStream_t s);
cudaError_t kv_qk_launch(const kv_qk_args &a, cudaStream_t s);
cudaError_t kv_commit_launch(const kv_commit_args &a, cudaStream_t s);

// The two attention kernels; both follow the schedule of kv_sched.cuh.
bool kv_attention_tc_supported(const kv_attention_args &a);
size_t kv_attention_tc_workspace(const kv_attention_args &a);
cudaError_t kv_attention_tc_launch(const kv_attention_args &a, void *workspace, cudaStream_t s);
size_t kv_attention_simt_workspace(const kv_attention_args &a);
cudaError_t kv_attention_simt_launch(const kv_attention_args &a, void *workspace, cudaStream_t s);
}  // namespace ssd
