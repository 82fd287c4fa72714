// Internal declarations of the attention-side calls (kv_*).
#pragma once
#include "common.cuh"

namespace ssd {
// SMs of the current device (152 on GB300, also where the attribute cannot be read).
inline int device_sms() {
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 152;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms <= 0) return 152;
    return sms;
}

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
