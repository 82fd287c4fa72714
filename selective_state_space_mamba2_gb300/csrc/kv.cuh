// Internal declarations of the attention-side calls (kv_*).
#pragma once
#include <atomic>

#include "common.cuh"

namespace ssd {
// SMs of the current device (152 on GB300, also where the attribute cannot be read).  Asked once per
// device: a decode step's call takes a few microseconds in all.
inline int device_sms() {
    static std::atomic<int> known[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 152;
    int sms = known[dev].load(std::memory_order_relaxed);
    if (sms == 0) {
        if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms <= 0) return 152;
        known[dev].store(sms, std::memory_order_relaxed);
    }
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
