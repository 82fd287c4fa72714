#include "kv_sched.cuh"
namespace ssd {
bool kv_attention_tc_supported(const kv_attention_args &a) { return false; }
size_t kv_attention_tc_workspace(const kv_attention_args &a) { return 0; }
cudaError_t kv_attention_tc_launch(const kv_attention_args &a, void *, cudaStream_t) { return cudaErrorNotSupported; }
}
