// Paged attention kernels of one pair of types (ep_attention_kernel.cuh).
#include "ep_attention_kernel.cuh"

namespace ep {
namespace attn {

cudaError_t launch_bf16_e4m3(const AttentionArgs& a, int sms, cudaStream_t stream) { return launch_type<__nv_bfloat16, true>(a, sms, stream); }

}  // namespace attn
}  // namespace ep
