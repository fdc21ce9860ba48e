// tree_f16_f16.cu -- the mixed-batch attention kernels with tree rows for K format
// MIXATTN_KV_F16 and V format MIXATTN_KV_F16.
#include "attention_kernel.cuh"

namespace mixattn {

cudaError_t launch_tree_attention_f16_f16(int head_dim, const AttnParams& p, unsigned int* err, cudaStream_t s) {
  if (head_dim == 64) return launch_attention_t<MIXATTN_KV_F16, MIXATTN_KV_F16, 64, true>(p, err, s);
  return launch_attention_t<MIXATTN_KV_F16, MIXATTN_KV_F16, 128, true>(p, err, s);
}

}  // namespace mixattn
