// tree_q4_q4.cu -- the mixed-batch attention kernels with tree rows for K format
// MIXATTN_KV_Q4_0 and V format MIXATTN_KV_Q4_0.
#include "attention_kernel.cuh"

namespace mixattn {

cudaError_t launch_tree_attention_q4_q4(int head_dim, const AttnParams& p, unsigned int* err, cudaStream_t s) {
  if (head_dim == 64) return launch_attention_t<MIXATTN_KV_Q4_0, MIXATTN_KV_Q4_0, 64, true>(p, err, s);
  return launch_attention_t<MIXATTN_KV_Q4_0, MIXATTN_KV_Q4_0, 128, true>(p, err, s);
}

}  // namespace mixattn
