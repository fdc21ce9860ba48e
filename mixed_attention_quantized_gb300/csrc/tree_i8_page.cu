// tree_i8_page.cu -- the mixed-batch attention kernels with tree rows for the
// page-scaled format MIXATTN_KV_I8_PAGE.
#include "page_attention.cuh"

namespace mixattn {

cudaError_t launch_tree_attention_i8_page(int head_dim, const AttnParams& p, unsigned int* err, cudaStream_t s) {
  if (head_dim == 64) return launch_page_attention_t<MIXATTN_KV_I8_PAGE, 64, true>(p, err, s);
  return launch_page_attention_t<MIXATTN_KV_I8_PAGE, 128, true>(p, err, s);
}

}  // namespace mixattn
