// attention_i8_page.cu -- instantiation of the mixed-batch attention kernels for the
// page-scaled format MIXATTN_KV_I8_PAGE (one translation unit per format so the build
// compiles them in parallel).
#include "page_attention.cuh"

namespace mixattn {

cudaError_t launch_attention_i8_page(int head_dim, const AttnParams& p, unsigned int* err, cudaStream_t s) {
  if (head_dim == 64) return launch_page_attention_t<MIXATTN_KV_I8_PAGE, 64>(p, err, s);
  return launch_page_attention_t<MIXATTN_KV_I8_PAGE, 128>(p, err, s);
}

}  // namespace mixattn
