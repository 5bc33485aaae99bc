// Tensor-core split kernel over a list of pages, int4 latents (r_k = r_v = 256);
// see decode_pages_tc.cu.
#include "decode_tc_kernel.cuh"

namespace palu {

cudaError_t launch_decode_pages_tc_int4(const DecodeArgs& a, cudaStream_t st) {
  if (a.r_k != 256 || a.r_v != 256) return cudaErrorInvalidValue;
  return a.act == PALU_BF16 ? launch_t<PALU_BF16, 2, PALU_INT4, true>(a, st)
                            : launch_t<PALU_F16, 2, PALU_INT4, true>(a, st);
}

}  // namespace palu
