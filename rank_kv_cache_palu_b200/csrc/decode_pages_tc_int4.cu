// Sparse decode step, int4 latents (r_k = r_v = 256): instantiations of
// decode_pages_kernel.cuh, apart from the 16-bit ones as the dense kernel's are.
#include "decode_pages_kernel.cuh"

namespace palu {

cudaError_t launch_decode_pages_tc_int4(const DecodeArgs& a, cudaStream_t st) {
  if (a.r_k != 256 || a.r_v != 256) return cudaErrorInvalidValue;
  return a.act == PALU_BF16 ? launch_pages_t<PALU_BF16, 2, PALU_INT4>(a, st)
                            : launch_pages_t<PALU_F16, 2, PALU_INT4>(a, st);
}

}  // namespace palu
