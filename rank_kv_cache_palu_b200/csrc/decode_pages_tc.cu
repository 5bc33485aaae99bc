// Sparse decode step, 16-bit latents: instantiations of decode_pages_kernel.cuh.
#include "decode_pages_kernel.cuh"

namespace palu {

cudaError_t launch_decode_pages_tc(const DecodeArgs& a, cudaStream_t st) {
  if (a.act == PALU_BF16)
    return a.r_v == 256 ? launch_pages_t<PALU_BF16, 2, PALU_BF16>(a, st)
                        : launch_pages_t<PALU_BF16, 1, PALU_BF16>(a, st);
  return a.r_v == 256 ? launch_pages_t<PALU_F16, 2, PALU_F16>(a, st) : launch_pages_t<PALU_F16, 1, PALU_F16>(a, st);
}

}  // namespace palu
