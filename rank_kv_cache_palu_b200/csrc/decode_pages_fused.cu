// Fused decode without rotary embedding over a list of pages per query and group
// (palu_decode_attn_pages): the SPARSE instantiations of decode_fused_kernel.cuh,
// apart from the dense ones so that neither's code moves the other's.
#include "decode_fused_kernel.cuh"

namespace palu {

cudaError_t launch_decode_pages_fused(const DecodeArgs& a, cudaStream_t st) {
  if (a.qn != 1) return cudaErrorInvalidValue;
  if (a.act == PALU_BF16)
    return a.r_v == 256 ? launch_t<PALU_BF16, 2, 1, true>(a, st) : launch_t<PALU_BF16, 1, 1, true>(a, st);
  return a.r_v == 256 ? launch_t<PALU_F16, 2, 1, true>(a, st) : launch_t<PALU_F16, 1, 1, true>(a, st);
}

}  // namespace palu
