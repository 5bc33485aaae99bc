// Tensor-core split kernel over a list of pages per query and group
// (palu_decode_attn_pages): the SPARSE instantiations of decode_tc_kernel.cuh,
// apart from the dense ones so that neither's code moves the other's.
//
// Method: "PALU 论文低秩投影分解" §把它放进一次真实推理流程里看, Decode 阶段 (keys
// rebuilt from the cached latents tile by tile, values kept in latent space).
#include "decode_tc_kernel.cuh"

namespace palu {

cudaError_t launch_decode_pages_tc(const DecodeArgs& a, cudaStream_t st) {
  if (a.act == PALU_BF16)
    return a.r_v == 256 ? launch_t<PALU_BF16, 2, PALU_BF16, true>(a, st)
                        : launch_t<PALU_BF16, 1, PALU_BF16, true>(a, st);
  return a.r_v == 256 ? launch_t<PALU_F16, 2, PALU_F16, true>(a, st)
                      : launch_t<PALU_F16, 1, PALU_F16, true>(a, st);
}

}  // namespace palu
