// Fused decode for attention without rotary embedding: the walk over every page
// of a sequence (kernel in decode_fused_kernel.cuh), the shape check and dispatch.
//
// Method: "PALU 论文低秩投影分解" §低秩投影分解 and §把它放进一次真实推理流程里看,
// Decode 阶段 (attention fused with the up-projection).
#include "decode_fused_kernel.cuh"

namespace palu {
namespace {

// A pass serves exactly 1, 2 or 4 queries of every sequence (the caller splits
// a step's queries into such passes).
template <int ACT, int NRV>
cudaError_t launch_q(const DecodeArgs& a, cudaStream_t st) {
  if (a.qn == 1) return launch_t<ACT, NRV, 1>(a, st);
  if (a.qn == 2) return launch_t<ACT, NRV, 2>(a, st);
  if (a.qn == 4) return launch_t<ACT, NRV, 4>(a, st);
  return cudaErrorInvalidValue;
}

}  // namespace

bool fused_decode_supported(const palu_config* c) {
  if (c->rope_base != 0.f) return false;
  if (c->page_size != kTile || c->head_dim > 128 || c->head_dim % 8 != 0 || c->group_size > kMaxG) return false;
  if (c->act_dtype != PALU_F16 && c->act_dtype != PALU_BF16) return false;
  if (c->latent_dtype != c->act_dtype) return false;
  if (c->rank_k % 64 != 0 || c->rank_k > 512) return false;
  if (c->rank_v != 128 && c->rank_v != 256) return false;
  return smem_layout<kFusedMaxQueries>(c->rank_k).total + 1024 <= 227 * 1024;
}

int fused_queries_per_pass() { return kFusedMaxQueries; }

size_t fused_query_bytes(const palu_config* c, int batch) {
  const size_t G = (size_t)(c->num_heads / c->group_size);
  return (size_t)batch * G * 2 * kMaxG * c->rank_k * 2;
}

cudaError_t launch_decode_fused(const DecodeArgs& a, cudaStream_t st) {
  if (a.page_list != nullptr) return launch_decode_pages_fused(a, st);
  if (a.act == PALU_BF16) return a.r_v == 256 ? launch_q<PALU_BF16, 2>(a, st) : launch_q<PALU_BF16, 1>(a, st);
  return a.r_v == 256 ? launch_q<PALU_F16, 2>(a, st) : launch_q<PALU_F16, 1>(a, st);
}

}  // namespace palu
