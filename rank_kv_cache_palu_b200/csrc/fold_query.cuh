// Folded queries of attention without rotary embedding: the key up-projection moved
// into the query, shared by the dense and the sparse fused kernels.
#pragma once

#include "palu_common.cuh"
#include "palu_internal.h"

namespace palu {
namespace {

constexpr int kMaxG = 4;            // heads per group the fused kernels take

// q̃ = B_k,h q_h (scaled) for the heads of one group, as hi + lo 16-bit rows:
// out[vb][g][h] = hi, out[vb][g][4 + h] = lo (h < gs; other rows zero), each
// r_k long, for virtual sequence vb = b·qslots + jj (query jj of the pass; a
// single query per step is qslots = 1).  CTA (g, 64 latent entries, 4 virtual
// sequences); thread (entry j, head h) holds the B_k row segment
// B_k[g][j][h·d_h, +d_h) in registers and takes its dot product with each
// query.
constexpr int kFoldSeqs = 4;
// IMAGE: three terms instead of two (rows h, 4 + h, 8 + h: 24 significant bits in bf16, as in
// float32; in f16 what is left below 2^-24 is dropped), stored as the 128-byte-swizzled K-major
// operand they become in shared memory, [64-entry chunk][12 rows][128 bytes], so that a bulk copy
// brings them there (the sparse kernel changes queries as it goes).
constexpr int kFoldTerms = 3;
template <int ACT, bool IMAGE>
__global__ void __launch_bounds__(256) fold_query_kernel(const __grid_constant__ DecodeArgs a, int qslots, void* qt) {
  using TA = typename Dt<ACT>::T;
  if constexpr (IMAGE) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the walk lays out its tiles
  // rows padded by 4 floats: the four heads' 16-byte reads of one warp land in distinct banks
  __shared__ __align__(16) float qs[kFoldSeqs][kMaxG][128 + 4];
  // blockIdx.x: entry gi of the group map (model group g)
  const int gi = blockIdx.x, jb = blockIdx.y, v0 = blockIdx.z * kFoldSeqs;
  const int g = a.gm.g[gi];
  const int r_k = a.gm.rk[gi];          // this entry's key rank; rows are a.r_k apart
  const int gs = a.gs, d_h = a.d_h;
  const int nvb = a.batch * qslots;
  auto live = [&](int vb) { return vb < nvb && vb % qslots < a.qn; };
  for (int i = threadIdx.x; i < kFoldSeqs * kMaxG * 128; i += blockDim.x) {
    const int bb = i / (kMaxG * 128), h = (i / 128) % kMaxG, d = i % 128;
    const int vb = v0 + bb;
    float v = 0.f;
    if (live(vb) && h < gs && d < d_h)
      v = Dt<ACT>::to_f(reinterpret_cast<const TA*>(a.q)[(size_t)(vb / qslots) * a.q_bstride +
                                                          (size_t)(vb % qslots) * a.H * d_h +
                                                          (size_t)(g * gs + h) * d_h + d]);
    qs[bb][h][d] = v;
  }
  __syncthreads();
  const int jl = threadIdx.x >> 2, h = threadIdx.x & 3;
  const int j = jb * 64 + jl;
  if (j >= r_k) return;
  // the row segment as 8-element vectors (d_h is a multiple of 8 here)
  uint4 bseg[16];
  const uint4* src = reinterpret_cast<const uint4*>(reinterpret_cast<const TA*>(a.Bk) +
                                                    ((size_t)a.gm.k_row0[gi] + j) * a.W + (size_t)h * d_h);
#pragma unroll
  for (int v = 0; v < 16; ++v) bseg[v] = (h < gs && v * 8 < d_h) ? __ldg(src + v) : make_uint4(0, 0, 0, 0);
  constexpr float kLog2e = 1.4426950408889634f;
  const float sc = a.sm_scale * kLog2e;
  for (int bb = 0; bb < kFoldSeqs; ++bb) {
    if (!live(v0 + bb)) continue;
    float acc0 = 0.f, acc1 = 0.f;
#pragma unroll
    for (int v = 0; v < 16; ++v) {
      const TA* e = reinterpret_cast<const TA*>(&bseg[v]);
      const float4 qa = *reinterpret_cast<const float4*>(&qs[bb][h][v * 8]);
      const float4 qb = *reinterpret_cast<const float4*>(&qs[bb][h][v * 8 + 4]);
      acc0 = fmaf(Dt<ACT>::to_f(e[0]), qa.x, acc0);
      acc1 = fmaf(Dt<ACT>::to_f(e[1]), qa.y, acc1);
      acc0 = fmaf(Dt<ACT>::to_f(e[2]), qa.z, acc0);
      acc1 = fmaf(Dt<ACT>::to_f(e[3]), qa.w, acc1);
      acc0 = fmaf(Dt<ACT>::to_f(e[4]), qb.x, acc0);
      acc1 = fmaf(Dt<ACT>::to_f(e[5]), qb.y, acc1);
      acc0 = fmaf(Dt<ACT>::to_f(e[6]), qb.z, acc0);
      acc1 = fmaf(Dt<ACT>::to_f(e[7]), qb.w, acc1);
    }
    float acc = (acc0 + acc1) * sc;
    constexpr int kTerms = IMAGE ? kFoldTerms : 2;
    TA* out = reinterpret_cast<TA*>(qt) + ((size_t)(v0 + bb) * a.gm.n + gi) * kTerms * kMaxG * a.r_k;
    if constexpr (IMAGE) out += (size_t)jb * kTerms * kMaxG * 64;
#pragma unroll
    for (int i = 0; i < kTerms; ++i) {
      const TA term = Dt<ACT>::from_f(acc);
      acc -= Dt<ACT>::to_f(term);
      const int n = i * kMaxG + h;
      if constexpr (IMAGE) out[n * 64 + ((jl >> 3) ^ (n & 7)) * 8 + (jl & 7)] = term;
      else out[(size_t)n * a.r_k + j] = term;
    }
  }
}

}  // namespace
}  // namespace palu
