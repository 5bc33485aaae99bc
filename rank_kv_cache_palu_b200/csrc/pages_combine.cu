// Log-sum-exp merge of the sparse decode step's segment partials (pages_walk.cuh),
// then the value up-projection out_h = a_h · B_v[g][:, cols_h].
//
// One CTA per (query, head): the list's main partial and its continuations (mostly one
// or none: a CTA of the walk ends inside few lists), then a GEMV over B_v's r_v rows,
// 16 column groups of 16 bytes × 16 row lanes.  Bound by latency and, for many queries,
// by the L2 reads of B_v (32 KB per CTA at r_v = 128).
#include <math.h>

#include "palu_common.cuh"
#include "palu_internal.h"
#include "pages_walk.cuh"

namespace palu {
namespace {

constexpr int kThreads = 256;

constexpr int kCols = 8;            // output columns of a thread: 16 bytes of a row of B_v
constexpr int kMaxRv = 256;
constexpr int kMaxHead = 128;
constexpr int kRowLanes = kThreads / (kMaxHead / kCols);   // threads that share a column group, a row each in turn

// NR: rows of B_v per thread, r_v / kRowLanes.
template <int ACT, int NR>
__global__ void __launch_bounds__(kThreads) pages_combine_kernel(const __grid_constant__ DecodeArgs a) {
  using TA = typename Dt<ACT>::T;
  constexpr int kRv = NR * kRowLanes;
  __shared__ float av[kRv];
  __shared__ float red[kThreads / 32][kMaxHead];
  const int hl = blockIdx.x, u = blockIdx.y, tid = threadIdx.x;
  const int gi = hl / a.gs, jh = hl % a.gs;
  const int g = a.gm.g[gi], h = g * a.gs + jh;   // model head
  const int heads = a.gm.n * a.gs, stride = kRv + kPartHead;
  TA* out = reinterpret_cast<TA*>(a.out) + (size_t)u * a.o_bstride + (size_t)h * a.d_h;
  float* lse = a.lse != nullptr ? a.lse + (size_t)u * a.lse_bstride + h : nullptr;

  // B_v and the list's count do not depend on the walk and are loaded while it ends; then the list's
  // segments and its main partial (whatever it holds where the list is empty) together.
  const int cg = tid % (kMaxHead / kCols), rl = tid / (kMaxHead / kCols);
  const TA* Bv = reinterpret_cast<const TA*>(a.Bv) + (size_t)a.gm.v_row0[gi] * a.W + jh * a.d_h + cg * kCols;
  uint4 b[NR];
#pragma unroll
  for (int k = 0; k < NR; ++k)
    b[k] = cg * kCols < a.d_h ? __ldg(reinterpret_cast<const uint4*>(Bv + (size_t)(k * kRowLanes + rl) * a.W))
                              : make_uint4(0, 0, 0, 0);
  const int count = a.page_counts[(size_t)u * a.G + g];
  await_previous();       // the walk: its segments and partials
  const float* main_part = a.part + ((size_t)u * heads + hl) * stride;
  const int2 seg = a.segments[(size_t)u * a.gm.n + gi];
  float m0 = main_part[0], l0 = (main_part[1] + main_part[2]) + (main_part[3] + main_part[4]);
  float v = tid < kRv ? main_part[kPartHead + tid] : 0.f;

  float M = -INFINITY, L = 0.f;
  if (count > 0) {
    M = m0;
    const float* cont = a.cont + ((size_t)seg.x * heads + hl) * stride;
    const size_t step = (size_t)heads * stride;
    for (int s = 0; s < seg.y; ++s) M = fmaxf(M, cont[s * step]);
    if (M != -INFINITY) {
      const float w0 = m0 == -INFINITY ? 0.f : expf(m0 - M);
      L = w0 * l0;
      v = m0 == -INFINITY ? 0.f : w0 * v;
      for (int s = 0; s < seg.y; ++s) {
        const float* p = cont + s * step;
        if (p[0] == -INFINITY) continue;
        const float w = expf(p[0] - M);
        L += w * ((p[1] + p[2]) + (p[3] + p[4]));
        if (tid < kRv) v = fmaf(w, p[kPartHead + tid], v);
      }
    }
  }
  if (M == -INFINITY) {
    for (int d = tid; d < a.d_h; d += kThreads) out[d] = Dt<ACT>::from_f(0.f);
    if (tid == 0 && lse != nullptr) *lse = -INFINITY;
    return;
  }
  if (tid < kRv) av[tid] = v * (1.f / L);
  __syncthreads();
  float acc[kCols];
#pragma unroll
  for (int c = 0; c < kCols; ++c) acc[c] = 0.f;
#pragma unroll
  for (int k = 0; k < NR; ++k) {
    const float x = av[k * kRowLanes + rl];
    const TA* e = reinterpret_cast<const TA*>(&b[k]);
#pragma unroll
    for (int c = 0; c < kCols; ++c) acc[c] = fmaf(x, Dt<ACT>::to_f(e[c]), acc[c]);
  }
  // a warp holds two rows' lanes of every column group, the block eight warps
#pragma unroll
  for (int c = 0; c < kCols; ++c) acc[c] += __shfl_xor_sync(0xffffffffu, acc[c], 16);
  if ((tid & 31) < 16) {
    float4* r = reinterpret_cast<float4*>(&red[tid >> 5][cg * kCols]);
    r[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
    r[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
  }
  __syncthreads();
  for (int d = tid; d < a.d_h; d += kThreads) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) s += red[w][d];
    out[d] = Dt<ACT>::from_f(s);
  }
  if (tid == 0 && lse != nullptr) *lse = M + logf(L);
}

template <int ACT>
cudaError_t launch(const DecodeArgs& a, cudaStream_t st) {
  cudaLaunchAttribute at = dependent_launch();
  cudaLaunchConfig_t c{};
  c.gridDim = dim3(a.gm.n * a.gs, a.batch);
  c.blockDim = dim3(kThreads);
  c.stream = st;
  c.attrs = &at;
  c.numAttrs = 1;
  count_launch();
  if (a.r_v == 128) return cudaLaunchKernelEx(&c, pages_combine_kernel<ACT, 128 / kRowLanes>, a);
  if (a.r_v == kMaxRv) return cudaLaunchKernelEx(&c, pages_combine_kernel<ACT, kMaxRv / kRowLanes>, a);
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_pages_combine(const DecodeArgs& a, cudaStream_t st) {
  if (a.act == PALU_F16) return launch<PALU_F16>(a, st);
  if (a.act == PALU_BF16) return launch<PALU_BF16>(a, st);
  return cudaErrorInvalidValue;
}

}  // namespace palu
