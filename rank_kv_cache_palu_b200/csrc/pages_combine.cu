// Log-sum-exp merge of the sparse decode step's segment partials (pages_walk.cuh),
// then the value up-projection out_h = a_h · B_v[g][:, cols_h].
//
// One CTA per (query, head): the list's main partial and its continuations (mostly one
// or none: a CTA of the walk ends inside few lists), then a GEMV over B_v's r_v rows,
// 64 output pairs × 4 interleaved row quarters, as in the dense combine.  Bound by the
// L2 reads of B_v (32 KB per CTA at r_v = 128) and by latency.
#include <math.h>

#include "palu_common.cuh"
#include "palu_internal.h"

namespace palu {
namespace {

constexpr int kThreads = 256;

template <typename T>
__device__ __forceinline__ float2 load_pair(const T* p) {
  const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(p));
  if constexpr (sizeof(T) == 2) {
    const T* e = reinterpret_cast<const T*>(&w);
    float2 r;
    if constexpr (__is_same(T, __half)) r = make_float2(__half2float(e[0]), __half2float(e[1]));
    else r = make_float2(__bfloat162float(e[0]), __bfloat162float(e[1]));
    return r;
  }
}

template <int ACT>
__global__ void __launch_bounds__(kThreads) pages_combine_kernel(const __grid_constant__ DecodeArgs a) {
  using TA = typename Dt<ACT>::T;
  extern __shared__ float smem[];
  float* av = smem;               // [r_v]
  float* red = av + a.r_v;        // [4][d_h] per-quarter outputs
  const int hl = blockIdx.x, u = blockIdx.y, tid = threadIdx.x;
  const int gi = hl / a.gs, jh = hl % a.gs;
  const int h = a.gm.g[gi] * a.gs + jh;   // model head
  const int heads = a.gm.n * a.gs, stride = a.r_v + kPartHead;
  const float* main_part = a.part + ((size_t)u * heads + hl) * stride;
  TA* out = reinterpret_cast<TA*>(a.out) + (size_t)u * a.o_bstride + (size_t)h * a.d_h;
  float* lse = a.lse != nullptr ? a.lse + (size_t)u * a.lse_bstride + h : nullptr;

  int n = 0;                              // partials of the list
  const float* cont = nullptr;
  if (a.page_counts[(size_t)u * a.G + a.gm.g[gi]] > 0) {
    const int2 seg = a.segments[(size_t)u * a.gm.n + gi];
    n = 1 + seg.y;
    cont = a.cont + ((size_t)seg.x * heads + hl) * stride;
  }
  auto partial = [&](int s) { return s == 0 ? main_part : cont + (size_t)(s - 1) * heads * stride; };
  float M = -INFINITY;
  for (int s = 0; s < n; ++s) M = fmaxf(M, partial(s)[0]);
  if (M == -INFINITY) {
    for (int d = tid; d < a.d_h; d += kThreads) out[d] = Dt<ACT>::from_f(0.f);
    if (tid == 0 && lse != nullptr) *lse = -INFINITY;
    return;
  }
  float L = 0.f;
  for (int s = 0; s < n; ++s) {
    const float* p = partial(s);
    const float w = p[0] == -INFINITY ? 0.f : expf(p[0] - M);
    L += w * ((p[1] + p[2]) + (p[3] + p[4]));
  }
  const float invL = 1.f / L;
  for (int r = tid; r < a.r_v; r += kThreads) {
    float v = 0.f;
    for (int s = 0; s < n; ++s) {
      const float* p = partial(s);
      if (p[0] != -INFINITY) v = fmaf(expf(p[0] - M), p[kPartHead + r], v);
    }
    av[r] = v * invL;
  }
  __syncthreads();
  const TA* Bv = reinterpret_cast<const TA*>(a.Bv) + (size_t)a.gm.v_row0[gi] * a.W + jh * a.d_h;
  const int d0 = 2 * (tid & 63), rq = tid >> 6;
  if (d0 < a.d_h) {
    float2 acc0 = make_float2(0.f, 0.f), acc1 = acc0;
#pragma unroll 8
    for (int r = rq; r < a.r_v; r += 8) {      // r_v is a multiple of 64
      const float2 b0 = load_pair(Bv + (size_t)r * a.W + d0);
      const float2 b1 = load_pair(Bv + (size_t)(r + 4) * a.W + d0);
      acc0.x = fmaf(av[r], b0.x, acc0.x);
      acc0.y = fmaf(av[r], b0.y, acc0.y);
      acc1.x = fmaf(av[r + 4], b1.x, acc1.x);
      acc1.y = fmaf(av[r + 4], b1.y, acc1.y);
    }
    red[rq * a.d_h + d0] = acc0.x + acc1.x;
    red[rq * a.d_h + d0 + 1] = acc0.y + acc1.y;
  }
  __syncthreads();
  for (int d = tid; d < a.d_h; d += kThreads)
    out[d] = Dt<ACT>::from_f((red[d] + red[a.d_h + d]) + (red[2 * a.d_h + d] + red[3 * a.d_h + d]));
  if (tid == 0 && lse != nullptr) *lse = M + logf(L);
}

}  // namespace

cudaError_t launch_pages_combine(const DecodeArgs& a, cudaStream_t st) {
  const size_t smem = sizeof(float) * (a.r_v + 4 * a.d_h);
  const dim3 grid(a.gm.n * a.gs, a.batch);
  if (a.act == PALU_F16) pages_combine_kernel<PALU_F16><<<grid, kThreads, smem, st>>>(a);
  else if (a.act == PALU_BF16) pages_combine_kernel<PALU_BF16><<<grid, kThreads, smem, st>>>(a);
  else return cudaErrorInvalidValue;
  count_launch();
  return cudaGetLastError();
}

}  // namespace palu
