// CUDA-core rebuild of a page's keys for one head, shared by the page-bounds kernel
// and the sparse decode kernel (float32 caches, and every shape the tensor-core
// kernels do not take).
//
// 256 threads; thread (pair i, token run g) owns channels i and i + d_h/2 of 16
// consecutive tokens, so a rotation stays in the thread.  Latents are staged 32
// entries at a time, transposed to [entry][token], so that a warp (32 pairs, one run)
// reads its 16 tokens' entries as four 16-byte broadcasts for 32 FMAs.
#pragma once

#include "palu_common.cuh"

namespace palu {
namespace {

constexpr int kKeyThreads = 256;
constexpr int kKeyRun = 16;      // tokens per thread
constexpr int kKeyChunk = 32;    // latent entries staged at a time (ranks are multiples of 32)

// Pairs a token run takes in threads (half the head, rounded up to whole warps), and
// tokens one pass covers.
__device__ __forceinline__ int key_lanes(int half) { return half <= 32 ? 32 : 64; }
__device__ __forceinline__ int key_tokens(int half) { return kKeyThreads / key_lanes(half) * kKeyRun; }
// Floats of the staging buffer.
__host__ __device__ inline int key_stage_floats(int half) { return kKeyChunk * ((half <= 32 ? 128 : 64) + 4); }

// Keys before rotation of tokens [t0, t0 + nt) of the block (rows past nt: zeros);
// Bk: the head's first column of the group's rows.  The whole block takes part.
template <int ACT, int LAT>
__device__ __forceinline__ void rebuild_keys(const uint8_t* blk, const uint8_t* sblk, int P, int t0, int nt, int r_k,
                                             const typename Dt<ACT>::T* Bk, int W, int half, float* zt,
                                             float (&k1)[kKeyRun], float (&k2)[kKeyRun]) {
  constexpr int kUnits = LAT == PALU_INT4 ? 1 : kKeyChunk * (LAT == PALU_F32 ? 4 : 2) / 16;   // 16-byte units
  constexpr int kPer = kKeyChunk / kUnits;                                                     // entries of a unit
  const int tokens = key_tokens(half), pitch = tokens + 4;
  const int i = threadIdx.x % key_lanes(half), g = threadIdx.x / key_lanes(half);
  const bool on = i < half;
  const long long ks_row = int4_scale_row(r_k);
#pragma unroll
  for (int t = 0; t < kKeyRun; ++t) k1[t] = k2[t] = 0.f;
  for (int r0 = 0; r0 < r_k; r0 += kKeyChunk) {
    __syncthreads();   // the previous chunk (or pass) is done with zt
    for (int e = threadIdx.x; e < tokens * kUnits; e += kKeyThreads) {
      const int tt = e % tokens, u = e / tokens;
      float v[kPer];
#pragma unroll
      for (int k = 0; k < kPer; ++k) v[k] = 0.f;
      if (tt < nt) {
        const int t = t0 + tt;
        const long long o = LAT == PALU_INT4 ? r0 / 2 : (long long)r0 * (LAT == PALU_F32 ? 4 : 2) + u * 16;
        const uint4 raw = __ldg(reinterpret_cast<const uint4*>(blk + swz_offset(t, o, P)));
        if constexpr (LAT == PALU_INT4) {
          const float s = __half2float(reinterpret_cast<const __half*>(sblk + (size_t)t * ks_row)[r0 >> 5]);
          const uint8_t* c = reinterpret_cast<const uint8_t*>(&raw);
#pragma unroll
          for (int k = 0; k < kPer; ++k) {
            const int code = (((k & 1) ? c[k >> 1] >> 4 : c[k >> 1] & 15) ^ 8) - 8;
            v[k] = Dt<ACT>::to_f(Dt<ACT>::from_f((float)code * s));
          }
        } else {
          const typename Dt<LAT>::T* x = reinterpret_cast<const typename Dt<LAT>::T*>(&raw);
#pragma unroll
          for (int k = 0; k < kPer; ++k) v[k] = Dt<LAT>::to_f(x[k]);
        }
      }
#pragma unroll
      for (int k = 0; k < kPer; ++k) zt[(u * kPer + k) * pitch + tt] = v[k];
    }
    __syncthreads();
#pragma unroll 4
    for (int r = 0; r < kKeyChunk; ++r) {
      const float b1 = on ? Dt<ACT>::to_f(Bk[(size_t)(r0 + r) * W + i]) : 0.f;
      const float b2 = on ? Dt<ACT>::to_f(Bk[(size_t)(r0 + r) * W + half + i]) : 0.f;
      const float4* z = reinterpret_cast<const float4*>(zt + r * pitch + g * kKeyRun);
#pragma unroll
      for (int q = 0; q < kKeyRun / 4; ++q) {
        const float4 x = z[q];
        k1[4 * q] = fmaf(x.x, b1, k1[4 * q]);
        k1[4 * q + 1] = fmaf(x.y, b1, k1[4 * q + 1]);
        k1[4 * q + 2] = fmaf(x.z, b1, k1[4 * q + 2]);
        k1[4 * q + 3] = fmaf(x.w, b1, k1[4 * q + 3]);
        k2[4 * q] = fmaf(x.x, b2, k2[4 * q]);
        k2[4 * q + 1] = fmaf(x.y, b2, k2[4 * q + 1]);
        k2[4 * q + 2] = fmaf(x.z, b2, k2[4 * q + 2]);
        k2[4 * q + 3] = fmaf(x.w, b2, k2[4 * q + 3]);
      }
    }
  }
}

}  // namespace
}  // namespace palu
