// Sparse decode step on CUDA cores (palu_decode_attn_pages): float32 caches and every
// shape the tensor-core kernels do not take.
//
// Method: "PALU 论文低秩投影分解" §把它放进一次真实推理流程里看, Decode 阶段.
//
// One CTA per (query, head, split of the list); a page's tokens in passes of 128 (64
// for heads wider than 64): rebuild and rotate the keys (simt_keys.cuh), score them
// (each thread its channel pair of 16 tokens, folded over the warp), online softmax,
// then the latent value sums with the tokens dealt over the threads that the rank
// leaves free.  Bound by the FMAs of the rebuild (2·r_k·d_h per token and head) for long lists and
// by latency for a page or two (one query, two float32 heads of 64, r 64, one page: 27 us
// with the combine).
#include <math.h>

#include "palu_common.cuh"
#include "palu_internal.h"
#include "simt_keys.cuh"

namespace palu {
namespace {

// Logical pages one CTA walks: entries [e0, e1) of its list.
struct ListRange {
  const int32_t* list;   // entry e0 of the list
  int n, T, npg, sb;     // entries, cached tokens, pages and index of the sequence
};

// This CTA's share (split blockIdx.x of a.S) of the list of virtual sequence vb
// and model group g.  Thread i checks every blockDim-th entry: lists ascend and
// name pages of the sequence (each page once, the partial last page last).
__device__ __forceinline__ ListRange list_range(const DecodeArgs& a, int vb, int g, DevStatus* st) {
  ListRange r;
  r.sb = vb / a.queries;
  int T = a.seq_lens[r.sb];
  const int cap = a.max_pages * a.P;
  if (T < 0 || T > cap) {
    if (threadIdx.x == 0) report(st, PALU_ERR_DEVICE_BOUNDS, 1000000 + r.sb);
    T = T < 0 ? 0 : cap;
  }
  r.T = T;
  r.npg = page_count(T, a.P);
  const size_t li = (size_t)vb * a.G + g;
  const int32_t* list = a.page_list + li * a.list_len;
  int n = a.page_counts[li];
  if (n < 0 || n > a.list_len) {
    if (threadIdx.x == 0) report(st, PALU_ERR_DEVICE_BOUNDS, 3000000 + vb);
    n = n < 0 ? 0 : a.list_len;
  }
  const int pps = (n + a.S - 1) / a.S;
  const int e0 = min(n, (int)blockIdx.x * pps), e1 = min(n, e0 + pps);
  for (int e = e0 + (int)threadIdx.x; e < e1; e += (int)blockDim.x) {
    const int lp = list[e];
    if (lp < 0 || lp >= r.npg || (e > 0 && list[e - 1] >= lp)) report(st, PALU_ERR_DEVICE_BOUNDS, 3000000 + vb);
  }
  r.list = list + e0;
  r.n = e1 - e0;
  return r;
}

// x of the lanes whose `bit` is clear and y of the others, each summed over the
// lane pair that differs in that bit.
__device__ __forceinline__ float fold(float x, float y, int bit, int lane) {
  const bool up = lane & bit;
  const float mine = up ? y : x, other = up ? x : y;
  return mine + __shfl_xor_sync(0xffffffffu, other, bit);
}

constexpr int kThreads = kKeyThreads;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxTokens = 128;
constexpr int kMaxRv = 512;

template <int ACT, int LAT>
__global__ void __launch_bounds__(kThreads) decode_pages_simt_kernel(const __grid_constant__ DecodeArgs a) {
  using TA = typename Dt<ACT>::T;
  extern __shared__ __align__(16) float zt[];        // staging; at the end the value sums of the token groups
  __shared__ float qr[2 * kMaxHalfDim];              // rotated, scaled query
  __shared__ float part_s[2][kMaxTokens], ps[kMaxTokens];
  __shared__ float wm[kWarps], wl[kWarps];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int hl = blockIdx.y, vb = blockIdx.z;
  const int gi = hl / a.gs, jh = hl % a.gs;
  const int h = a.gm.g[gi] * a.gs + jh;   // model head
  const int r_k = a.gm.rk[gi], half = a.d_h / 2;
  DevStatus* st = reinterpret_cast<DevStatus*>(a.status);
  const ListRange lr = list_range(a, vb, a.gm.g[gi], st);

  // rotated query with the softmax scale folded in
  const TA* qh = reinterpret_cast<const TA*>(a.q) + (size_t)vb * a.q_bstride + (size_t)h * a.d_h;
  const int qpos = a.q_pos[(size_t)vb * a.qpos_bstride];
  for (int i = tid; i < half; i += kThreads) {
    const float x1 = Dt<ACT>::to_f(qh[i]), x2 = Dt<ACT>::to_f(qh[i + half]);
    float c = 1.f, s = 0.f;
    if (a.rope) rope_cs_accurate(qpos, a.omega[i], c, s);
    qr[i] = (x1 * c - x2 * s) * a.sm_scale;
    qr[i + half] = (x2 * c + x1 * s) * a.sm_scale;
  }

  const int lanes = key_lanes(half), tokens = key_tokens(half);
  const int i = tid % lanes, run = tid / lanes;
  __syncthreads();
  const float q1 = i < half ? qr[i] : 0.f, q2 = i < half ? qr[i + half] : 0.f;
  // value sums: thread (latent entry rv, token group vg)
  const int rpad = a.r_v >= kThreads ? kThreads : a.r_v, vgroups = kThreads / rpad;
  const int rv = tid % rpad, vg = tid / rpad;
  const bool von = vg < vgroups;
  float acc[kMaxRv / kThreads] = {0.f, 0.f};
  float m_run = -INFINITY, l_run = 0.f;
  const TA* Bk = reinterpret_cast<const TA*>(a.Bk) + (size_t)a.gm.k_row0[gi] * a.W + jh * a.d_h;

  for (int e = 0; e < lr.n; ++e) {
    const int lp = lr.list[e];
    if (lp < 0 || lp >= lr.npg) continue;            // reported by list_range
    const int page = a.page_table[(size_t)lr.sb * a.max_pages + lp];
    if (page < 0 || page >= a.num_pages) {
      if (tid == 0) report(st, PALU_ERR_DEVICE_BOUNDS, 2000000 + lr.sb);
      continue;
    }
    const uint8_t* zk = a.gm.zk[gi] + (size_t)page * a.gm.k_page;
    const uint8_t* zv = a.gm.zv[gi] + (size_t)page * a.gm.v_page;
    const uint8_t* zks = LAT == PALU_INT4 ? a.gm.zks[gi] + (size_t)page * a.gm.ks_page : nullptr;
    const uint8_t* zvs = LAT == PALU_INT4 ? a.gm.zvs[gi] + (size_t)page * a.gm.vs_page : nullptr;
    // a query of several sees the tokens up to its own (a position may be any where they are explicit)
    const int seen = a.causal && a.pos_pool == nullptr ? min(lr.T, max(0, min(qpos, lr.T) + 1)) : lr.T;
    const int rows = min(a.P, max(0, seen - lp * a.P));
    auto position = [&](int t) {
      return a.pos_pool != nullptr ? a.pos_pool[(size_t)page * a.P + t] : lp * a.P + t;
    };
    for (int t0 = 0; t0 < rows; t0 += tokens) {
      const int nt = min(tokens, rows - t0);
      float k1[kKeyRun], k2[kKeyRun];
      rebuild_keys<ACT, LAT>(zk, zks, a.P, t0, nt, r_k, Bk, a.W, half, zt, k1, k2);
      float s[kKeyRun];
#pragma unroll
      for (int t = 0; t < kKeyRun; ++t) {
        const int tt = run * kKeyRun + t;
        float c = 1.f, sn = 0.f;
        if (a.rope && i < half && tt < nt) rope_cs_accurate(position(t0 + tt), a.omega[i], c, sn);
        s[t] = fmaf(k1[t] * c - k2[t] * sn, q1, (k2[t] * c + k1[t] * sn) * q2);
      }
      // sum over the warp's pairs: lane l (and l + 16) is left with token l of the run
#pragma unroll
      for (int n = kKeyRun / 2, bit = 1; n > 0; n >>= 1, bit <<= 1)
#pragma unroll
        for (int t = 0; t < n; ++t) s[t] = fold(s[2 * t], s[2 * t + 1], bit, lane);
      const float sum = s[0] + __shfl_xor_sync(0xffffffffu, s[0], 16);
      if (lane < kKeyRun) part_s[i >> 5][run * kKeyRun + lane] = sum;
      __syncthreads();
      float sc = -INFINITY;
      if (tid < nt && (!a.causal || position(t0 + tid) <= qpos))
        sc = lanes == 64 ? part_s[0][tid] + part_s[1][tid] : part_s[0][tid];
      float m = sc;
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
      if (lane == 0) wm[warp] = m;
      __syncthreads();
      float m_new = m_run;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) m_new = fmaxf(m_new, wm[w]);
      const float p = sc != -INFINITY ? expf(sc - m_new) : 0.f;
      if (tid < tokens) ps[tid] = p;
      float l = p;
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
      if (lane == 0) wl[warp] = l;
      __syncthreads();
      const float resc = m_run == -INFINITY ? 0.f : expf(m_run - m_new);
      l_run *= resc;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) l_run += wl[w];
      m_run = m_new;
      if (von) {
#pragma unroll
        for (int k = 0; k < kMaxRv / kThreads; ++k) {
          const int r = rv + k * kThreads;
          if (r >= a.r_v) continue;
          float v = acc[k] * resc;
#pragma unroll 8
          for (int t = vg; t < nt; t += vgroups) {
            const float z = load_latent<LAT, ACT>(
                zv, t0 + t, a.P, LAT == PALU_INT4 ? zvs + (size_t)(t0 + t) * a.vs_row : nullptr, r);
            v = ps[t] != 0.f ? fmaf(ps[t], z, v) : v;      // a masked token's latents may be anything
          }
          acc[k] = v;
        }
      }
      // (the next pass's staging waits for every thread before it touches zt, and its scores
      // for the whole block before ps and wl are written again)
    }
  }

  float* out = a.part + (((size_t)vb * a.gm.n * a.gs + hl) * a.S + blockIdx.x) * (a.r_v + 2);
  if (tid == 0) {
    out[0] = m_run;
    out[1] = l_run;
  }
  if (vgroups > 1) {
    __syncthreads();
    if (von) zt[vg * rpad + rv] = acc[0];
    __syncthreads();
    if (tid < rpad) {
      float v = 0.f;
      for (int w = 0; w < vgroups; ++w) v += zt[w * rpad + tid];
      out[2 + tid] = v;
    }
  } else {
#pragma unroll
    for (int k = 0; k < kMaxRv / kThreads; ++k)
      if (von && rv + k * kThreads < a.r_v) out[2 + rv + k * kThreads] = acc[k];
  }
}

template <int ACT, int LAT>
cudaError_t launch_t(const DecodeArgs& a, cudaStream_t st) {
  const size_t smem = sizeof(float) * key_stage_floats(a.d_h / 2);   // at least kThreads floats
  decode_pages_simt_kernel<ACT, LAT><<<dim3(a.S, a.gm.n * a.gs, a.batch), kThreads, smem, st>>>(a);
  count_launch();
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_decode_pages_simt(const DecodeArgs& a, cudaStream_t st) {
  if (a.act == PALU_F32 && a.lat == PALU_F32) return launch_t<PALU_F32, PALU_F32>(a, st);
  if (a.act == PALU_F16 && a.lat == PALU_F16) return launch_t<PALU_F16, PALU_F16>(a, st);
  if (a.act == PALU_BF16 && a.lat == PALU_BF16) return launch_t<PALU_BF16, PALU_BF16>(a, st);
  if (a.act == PALU_F16 && a.lat == PALU_INT4) return launch_t<PALU_F16, PALU_INT4>(a, st);
  if (a.act == PALU_BF16 && a.lat == PALU_INT4) return launch_t<PALU_BF16, PALU_INT4>(a, st);
  return cudaErrorInvalidValue;
}

}  // namespace palu
