// Page lists of the sparse decode step (palu_decode_attn_pages) for the CUDA-core
// split kernel; the tensor-core kernels walk them as pages_walk.cuh lays out.
#pragma once

#include "palu_common.cuh"
#include "palu_internal.h"

namespace palu {
namespace {

// Logical pages one CTA walks: entries [e0, e1) of its list.
struct ListRange {
  const int32_t* list;   // entry e0 of the list
  int n, T, npg, sb;     // entries, cached tokens, pages and index of the sequence
  bool ragged_last;      // the last entry is the sequence's partial last page
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
  r.npg = (T + a.P - 1) / a.P;
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
  r.ragged_last = r.n > 0 && T % a.P != 0 && r.list[r.n - 1] >= r.npg - 1;
  return r;
}

}  // namespace
}  // namespace palu
