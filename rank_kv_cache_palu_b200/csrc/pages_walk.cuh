// The walk of the sparse decode kernels (palu_decode_attn_pages) over page lists.
//
// A launch covers, for each block column y (a head group, or a head pair of one),
// the lists of `units` queries back to back: Σ count[u] tiles of one page.  The
// column's CTAs take equal runs of q = ceil(tiles / CTAs) consecutive tiles whatever
// lists they belong to, so every SM works to the end however the list lengths are
// spread, a CTA keeps what its lists share (B_k of the head pair) and its pipeline
// runs on across lists.  A CTA's tiles of one list are a segment; the segment that
// holds a list's first page writes the list's main partial, every other one (only the
// CTA's first can be) the CTA's own continuation partial.
#pragma once

#include "palu_common.cuh"
#include "palu_internal.h"

namespace palu {
namespace {

constexpr int kWalkTiles = 128;    // tiles of one CTA, at most
constexpr int kWalkUnits = 2048;   // queries one launch enumerates

struct Tile {
  int page;    // physical page; -1: outside the pool (reported, its data are another page's)
  int lp;      // logical page
  int unit;    // query
  int info;    // rows the query sees (0..128) and the flags below
};
constexpr int kTileRows = 255, kTileFirst = 256, kTileLast = 512, kTileCont = 1024;
__device__ __forceinline__ int tile_rows(int info) { return info & kTileRows; }

// What a partial page's unused rows are filled with in shared memory: the page's own
// bytes there may be anything (NaN included), and a weight of 0 does not silence a NaN.
// (A loop over the valid rows on CUDA cores, the alternative, took the no-RoPE step of
// 14 queries x 64 pages from 143 to 221 us.)
__device__ uint4 g_zero_rows[128 * 128 / 16];

// Fills tiles[] of this CTA (block (x, y) of gridDim.x CTAs per column) for model
// group g and returns their number.  prefix: shared memory of a.batch + 1 ints, free
// again after the call.  The whole block takes part.  `owner`: this CTA writes the
// segment records [unit][entry gi] = (first continuation CTA, how many) of the lists
// whose main segment it holds.
__device__ __forceinline__ int walk_tiles(const DecodeArgs& a, int g, int gi, bool owner, Tile* tiles, int* prefix,
                                          DevStatus* st) {
  const int tid = threadIdx.x, lane = tid & 31;
  const int units = a.batch;
  if (tid < 32) {
    int run = 0;
    if (lane == 0) prefix[0] = 0;
    for (int u0 = 0; u0 < units; u0 += 32) {
      const int u = u0 + lane;
      int n = 0;
      if (u < units) {
        n = a.page_counts[(size_t)u * a.G + g];
        if (n < 0 || n > a.list_len) {
          if (blockIdx.x == 0) report(st, PALU_ERR_DEVICE_BOUNDS, 3000000 + u);
          n = n < 0 ? 0 : a.list_len;
        }
      }
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, n, off);
        if (lane >= off) n += o;
      }
      if (u < units) prefix[u + 1] = run + n;
      run += __shfl_sync(0xffffffffu, n, 31);
    }
  }
  __syncthreads();
  const int total = prefix[units];
  const int q = (total + (int)gridDim.x - 1) / (int)gridDim.x;
  const int i0 = min(total, (int)blockIdx.x * q), n = min(total, i0 + q) - i0;
  for (int k = tid; k < n; k += (int)blockDim.x) {
    const int idx = i0 + k;
    int lo = 0, hi = units - 1;            // the last unit whose first tile is <= idx
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (prefix[mid] <= idx) lo = mid;
      else hi = mid - 1;
    }
    const int u = lo, e = idx - prefix[u], end = prefix[u + 1];
    const int32_t* list = a.page_list + ((size_t)u * a.G + g) * a.list_len;
    const int lp = list[e], before = e > 0 ? list[e - 1] : -1;
    const int sb = u / a.queries;
    const int cap = a.max_pages * a.P;
    int T = a.seq_lens[sb];
    if (T < 0 || T > cap) {
      report(st, PALU_ERR_DEVICE_BOUNDS, 1000000 + sb);
      T = T < 0 ? 0 : cap;
    }
    const int npg = page_count(T, a.P);
    Tile t;
    t.unit = u;
    t.lp = lp;
    t.page = -1;
    int rows = 0;
    if (lp <= before || lp < 0 || lp >= npg) {
      report(st, PALU_ERR_DEVICE_BOUNDS, 3000000 + u);   // not ascending, or past the sequence
      t.lp = 0;
    } else {
      // a query of several sees the tokens up to its own: where positions are the tokens' places the
      // later ones are rows past the end to it, so nothing of them reaches the value product
      const int seen = a.causal && a.pos_pool == nullptr ? min(T, max(0, min(a.q_pos[u], T) + 1)) : T;
      rows = min(a.P, max(0, seen - lp * a.P));
      t.page = a.page_table[(size_t)sb * a.max_pages + lp];
      if (t.page < 0 || t.page >= a.num_pages) {
        report(st, PALU_ERR_DEVICE_BOUNDS, 2000000 + sb);
        t.page = -1;
      }
    }
    t.info = rows | (k == 0 || e == 0 ? kTileFirst : 0) | (k == n - 1 || idx == end - 1 ? kTileLast : 0) |
             (e > k ? kTileCont : 0);      // the list's first page lies in an earlier CTA
    tiles[k] = t;
    if (owner && e == 0) {
      const int last_cta = (end - 1) / q;
      a.segments[(size_t)u * a.gm.n + gi] = make_int2((int)blockIdx.x + 1, last_cta - (int)blockIdx.x);
    }
  }
  __syncthreads();
  return n;
}

// The kernels of a step follow one another as programmatic dependents: each lets the next one start
// (start_next), which does what it can without this one's results, then waits for all of them
// (await_previous; at once where the launch before was an ordinary one).
__device__ __forceinline__ void start_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void await_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Launch attribute of a programmatic dependent of the launch before it in the stream.
inline cudaLaunchAttribute dependent_launch() {
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  return at;
}

// A softmax weight reaches the 16-bit value MMA as the sum of three numbers of its type, rows of the
// product that padding would take anyway: 24 significant bits in bf16, as in float32, 33 in f16.  F16
// weights are scaled by 2^15 (the largest, 1, still fits), or those below 2^-25 would vanish beside a
// large one, however many they are.
constexpr int kWeightTerms = 3;
template <int ACT> constexpr float kWeightScale = ACT == PALU_F16 ? 0x1p15f : 1.f;
template <int ACT>
__device__ __forceinline__ void split_weight(float p, uint16_t (&term)[kWeightTerms]) {
  float rest = p * kWeightScale<ACT>;
#pragma unroll
  for (int i = 0; i < kWeightTerms; ++i) {
    const auto v = Dt<ACT>::from_f(rest);
    term[i] = *reinterpret_cast<const uint16_t*>(&v);
    rest -= Dt<ACT>::to_f(v);       // exact
  }
}

// Partial of the segment that tile t ends, for head hl of the launch:
// m, l of the four warps, then a[r_v] (float32).
__device__ __forceinline__ float* segment_part(const DecodeArgs& a, const Tile& t, int hl) {
  const int heads = a.gm.n * a.gs;
  return (t.info & kTileCont) ? a.cont + ((size_t)blockIdx.x * heads + hl) * (a.r_v + kPartHead)
                              : a.part + ((size_t)t.unit * heads + hl) * (a.r_v + kPartHead);
}

}  // namespace
}  // namespace palu
