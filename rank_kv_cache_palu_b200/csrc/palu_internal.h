// Internal interface between the C-ABI layer (palu_abi.cu) and the kernel
// launchers.  Host-side only; not part of the public ABI.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "palu.h"

namespace palu {

constexpr int kMaxHalfDim = 64;  // head_dim <= 128
constexpr int kMaxGroups = 64;   // head groups per layer
constexpr int kPartHead = 8;     // floats ahead of a[r_v] in a segment's partial: m, l of four warps

// Where the head groups a launch covers keep their latents.  All groups of a
// launch share one rank pair (r_k, r_v); a layer whose groups have different
// ranks runs one launch per rank pair.  With one pool for all groups (equal
// ranks), group g's block of page pg starts at pool + (pg·G + g)·P·row; with a
// pool per group, at pool_g + pg·P·row_g.  Either way: base[g] + pg·page.
struct GroupMap {
  int n;                                // groups this launch covers
  uint16_t g[kMaxGroups];               // model group of entry i (heads g·gs .. g·gs + gs − 1)
  const uint8_t* zk[kMaxGroups];        // per model group: block of page 0
  const uint8_t* zv[kMaxGroups];
  const uint8_t* zks[kMaxGroups];       // int4 scale rows (NULL otherwise)
  const uint8_t* zvs[kMaxGroups];
  long long k_page, v_page, ks_page, vs_page;   // bytes from one page's block to the next
  uint16_t k_row0[kMaxGroups];          // first row of the group in B_k (= first column in A_k)
  uint16_t v_row0[kMaxGroups];          // same for B_v / A_v
  uint16_t rk[kMaxGroups];              // key rank of the entry (decode launches may mix key ranks;
                                        // the launch's r_k is their maximum, r_v is shared)
};

// Everything a decode launch needs, already validated.
struct DecodeArgs {
  int H, d_h, gs, G, W, r_k, r_v, P;
  int batch, max_pages, num_pages, S;
  int act, lat;        // palu_dtype values
  int rope;            // 0: RoPE off
  float sm_scale;      // 1/sqrt(d_h)
  const void* q;
  const int32_t* q_pos;
  // Per-sequence strides of q / q_pos / out / lse (elements): H·d_h, 1, H·d_h,
  // H for one query per sequence; Q times that when a step holds Q queries
  // and one launch serves one of them.
  long long q_bstride, o_bstride;
  int qpos_bstride, lse_bstride;
  int causal;          // 1: a token counts only if its position <= the query's position
  int qn;              // queries of each sequence this launch serves (the fused kernel takes
                       // several per pass; their partials sit at virtual sequence b·qn + j)
  GroupMap gm;
  const int32_t* pos_pool;
  const int32_t* page_table;
  const int32_t* seq_lens;
  const void* Bk;      // [bk_rows][W]: group entry i's rows start at gm.k_row0[i]
  const void* Bv;      // [bv_rows][W]
  int bk_rows, bv_rows;
  int bk_box;          // rows per tensor-map box of B_k: the key rank when every entry has it, else 64
  void* out;
  float* lse;
  float* part;         // [batch·qn][gm.n·gs][S][r_v + 2] float32, heads in group-map order
  void* fused_q;       // fused (no-RoPE) path: folded queries [batch·qn][gm.n][8][r_k], act dtype
  void* status;        // DevStatus*
  long long k_row, v_row, ks_row, vs_row;  // bytes per latent / scale row
  uint64_t omega[kMaxHalfDim];             // RoPE frequencies as 64-bit fixed-point turns
  long long* trace;                        // phase trace (palu_debug_trace) or NULL
  int trace_tiles;
  long long wait_cycles;                   // bound of every wait in the tensor-core kernels (SM cycles)
  int stall_test;                          // timeout-path test: the MMA thread first waits on a phase
                                           // that nothing completes, so the launch times out
  // Sparse steps (palu_decode_attn_pages): every query is a sequence of its own (batch = sequences ×
  // queries, qn = 1), reading page-table row and length b / queries and only the logical pages
  // page_list[(b·G + model group)·list_len + i], i < page_counts[b·G + model group].
  const int32_t* page_list;   // NULL: every page
  const int32_t* page_counts;
  int list_len, queries;
  int walk_ctas;              // tensor-core and fused kernels: CTAs per block column (see pages_walk.cuh)
  float* cont;                // [walk_ctas][gm.n·gs][r_v + kPartHead] continuation partials (part: the main ones,
                              // [batch][gm.n·gs][r_v + kPartHead])
  int2* segments;             // [batch][gm.n]: first continuation CTA of a list and how many there are
};

// Phase-trace buffer set by palu_debug_trace (NULL: off).
struct TraceSetting {
  void* buffer;
  size_t bytes;
  int tiles;
};
TraceSetting trace_setting();

struct CompressArgs {
  int n, d_model, G, r_k, r_v, P, num_pages;
  int act, lat;
  const void* x;
  const void* Ak;
  const void* Av;
  const int32_t* slots;
  const int32_t* positions;
  GroupMap gm;         // the groups of this launch; A column offsets in k_row0 / v_row0
  long long a_kcols, a_vcols;   // columns of A_k / A_v (row strides in elements)
  // Output columns of this launch, key side: entry i owns [kcol[i], kcol[i + 1]) (its rank
  // wide; ranks may differ between entries), kcol[gm.n] = ncols_k; likewise the value side.
  int ncols_k, ncols_v;
  uint16_t kcol[kMaxGroups + 1], vcol[kMaxGroups + 1];
  int32_t* pos_pool;
  void* status;
  float* scratch;  // workspace past the status header
  size_t scratch_bytes;
  long long k_row, v_row, ks_row, vs_row;
  long long wait_cycles;   // as in DecodeArgs
  int stall_test;
};

// Wait bound and stall switch of the timeout-path test (palu_debug_timeout_test).
struct TimeoutTest {
  long long wait_cycles;   // <= 0: the default (about a second)
  int stall;
};
TimeoutTest timeout_test_setting();

// CUDA-core kernels (any supported dtype; the only path for float32).
cudaError_t launch_decode_simt(const DecodeArgs& a, cudaStream_t st);
// The CUDA-core split kernel over page lists (DecodeArgs::page_list set); launch_decode_simt calls it.
cudaError_t launch_decode_pages_simt(const DecodeArgs& a, cudaStream_t st);
cudaError_t launch_combine(const DecodeArgs& a, cudaStream_t st);
// The merge after a walk over page lists (DecodeArgs::segments set); launch_combine calls it.
cudaError_t launch_pages_combine(const DecodeArgs& a, cudaStream_t st);
cudaError_t launch_compress_simt(const CompressArgs& a, cudaStream_t st);

// Page bounds and page selection (see palu_page_bounds, palu_select_pages).
cudaError_t launch_page_bounds(const palu_config* c, const GroupMap& gm, int bk_rows, int batch, const int32_t* first,
                               const int32_t* pos_pool, const int32_t* page_table, int max_pages,
                               const int32_t* seq_lens, int num_pages, const void* B_k, void* bounds,
                               const uint64_t* omega, void* workspace, cudaStream_t st);
size_t select_workspace(const palu_config* c, int batch, int num_queries, int max_pages);
cudaError_t launch_select(const palu_config* c, int batch, int num_queries, const void* q, const int32_t* q_pos,
                          const void* bounds, bool explicit_pos, const int32_t* page_table, int max_pages,
                          const int32_t* seq_lens, int num_pages, int num_first, int num_last, int list_len,
                          int32_t* page_list, int32_t* page_counts, float* page_scores, const uint64_t* omega,
                          void* workspace, cudaStream_t st);

// PALU_OK, or PALU_ERR_CUDA with the error's text kept for palu_last_cuda_error.
palu_status cuda_status(cudaError_t e);

// Lets a launch of `kernel` take `bytes` of dynamic shared memory, beside at most `fixed` bytes of the kernel's
// own.  The limit is state of the kernel on the device, so every call sets the same one, the largest there
// is: with a limit of its own, a call could lower it between another host thread's and that one's launch.
template <class K>
cudaError_t allow_shared(K* kernel, size_t bytes, size_t fixed = 0) {
  if (bytes + fixed <= 48 * 1024) return cudaSuccess;       // what every launch may take
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)(227 * 1024 - fixed));
}

// Whether a tensor map could be encoded.  The encoder needs a context current to the calling host thread, and
// a thread whose first CUDA call is one of this library's has none yet: it gets the current device's.
template <class F>
bool encoded(F encode) {
  CUresult r = encode();
  if (r == CUDA_ERROR_INVALID_CONTEXT) {
    int device = 0;
    if (cudaGetDevice(&device) == cudaSuccess && cudaSetDevice(device) == cudaSuccess) r = encode();
  }
  return r == CUDA_SUCCESS;
}

// Counts kernel launches (palu_kernel_launches); call once per launch.
void count_launch(int n = 1);

// Row bytes of the pools for a config.
inline long long latent_row_bytes(int lat, int r) {
  switch (lat) {
    case PALU_F32: return 4LL * r;
    case PALU_F16:
    case PALU_BF16: return 2LL * r;
    case PALU_INT4: return r / 2;
  }
  return 0;
}
inline long long scale_row_bytes(int lat, int r) {
  if (lat != PALU_INT4) return 0;
  long long b = 2LL * (r / 32);
  return (b + 15) / 16 * 16;
}

}  // namespace palu
