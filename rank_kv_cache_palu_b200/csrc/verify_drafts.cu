// Verification of drafted tokens against the target's probabilities.
//
// Draft i (token x) is accepted when u_i·q_i(x) < p_i(x); after a accepted drafts
// the next token is drawn from max(p_a - q_a, 0) (p_a alone when none was refused)
// by inverting its running sum at u·total.  Accepting needs 2 numbers per draft,
// the draw one row of each array, so the kernel reads the rows of draft a only:
// 2·vocab entries per sequence, bound by memory for a batch and by the launch and
// its chain of dependent loads for one sequence.
//
// A token is a whole number that must not depend on how a sum was rounded, so the
// product, the differences and the sums are taken in float64: u·q of two 16- or
// 32-bit numbers is exact there, and two orders of summation differ by ~1e-16 of
// the total, far below one weight.
//
// A row is cut into chunks, one CTA each; each CTA leaves its chunk's sum in the
// workspace, and the sequence's last CTA (a ticket) adds the sums in order, finds
// the chunk where the running sum crosses u·total and looks through that chunk
// alone.  Every order of addition is fixed, so results do not change from call to
// call.
#include "palu_common.cuh"
#include "palu_internal.h"

namespace palu {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMinChunk = 2048;

struct VerifyArgs {
  int D, V, chunk, chunks;
  const void* target;
  const void* draft;
  long long target_ld, draft_ld;
  const int32_t* draft_tokens;
  const int32_t* draft_lens;
  const float* u_accept;
  const float* u_sample;
  int32_t* tokens;
  int32_t* num_accepted;
  int32_t* rollback;
  DevStatus* st;
  unsigned* tickets;   // [batch]
  double* sums;        // [batch][chunks]
};

// Entries per chunk: enough CTAs to fill the GPU (about 8 of 148 each) for any
// batch, but no chunk below kMinChunk entries, where the CTAs would cost more
// than the reads they spread.
int chunk_of(int batch, int vocab) {
  const long long ctas = 148 * 8;
  long long c = ((long long)vocab * (batch > 0 ? batch : 1) + ctas - 1) / ctas;
  c = (c + kThreads - 1) / kThreads * kThreads;
  return (int)(c < kMinChunk ? kMinChunk : c);
}

// Sum over the block, the same on every thread and in every run.
__device__ __forceinline__ double block_sum(double v, double* buf) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
  __syncthreads();
  double s = 0.0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) s += buf[w];
  __syncthreads();
  return s;
}

template <int DT>
struct Row {
  using T = typename Dt<DT>::T;
  const T* p;
  const T* q;     // NULL: nothing is subtracted, but for the certain draft x
  int x;          // token of a refused draft that was certain, else -1
  __device__ __forceinline__ double weight(int v) const {
    const double a = (double)Dt<DT>::to_f(p[v]);
    const double b = q != nullptr ? (double)Dt<DT>::to_f(q[v]) : v == x ? 1.0 : 0.0;
    const double w = a - b;
    return w > 0.0 && w < (double)INFINITY ? w : 0.0;
  }
  // Σ weights of [v0, v1), this thread's share: every kThreads-th entry
  __device__ __forceinline__ double share(int v0, int v1) const {
    double s = 0.0;
    int v = v0 + (int)threadIdx.x;
    if (q != nullptr) {
      for (; v + 7 * kThreads < v1; v += 8 * kThreads) {
        T a[8], b[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          a[k] = p[v + k * kThreads];
          b[k] = q[v + k * kThreads];
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const double w = (double)Dt<DT>::to_f(a[k]) - (double)Dt<DT>::to_f(b[k]);
          s += w > 0.0 && w < (double)INFINITY ? w : 0.0;
        }
      }
    }
    for (; v < v1; v += kThreads) s += weight(v);
    return s;
  }
  // The first entry of [v0, v1) where base + the running sum exceeds `at` (-1: none does), and the
  // last entry of positive weight (-1: none).  The whole block takes part and gets the answer.
  __device__ int find(int v0, int v1, double base, double at, double* buf, int* ibuf) const {
    const int per = (v1 - v0 + kThreads - 1) / kThreads;
    const int a = min(v1, v0 + (int)threadIdx.x * per), b = min(v1, a + per);
    double mine = 0.0;
    int last = -1;
    for (int v = a; v < b; ++v) {
      const double w = weight(v);
      mine += w;
      if (w > 0.0) last = v;
    }
    // exclusive prefix over the threads
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    double s = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const double o = __shfl_up_sync(0xffffffffu, s, off);
      if (lane >= off) s += o;
    }
    if (lane == 31) buf[warp] = s;
    if (threadIdx.x == 0) {
      ibuf[0] = INT32_MAX;
      ibuf[1] = -1;
    }
    __syncthreads();
    double run = base + (s - mine);
    for (int w = 0; w < warp; ++w) run += buf[w];
    for (int v = a; v < b; ++v) {
      const double w = weight(v);
      run += w;
      if (w > 0.0 && run > at) {
        atomicMin(&ibuf[0], v);
        break;
      }
    }
    if (last >= 0) atomicMax(&ibuf[1], last);
    __syncthreads();
    const int hit = ibuf[0] != INT32_MAX ? ibuf[0] : ibuf[1];
    __syncthreads();
    return hit;
  }
};

template <int DT>
__global__ void __launch_bounds__(kThreads) verify_kernel(const VerifyArgs a) {
  using T = typename Dt<DT>::T;
  __shared__ double buf[kWarps];
  __shared__ int ibuf[2];
  __shared__ int accepted, is_last;
  const int b = blockIdx.y, tid = threadIdx.x;
  int n = a.draft_lens != nullptr ? a.draft_lens[b] : a.D;
  if (n < 0 || n > a.D) {
    if (blockIdx.x == 0 && tid == 0) report(a.st, PALU_ERR_DEVICE_BOUNDS, 1000000 + b);
    n = n < 0 ? 0 : a.D;
  }
  const T* target = static_cast<const T*>(a.target) + (size_t)b * (a.D + 1) * a.target_ld;
  const T* draft = a.draft != nullptr ? static_cast<const T*>(a.draft) + (size_t)b * a.D * a.draft_ld : nullptr;
  const int32_t* xs = a.draft_tokens + (size_t)b * a.D;
  if (tid < 32) {   // one lane per draft (PALU_MAX_DRAFTS = 32)
    bool yes = false;
    if (tid < n) {
      const int x = xs[tid];
      if (x < 0 || x >= a.V) {
        if (blockIdx.x == 0) report(a.st, PALU_ERR_DEVICE_BOUNDS, 2000000 + b);
      } else {
        const double p = (double)Dt<DT>::to_f(target[(size_t)tid * a.target_ld + x]);
        const double q = draft != nullptr ? (double)Dt<DT>::to_f(draft[(size_t)tid * a.draft_ld + x]) : 1.0;
        yes = (double)a.u_accept[(size_t)b * a.D + tid] * q < p;
      }
    }
    const unsigned no = ~__ballot_sync(0xffffffffu, yes);
    if (tid == 0) accepted = no == 0 ? 32 : __ffs(no) - 1;   // n <= 32 lanes can say yes
  }
  __syncthreads();
  const int acc = accepted;
  const bool refused = acc < n;
  Row<DT> row;
  row.p = target + (size_t)acc * a.target_ld;
  row.q = refused && draft != nullptr ? draft + (size_t)acc * a.draft_ld : nullptr;
  row.x = refused && draft == nullptr ? xs[acc] : -1;
  const int v0 = blockIdx.x * a.chunk, v1 = min(a.V, v0 + a.chunk);
  const double mine = block_sum(row.share(v0, v1), buf);

  if (a.chunks > 1) {
    if (tid == 0) {
      a.sums[(size_t)b * a.chunks + blockIdx.x] = mine;
      __threadfence();
      is_last = atomicAdd(&a.tickets[b], 1u) == (unsigned)a.chunks - 1;
    }
    __syncthreads();
    if (!is_last) return;
    __threadfence();
  }
  // the sequence's last CTA draws the token
  const double* sums = a.sums + (size_t)b * a.chunks;
  double total = 0.0;
  for (int c = 0; c < a.chunks; ++c) total += a.chunks > 1 ? __ldcg(sums + c) : mine;
  int hit = -1;
  if (total > 0.0) {
    const double at = (double)a.u_sample[b] * total;
    double base = 0.0;
    int c = 0, live = 0;       // live: the last chunk of positive sum, where a running sum cut short ends
    double live_base = 0.0;
    for (; c < a.chunks; ++c) {
      const double s = a.chunks > 1 ? __ldcg(sums + c) : mine;
      if (s > 0.0) {
        live = c;
        live_base = base;
        if (base + s > at) break;
      }
      base += s;
    }
    hit = row.find(live * a.chunk, min(a.V, (live + 1) * a.chunk), live_base, at, buf, ibuf);
  } else if (refused) {
    // p <= q everywhere: the target's own row
    row.q = nullptr;
    row.x = -1;
    total = block_sum(row.share(0, a.V), buf);
    if (total > 0.0) hit = row.find(0, a.V, 0.0, (double)a.u_sample[b] * total, buf, ibuf);
  }
  for (int i = tid; i <= a.D; i += kThreads)
    a.tokens[(size_t)b * (a.D + 1) + i] = i < acc ? xs[i] : i == acc ? hit : -1;
  if (tid == 0) {
    a.num_accepted[b] = acc;
    if (a.rollback != nullptr) a.rollback[b] = acc - n;
    if (a.chunks > 1) a.tickets[b] = 0;
  }
}

size_t align256(size_t x) { return (x + 255) / 256 * 256; }

// The tickets follow the status word and have room for the largest batch, so that no call of other
// sizes leaves anything but zeros there; then the chunk sums.
struct Layout {
  int chunk, chunks;
  size_t sums, total;
};
Layout layout(int batch, int vocab) {
  Layout l;
  l.chunk = chunk_of(batch, vocab);
  l.chunks = (vocab + l.chunk - 1) / l.chunk;
  l.sums = sizeof(DevStatus) + sizeof(unsigned) * PALU_VERIFY_MAX_BATCH;
  l.total = l.sums + align256(sizeof(double) * (size_t)batch * l.chunks);
  return l;
}

palu_status check_sizes(int batch, int num_drafts, int vocab) {
  if (batch < 0 || num_drafts < 0 || vocab <= 0) return PALU_ERR_INVALID_ARG;
  if (num_drafts > PALU_MAX_DRAFTS || batch > PALU_VERIFY_MAX_BATCH || vocab > (1 << 28)) return PALU_ERR_UNSUPPORTED;
  return PALU_OK;
}

}  // namespace
}  // namespace palu

extern "C" palu_status palu_verify_workspace_size(int batch, int num_drafts, int vocab, size_t* bytes) {
  const palu_status s = palu::check_sizes(batch, num_drafts, vocab);
  if (s != PALU_OK) return s;
  if (bytes == nullptr) return PALU_ERR_INVALID_ARG;
  *bytes = palu::layout(batch, vocab).total;
  return PALU_OK;
}

extern "C" palu_status palu_verify_drafts(int dtype, int batch, int num_drafts, int vocab, const void* target_probs,
                                          long long target_ld, const void* draft_probs, long long draft_ld,
                                          const int32_t* draft_tokens, const int32_t* draft_lens,
                                          const float* u_accept, const float* u_sample, int32_t* tokens,
                                          int32_t* num_accepted, int32_t* rollback, void* workspace,
                                          size_t workspace_bytes, palu_stream_t stream) {
  const palu_status s = palu::check_sizes(batch, num_drafts, vocab);
  if (s != PALU_OK) return s;
  if (dtype != PALU_F32 && dtype != PALU_F16 && dtype != PALU_BF16)
    return dtype == PALU_INT4 ? PALU_ERR_UNSUPPORTED : PALU_ERR_INVALID_ARG;
  if (target_ld < vocab || (draft_probs != nullptr && draft_ld < vocab)) return PALU_ERR_INVALID_ARG;
  const palu::Layout l = palu::layout(batch, vocab);
  if (workspace == nullptr || workspace_bytes < l.total) return PALU_ERR_WORKSPACE;
  if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return PALU_ERR_ALIGNMENT;
  if (batch == 0) return PALU_OK;
  if (!target_probs || !u_sample || !tokens || !num_accepted) return PALU_ERR_INVALID_ARG;
  if (num_drafts > 0 && (!draft_tokens || !u_accept)) return PALU_ERR_INVALID_ARG;
  const uintptr_t elt = dtype == PALU_F32 ? 4 : 2;
  if (reinterpret_cast<uintptr_t>(target_probs) % elt || reinterpret_cast<uintptr_t>(draft_probs) % elt)
    return PALU_ERR_ALIGNMENT;
  const void* words[] = {draft_tokens, draft_lens, u_accept, u_sample, tokens, num_accepted, rollback};
  for (const void* p : words)
    if (reinterpret_cast<uintptr_t>(p) & 3u) return PALU_ERR_ALIGNMENT;
  char* ws = static_cast<char*>(workspace);
  const palu::VerifyArgs a{num_drafts, vocab, l.chunk, l.chunks, target_probs,
                           num_drafts > 0 ? draft_probs : nullptr, target_ld, draft_ld, draft_tokens, draft_lens,
                           u_accept, u_sample, tokens, num_accepted, rollback,
                           reinterpret_cast<palu::DevStatus*>(ws),
                           reinterpret_cast<unsigned*>(ws + sizeof(palu::DevStatus)),
                           reinterpret_cast<double*>(ws + l.sums)};
  const dim3 grid(l.chunks, batch);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (dtype == PALU_F32) palu::verify_kernel<PALU_F32><<<grid, palu::kThreads, 0, st>>>(a);
  else if (dtype == PALU_F16) palu::verify_kernel<PALU_F16><<<grid, palu::kThreads, 0, st>>>(a);
  else palu::verify_kernel<PALU_BF16><<<grid, palu::kThreads, 0, st>>>(a);
  palu::count_launch();
  return palu::cuda_status(cudaGetLastError());
}
