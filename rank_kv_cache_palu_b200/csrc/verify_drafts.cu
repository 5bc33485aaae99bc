// Verification of drafted tokens against the target's probabilities.
//
// Draft i (token x) is accepted when u_i·q_i(x) < p_i(x); after a accepted drafts
// the next token is drawn from max(p_a - q_a, 0) (p_a alone when none was refused)
// by inverting its running sum at u·total.  Accepting needs 2 numbers per draft,
// the draw one row of each array, so the kernel reads the rows of draft a only:
// 2·vocab entries per sequence.  Bound by its chain of phases: gathering the drafts'
// probabilities (1.6 us), summing the row (8.7 us at 64 x 128k bf16 for 33 MB, half
// of it waiting for loads, half conversions and sums), the ticket (2 us) and the draw
// (2.6 us).  Measured: 64 sequences x 128,003 bf16 14.8 to 15.3 us (2.2 TB/s), one sequence
// x 32,000 float32 6.3 us.
//
// A token is a whole number that must not depend on how a sum was rounded, so the
// product, the differences and the sums are taken in float64: u·q of two 16- or
// 32-bit numbers is exact there, and two orders of summation differ by ~1e-16 of
// the total, far below one weight.
//
// A row is cut into groups of 256 entries; every warp leaves the sums of its groups
// in the workspace, and the sequence's last CTA (a ticket) finds the group where the
// running sum crosses u·total and one warp looks through that group alone.  Every
// order of addition is fixed, so results do not change from call to call.
#include "palu_common.cuh"
#include "palu_internal.h"

namespace palu {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kGroup = 256;   // entries one partial sum covers: a warp's, 8 a lane
constexpr int kKept = 1024;   // group sums the drawing CTA keeps from its first pass over them

struct VerifyArgs {
  int D, V, share, groups;
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
  double* sums;        // [batch][groups]
};

// Groups per CTA: about four CTAs for each of the 148 SMs whatever the batch (64 x 128k: 48 to 64
// groups a CTA measured best), but at least one group for every warp, below
// which CTAs cost more than the reads they spread.
int share_of(int batch, int groups) {
  const long long ctas = 148 * 4;
  long long c = ((long long)groups * (batch > 0 ? batch : 1) + ctas - 1) / ctas;
  c = (c + kWarps - 1) / kWarps * kWarps;
  return (int)(c < kWarps ? kWarps : c);
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

// The row of weights a token is drawn from.  VEC: rows start on 16 bytes and are
// read 8 entries at a time; else entry by entry, coalesced across the warp.
template <int DT, bool VEC>
struct Row {
  using T = typename Dt<DT>::T;
  const T* p;
  const T* q;     // NULL: nothing is subtracted, but for the certain draft x
  int x;          // token of a refused draft that was certain, else -1

  __device__ __forceinline__ static double weight_of(float a, float b) {
    const double w = (double)a - (double)b;
    return w > 0.0 && w < (double)INFINITY ? w : 0.0;
  }
  __device__ __forceinline__ double weight(int v) const {
    return weight_of(Dt<DT>::to_f(p[v]), q != nullptr ? Dt<DT>::to_f(q[v]) : v == x ? 1.f : 0.f);
  }
  // Σ of 8 weights, exactly as in float64.  The difference of two 16-bit numbers is
  // nearly always a float32 (a - (a - b) gives b back exactly when it is): then one
  // conversion an entry does; a group with any other entry is summed anew.
  __device__ __forceinline__ static double sum_of(const float* a, const float* b) {
    double s = 0.0;
    if constexpr (DT != PALU_F32) {
      bool fine = true;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float d = a[k] - b[k];
        fine = fine && a[k] - d == b[k] && d < INFINITY;
        s += (double)fmaxf(d, 0.f);
      }
      if (fine) return s;
      s = 0.0;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) s += weight_of(a[k], b[k]);
    return s;
  }
  // This lane's 8 entries of the group of 256 that starts at v0, which lies whole in the row.
  struct Raw {
    uint4 a[8 * sizeof(T) / 16], b[8 * sizeof(T) / 16];
  };
  __device__ __forceinline__ void load(int v0, Raw& raw) const {
    const int lane = threadIdx.x & 31;
    if constexpr (VEC) {
#pragma unroll
      for (int w = 0; w < 8 * (int)sizeof(T) / 16; ++w) {
        raw.a[w] = __ldg(reinterpret_cast<const uint4*>(p + v0 + 8 * lane) + w);
        raw.b[w] = q != nullptr ? __ldg(reinterpret_cast<const uint4*>(q + v0 + 8 * lane) + w) : make_uint4(0, 0, 0, 0);
      }
    } else {
      T* a = reinterpret_cast<T*>(raw.a);
      T* b = reinterpret_cast<T*>(raw.b);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        a[k] = p[v0 + 32 * k + lane];
        b[k] = q != nullptr ? q[v0 + 32 * k + lane] : Dt<DT>::from_f(0.f);
      }
    }
  }
  __device__ __forceinline__ double lane_sum(int v0, const Raw& raw) const {
    const int lane = threadIdx.x & 31;
    float a[8], b[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      a[k] = Dt<DT>::to_f(reinterpret_cast<const T*>(raw.a)[k]);
      b[k] = Dt<DT>::to_f(reinterpret_cast<const T*>(raw.b)[k]);
    }
    if (x >= v0 && x < v0 + kGroup) {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if ((VEC ? v0 + 8 * lane + k : v0 + 32 * k + lane) == x) b[k] = 1.f;
    }
    return sum_of(a, b);
  }
  // Σ weights of the group of 256 entries that starts at v0, loaded if it is a whole one (the whole
  // warp takes part and gets it)
  __device__ __forceinline__ double group_sum(int v0, int V, const Raw& raw) const {
    double s = 0.0;
    if (v0 + kGroup <= V) {
      s = lane_sum(v0, raw);
    } else {
      const int v = v0 + 8 * ((int)threadIdx.x & 31);
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (v + k < V) s += weight(v + k);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    return s;
  }
  // The first entry of the group at v0 where base + the running sum exceeds `at`; where rounding
  // lets none do so the last entry of positive weight.  One warp; every lane gets the answer.
  __device__ __forceinline__ int find(int v0, int V, double base, double at) const {
    const int lane = threadIdx.x & 31, v = v0 + 8 * lane;
    double w[8], s = 0.0;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      w[k] = v + k < V ? weight(v + k) : 0.0;
      s += w[k];
    }
    double run = s;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const double o = __shfl_up_sync(0xffffffffu, run, off);
      if (lane >= off) run += o;
    }
    run = base + (run - s);
    int hit = INT32_MAX, last = -1;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      run += w[k];
      if (w[k] > 0.0) {
        last = v + k;
        if (run > at && hit == INT32_MAX) hit = v + k;
      }
    }
    hit = __reduce_min_sync(0xffffffffu, hit);
    last = __reduce_max_sync(0xffffffffu, last);
    return hit != INT32_MAX ? hit : last;
  }
};

// Inclusive sum of s over the warp.
__device__ __forceinline__ double warp_scan(double s) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const double o = __shfl_up_sync(0xffffffffu, s, off);
    if (lane >= off) s += o;
  }
  return s;
}

// The draw, by one CTA, from the group sums of the whole row: the first group whose running sum
// passes u·total (the last one of positive sum if rounding hides it), then the entry within it.
// -1: no positive weight.
template <class R>
__device__ int draw(const R& row, const double* sums, int groups, int V, float u, double* kept, double* buf, int* ibuf) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  double part = 0.0;
#pragma unroll 4
  for (int i = tid; i < groups; i += kThreads) {
    const double s = __ldcg(sums + i);
    if (i < kKept) kept[i] = s;          // read again by the same thread
    part += s;
  }
  const double total = block_sum(part, buf);
  if (!(total > 0.0)) return -1;
  const double at = (double)u * total;
  if (tid == 0) {
    ibuf[0] = INT32_MAX;
    ibuf[1] = -1;
  }
  double run = 0.0, base = 0.0;   // base: the running sum ahead of this thread's group
  int won = -1;
  for (int g0 = 0; g0 < groups; g0 += kThreads) {
    const int i = g0 + tid;
    const double s = i >= groups ? 0.0 : i < kKept ? kept[i] : __ldcg(sums + i);
    const double upto = warp_scan(s);
    if (lane == 31) buf[warp] = upto;
    __syncthreads();
    double ahead = run;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) ahead += buf[w];
      run += buf[w];
    }
    if (s > 0.0) {
      base = ahead + (upto - s);
      won = i;
      if (ahead + upto > at) atomicMin(&ibuf[0], i);
      atomicMax(&ibuf[1], i);
    }
    __syncthreads();
    if (ibuf[0] != INT32_MAX) break;
  }
  const int group = ibuf[0] != INT32_MAX ? ibuf[0] : ibuf[1];
  if (won == group) buf[0] = base;
  __syncthreads();
  if (warp == 0) {
    const int hit = row.find(group * kGroup, V, buf[0], at);
    if (lane == 0) ibuf[2] = hit;
  }
  __syncthreads();
  return ibuf[2];
}

template <int DT, bool VEC>
__global__ void __launch_bounds__(kThreads, 4) verify_kernel(const VerifyArgs a) {
  using T = typename Dt<DT>::T;
  __shared__ double buf[kWarps], kept[kKept];
  __shared__ int ibuf[3];
  __shared__ int accepted, is_last;
  const int b = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int n = a.draft_lens != nullptr ? a.draft_lens[b] : a.D;
  if (n < 0 || n > a.D) {
    if (blockIdx.x == 0 && tid == 0) report(a.st, PALU_ERR_DEVICE_BOUNDS, 1000000 + b);
    n = n < 0 ? 0 : a.D;
  }
  const float u = a.u_sample[b];   // wanted at the very end: its load must not wait until then
  const T* target = static_cast<const T*>(a.target) + (size_t)b * (a.D + 1) * a.target_ld;
  const T* draft = a.draft != nullptr ? static_cast<const T*>(a.draft) + (size_t)b * a.D * a.draft_ld : nullptr;
  const int32_t* xs = a.draft_tokens + (size_t)b * a.D;
  if (tid < 32) {   // one lane per draft (PALU_MAX_DRAFTS = 32)
    bool yes = false;
    if (tid < a.D) {
      const int x = xs[tid];                                    // independent of n: its load overlaps n's
      const float ua = a.u_accept[(size_t)b * a.D + tid];
      const bool in = x >= 0 && x < a.V;
      if (!in && tid < n && blockIdx.x == 0) report(a.st, PALU_ERR_DEVICE_BOUNDS, 2000000 + b);
      if (in) {
        const double p = (double)Dt<DT>::to_f(target[(size_t)tid * a.target_ld + x]);
        const double q = draft != nullptr ? (double)Dt<DT>::to_f(draft[(size_t)tid * a.draft_ld + x]) : 1.0;
        yes = tid < n && (double)ua * q < p;
      }
    }
    const unsigned no = ~__ballot_sync(0xffffffffu, yes);
    if (tid == 0) accepted = no == 0 ? 32 : __ffs(no) - 1;      // n <= 32 lanes can say yes
  }
  __syncthreads();
  const int acc = accepted;
  const bool refused = acc < n;
  Row<DT, VEC> row;
  row.p = target + (size_t)acc * a.target_ld;
  row.q = refused && draft != nullptr ? draft + (size_t)acc * a.draft_ld : nullptr;
  row.x = refused && draft == nullptr ? xs[acc] : -1;
  double* sums = a.sums + (size_t)b * a.groups;
  // each warp kAhead groups at a time, the next ones on their way meanwhile (14.8 us at 64 x 128k
  // against 15.8 without; 64 registers, so four CTAs fit an SM)
  auto sum_groups = [&](int g0, int g1) {
    constexpr int kAhead = sizeof(T) == 2 ? 2 : 1;
    using Raw = typename Row<DT, VEC>::Raw;
    Raw now[kAhead], next[kAhead];
    auto load = [&](int g, Raw* raw) {
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
        if (g + k < g1 && (g + k + 1) * kGroup <= a.V) row.load((g + k) * kGroup, raw[k]);
    };
    int g = g0 + warp * kAhead;
    load(g, now);
    for (; g < g1; g += kWarps * kAhead) {
      load(g + kWarps * kAhead, next);
      double s[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) s[k] = g + k < g1 ? row.group_sum((g + k) * kGroup, a.V, now[k]) : 0.0;
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        if (lane == 0 && g + k < g1) sums[g + k] = s[k];
        now[k] = next[k];
      }
    }
  };
  sum_groups(blockIdx.x * a.share, min(a.groups, (int)(blockIdx.x + 1) * a.share));

  if (gridDim.x > 1) {
    __threadfence();
    __syncthreads();
    if (tid == 0) is_last = atomicAdd(&a.tickets[b], 1u) == gridDim.x - 1;
    __syncthreads();
    if (!is_last) return;
    __threadfence();
  } else {
    __syncthreads();
  }
  // the sequence's last CTA draws the token
  int hit = draw(row, sums, a.groups, a.V, u, kept, buf, ibuf);
  if (hit < 0 && refused) {
    // p <= q everywhere: the target's own row
    row.q = nullptr;
    row.x = -1;
    sum_groups(0, a.groups);
    __threadfence();
    __syncthreads();
    hit = draw(row, sums, a.groups, a.V, u, kept, buf, ibuf);
  }
  for (int i = tid; i <= a.D; i += kThreads)
    a.tokens[(size_t)b * (a.D + 1) + i] = i < acc ? xs[i] : i == acc ? hit : -1;
  if (tid == 0) {
    a.num_accepted[b] = acc;
    if (a.rollback != nullptr) a.rollback[b] = acc - n;
    if (gridDim.x > 1) a.tickets[b] = 0;
  }
}

template <int DT>
void launch(const VerifyArgs& a, dim3 grid, cudaStream_t st) {
  const long long elt = Dt<DT>::bytes;
  const bool vec = (reinterpret_cast<uintptr_t>(a.target) | reinterpret_cast<uintptr_t>(a.draft)) % 16 == 0 &&
                   a.target_ld * elt % 16 == 0 && (a.draft == nullptr || a.draft_ld * elt % 16 == 0);
  if (vec) verify_kernel<DT, true><<<grid, kThreads, 0, st>>>(a);
  else verify_kernel<DT, false><<<grid, kThreads, 0, st>>>(a);
}

size_t align256(size_t x) { return (x + 255) / 256 * 256; }

// The tickets follow the status word and have room for the largest batch, so that no call of other
// sizes leaves anything but zeros there; then the group sums.
struct Layout {
  int groups;
  size_t sums, total;
};
Layout layout(int batch, int vocab) {
  Layout l;
  l.groups = (vocab + kGroup - 1) / kGroup;
  l.sums = sizeof(DevStatus) + sizeof(unsigned) * PALU_VERIFY_MAX_BATCH;
  l.total = l.sums + align256(sizeof(double) * (size_t)batch * l.groups);
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
  const int share = palu::share_of(batch, l.groups);
  const palu::VerifyArgs a{num_drafts, vocab, share, l.groups, target_probs,
                           num_drafts > 0 ? draft_probs : nullptr, target_ld, draft_ld, draft_tokens, draft_lens,
                           u_accept, u_sample, tokens, num_accepted, rollback,
                           reinterpret_cast<palu::DevStatus*>(ws),
                           reinterpret_cast<unsigned*>(ws + sizeof(palu::DevStatus)),
                           reinterpret_cast<double*>(ws + l.sums)};
  const dim3 grid((l.groups + share - 1) / share, batch);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (dtype == PALU_F32) palu::launch<PALU_F32>(a, grid, st);
  else if (dtype == PALU_F16) palu::launch<PALU_F16>(a, grid, st);
  else palu::launch<PALU_BF16>(a, grid, st);
  palu::count_launch();
  return palu::cuda_status(cudaGetLastError());
}
