// Append plan: pages, slots and positions of the tokens a serving step appends,
// from the sequences' lengths and the stack of free pages.
//
// Two prefix sums over the sequences settle everything: Σ max(num_new, 0) gives
// every sequence its rows, and Σ (pages needed) gives every sequence its place in
// the free stack (its i-th new page is free_pages[num_free - 1 - before - i]) and,
// where it exceeds num_free, the refusals.  A row's page then comes from the page
// table or from the stack; no row depends on another CTA's result.
//
// So one launch serves any size: every CTA takes both prefix sums over all
// sequences for itself (8 bytes a sequence, from L2) and writes its own share of
// the rows, and the CTA that finishes last (a ticket in the workspace) alone
// updates what the others have read: lengths, the stack and its count.
//
// Bound by latency: the launch, the prefix sums' loads, one table lookup, and with more
// than one CTA the ticket and the pages given back behind it.  Measured: 256 rows (one
// each of 256 sequences) 5.8 us, 500,009 rows of 64 sequences with drops and refusals
// among them 12.0 us, of which 0.6 us is the 4 MB written.  A thread takes four
// consecutive rows, found by one search and stored as 16 bytes (rows 512 apart: 15.5 us),
// or one row below 75k rows (256 rows with four a thread: 7.1 us).
#include "palu_common.cuh"
#include "palu_internal.h"

namespace palu {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kStatic = 512;      // room for the kernel's static shared memory

// Quotients by the page size, which is known only at run time: n / P = (n·m) >> s for
// 0 <= n < 2^31 with s = 31 + ceil(log2 P) and m = ceil(2^s / P) (m·P exceeds 2^s by less
// than P <= 2^(s - 31), so the product is off by less than 1 / P).
struct Divisor {
  unsigned long long m;
  int s;
};
Divisor divisor_of(int P) {
  Divisor d{0, 31};
  while ((1ull << (d.s - 31)) < (unsigned long long)P) ++d.s;
  d.m = ((1ull << d.s) + P - 1) / P;
  return d;
}

struct PlanArgs {
  int batch, P, max_pages, num_pages, n_rows;
  Divisor by;
  const int32_t* num_new;
  int32_t* seq_lens;
  int32_t* page_table;
  int32_t* free_pages;
  int32_t* num_free;
  int32_t* slots;
  int32_t* positions;
  int32_t* row_starts;
  int32_t* taken;
  DevStatus* st;
  unsigned* ticket;
};

// Exclusive prefix sum of v over the block; total receives the sum.
__device__ __forceinline__ long long block_scan(long long v, long long* warp_sums, long long& total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  long long s = v;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long o = __shfl_up_sync(0xffffffffu, s, off);
    if (lane >= off) s += o;
  }
  if (lane == 31) warp_sums[warp] = s;
  __syncthreads();
  long long before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const long long x = warp_sums[w];
    if (w < warp) before += x;
    all += x;
  }
  __syncthreads();
  total = all;
  return before + s - v;
}

// tokens / P and pages that hold that many (0 <= tokens <= max_pages·P < 2^31).
__device__ __forceinline__ int page_of(const PlanArgs& a, int tokens) {
  return (int)(((unsigned long long)(unsigned)tokens * a.by.m) >> a.by.s);
}
__device__ __forceinline__ int pages_of(const PlanArgs& a, int tokens) {
  return tokens > 0 ? page_of(a, tokens - 1) + 1 : 0;
}

__device__ __forceinline__ bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// The last i < n with start[i] <= r (start[0] <= r).
__device__ __forceinline__ int last_from(const int32_t* start, int n, long long r) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (start[mid] <= r) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// ROWS: consecutive rows a thread looks up side by side.
template <int ROWS>
__global__ void __launch_bounds__(kThreads, 2) plan_kernel(const PlanArgs a) {
  extern __shared__ int32_t smem[];
  int32_t* start = smem;                  // [batch + 1] first row of each sequence
  int32_t* len = start + a.batch + 1;     // [batch] length before the call
  int32_t* take = len + a.batch;          // [batch] tokens appended (0: refused or none) or dropped
  int32_t* before = take + a.batch;       // [batch] pages taken off the stack by earlier sequences
  __shared__ long long warp_sums[kWarps];
  __shared__ int last;
  const int tid = threadIdx.x;

  const int F0 = *a.num_free;
  const bool bad_free = F0 < 0 || F0 > a.num_pages;
  const int F = bad_free ? 0 : F0;
  if (bad_free && blockIdx.x == 0 && tid == 0) report(a.st, PALU_ERR_DEVICE_BOUNDS, 4000000);
  const long long cap = (long long)a.max_pages * a.P;

  long long rows = 0, through = 0, got = 0, back = 0;   // running totals over the sequences
  for (int b0 = 0; b0 < a.batch; b0 += kThreads) {
    const int b = b0 + tid;
    const bool in = b < a.batch;
    const int L = in ? a.seq_lens[b] : 0;
    int n = in ? a.num_new[b] : 0;
    long long total;
    const long long grow = n > 0 ? n : 0;
    const long long s0 = rows + block_scan(grow, warp_sums, total);
    rows += total;
    const long long left = (long long)L + n;
    const bool bad = in && (L < 0 || L > cap || left < 0 || left > cap || s0 + grow > a.n_rows);
    if (bad) {
      if (blockIdx.x == 0) report(a.st, PALU_ERR_DEVICE_BOUNDS, 5000000 + b);
      n = 0;
    }
    // pages to get, negative: given back
    int need = bad || !in ? 0 : pages_of(a, (int)left) - pages_of(a, L);
    const long long need_up = need > 0 ? need : 0;
    const long long p0 = through + block_scan(need_up, warp_sums, total);
    through += total;
    if (p0 + need_up > F && need_up > 0) {
      n = 0;
      need = 0;
    }
    if (need > 0 && p0 + need > got) got = p0 + need;   // admitted sequences come before the first refused
    if (need < 0) back -= need;
    if (in) {
      start[b] = (int)min(s0, (long long)INT32_MAX);
      len[b] = L;
      take[b] = n;
      before[b] = (int)min(p0, (long long)INT32_MAX);
      if (blockIdx.x == 0) {
        if (a.row_starts != nullptr) a.row_starts[b] = start[b];
        if (a.taken != nullptr) a.taken[b] = n;
      }
    }
  }
  if (tid == 0) {
    start[a.batch] = (int)min(rows, (long long)INT32_MAX);
    if (blockIdx.x == 0 && a.row_starts != nullptr) a.row_starts[a.batch] = start[a.batch];
  }
  __syncthreads();

  // this CTA's rows, ROWS consecutive ones a thread: the sequence is searched for once and
  // followed, the table lookups overlap
  const int total_rows = start[a.batch];
  const bool wide = aligned16(a.slots) && aligned16(a.positions);
  for (long long r0 = ((long long)blockIdx.x * kThreads + tid) * ROWS; r0 < a.n_rows;
       r0 += (long long)gridDim.x * kThreads * ROWS) {
    int b[ROWS], pos[ROWS], fresh[ROWS], page[ROWS], slot[ROWS];
    int at = -1;                              // sequence of the last row looked at
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
      const long long r = r0 + k;
      b[k] = -1;
      pos[k] = fresh[k] = page[k] = 0;
      if (r >= total_rows) continue;
      if (at < 0) at = last_from(start, a.batch, r);
      else if (start[at + 1] <= r) at = start[at + 2] > r ? at + 1 : last_from(start, a.batch, r);
      if (take[at] <= 0) continue;
      b[k] = at;
      pos[k] = len[at] + (int)(r - start[at]);
      const int lp = page_of(a, pos[k]);
      fresh[k] = lp - pages_of(a, len[at]);   // >= 0: a page taken by this call
      page[k] = fresh[k] >= 0 ? a.free_pages[F - 1 - before[at] - fresh[k]]
                              : a.page_table[(size_t)at * a.max_pages + lp];
    }
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
      slot[k] = -1;
      if (b[k] < 0) continue;
      const int lp = page_of(a, pos[k]), off = pos[k] - lp * a.P;
      if (off == 0 && fresh[k] >= 0)          // every new page starts with a new token
        a.page_table[(size_t)b[k] * a.max_pages + lp] = page[k];
      if (page[k] < 0 || page[k] >= a.num_pages) report(a.st, PALU_ERR_DEVICE_BOUNDS, 6000000 + b[k]);
      else slot[k] = page[k] * a.P + off;
    }
    if (ROWS == 4 && wide && r0 + ROWS <= a.n_rows) {
      *reinterpret_cast<int4*>(a.slots + r0) = make_int4(slot[0], slot[1 % ROWS], slot[2 % ROWS], slot[3 % ROWS]);
      *reinterpret_cast<int4*>(a.positions + r0) = make_int4(pos[0], pos[1 % ROWS], pos[2 % ROWS], pos[3 % ROWS]);
    } else {
      for (int k = 0; k < ROWS && r0 + k < a.n_rows; ++k) {
        a.slots[r0 + k] = slot[k];
        a.positions[r0 + k] = pos[k];
      }
    }
  }

  // the last CTA to get here updates what every CTA has read
  if (gridDim.x > 1) {
    __syncthreads();
    if (tid == 0) {
      __threadfence();
      last = atomicAdd(a.ticket, 1u) == gridDim.x - 1;
    }
    __syncthreads();
    if (!last) return;
    __threadfence();
    if (tid == 0) *a.ticket = 0;
  } else {
    __syncthreads();
  }
  // pages got: the largest admitted prefix; pages given back: their sum
  long long taken_pages = got, given = back;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    taken_pages = max(taken_pages, __shfl_xor_sync(0xffffffffu, taken_pages, off));
    given += __shfl_xor_sync(0xffffffffu, given, off);
  }
  __shared__ long long wmax[kWarps];
  if ((tid & 31) == 0) {
    wmax[tid >> 5] = taken_pages;
    warp_sums[tid >> 5] = given;
  }
  __syncthreads();
  taken_pages = 0;
  given = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    taken_pages = max(taken_pages, wmax[w]);
    given += warp_sums[w];
  }
  __syncthreads();
  const long long left = F - taken_pages;     // stack height before the pages given back
  if (given > 0) {
    // page j (in (sequence, page) order) of those given back goes to left + given - 1 - j;
    // `start` now holds each sequence's first such page, so that every page has a thread
    long long done = 0;
    for (int b0 = 0; b0 < a.batch; b0 += kThreads) {
      const int b = b0 + tid;
      int pages = 0;
      if (b < a.batch && take[b] < 0)
        pages = pages_of(a, len[b]) - pages_of(a, len[b] + take[b]);
      long long total;
      const long long j0 = done + block_scan(pages, warp_sums, total);
      done += total;
      if (b < a.batch) start[b] = (int)min(j0, (long long)INT32_MAX);
    }
    __syncthreads();
    bool bad = false;
    for (long long j = tid; j < given; j += kThreads) {
      const int lo = last_from(start, a.batch, j);   // the sequence of page j
      const int lp = pages_of(a, len[lo] + take[lo]) + (int)(j - start[lo]);
      int32_t* entry = a.page_table + (size_t)lo * a.max_pages + lp;
      const int page = *entry;
      *entry = -1;
      if (page < 0 || page >= a.num_pages) {
        report(a.st, PALU_ERR_DEVICE_BOUNDS, 6000000 + lo);
        bad = true;
      }
      const long long at = left + given - 1 - j;
      if (at < a.num_pages) a.free_pages[at] = page;
      else report(a.st, PALU_ERR_DEVICE_BOUNDS, 4000001);   // more pages given back than the pool has
    }
    if (__syncthreads_or(bad)) {
      // numbers outside the pool among them: the others close up
      const long long end = min(left + given, (long long)a.num_pages);
      long long top = left;
      for (long long i0 = left; i0 < end; i0 += kThreads) {
        const int page = i0 + tid < end ? a.free_pages[i0 + tid] : -1;
        const bool good = page >= 0 && page < a.num_pages;
        long long total;
        const long long at = top + block_scan(good, warp_sums, total);   // (every thread has read by its first barrier)
        if (good) a.free_pages[at] = page;
        top += total;
      }
      given = top - left;
    }
  }
  for (int b = tid; b < a.batch; b += kThreads)
    if (take[b] != 0) a.seq_lens[b] = len[b] + take[b];
  if (tid == 0) *a.num_free = (int)min(left + given, (long long)a.num_pages);
}

// Rows up to which each has a thread of its own, as many as fit a CTA on every SM.  One a thread
// against four, 16 sequences: 20k rows 8.2 to 9.5 us, 75k 8.6 to 9.9, 90k 9.9 to 9.7, 200k 12.4 to
// 10.1, 500k 20.2 to 12.2; 256 sequences: 75k 9.5 to 10.9, 90k 10.9 both, 200k 13.2 to 10.9.
constexpr int kSmall = 148 * kThreads;

template <int ROWS>
cudaError_t launch(const PlanArgs& a, cudaStream_t st) {
  const size_t smem = sizeof(int32_t) * (4 * (size_t)a.batch + 1);
  const cudaError_t e = allow_shared(plan_kernel<ROWS>, smem, kStatic);
  if (e != cudaSuccess) return e;
  const long long per = (long long)kThreads * ROWS;
  long long grid = (a.n_rows + per - 1) / per;
  grid = grid < 1 ? 1 : grid > 8 * 148 ? 8 * 148 : grid;
  plan_kernel<ROWS><<<(int)grid, kThreads, smem, st>>>(a);
  count_launch();
  return cudaGetLastError();
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

}  // namespace
}  // namespace palu

extern "C" palu_status palu_plan_workspace_size(int batch, size_t* bytes) {
  if (bytes == nullptr || batch < 0) return PALU_ERR_INVALID_ARG;
  *bytes = 512;   // status word, ticket
  return PALU_OK;
}

extern "C" palu_status palu_plan_append(int page_size, int batch, int max_pages, int num_pages, int n_rows,
                                        const int32_t* num_new, int32_t* seq_lens, int32_t* page_table,
                                        int32_t* free_pages, int32_t* num_free, int32_t* slot_mapping,
                                        int32_t* positions, int32_t* row_starts, int32_t* taken, void* workspace,
                                        size_t workspace_bytes, palu_stream_t stream) {
  if (page_size <= 0 || batch < 0 || max_pages <= 0 || num_pages <= 0 || n_rows < 0) return PALU_ERR_INVALID_ARG;
  if (page_size % 8 != 0) return PALU_ERR_ALIGNMENT;
  if (batch > PALU_PLAN_MAX_BATCH || (long long)num_pages * page_size > INT32_MAX ||
      (long long)max_pages * page_size > INT32_MAX)
    return PALU_ERR_UNSUPPORTED;
  if (workspace == nullptr || workspace_bytes < 512) return PALU_ERR_WORKSPACE;
  if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return PALU_ERR_ALIGNMENT;
  if (batch > 0 && (!num_new || !seq_lens || !page_table)) return PALU_ERR_INVALID_ARG;
  if (!free_pages || !num_free || (n_rows > 0 && (!slot_mapping || !positions))) return PALU_ERR_INVALID_ARG;
  const void* all[] = {num_new, seq_lens, page_table, free_pages, num_free, slot_mapping, positions, row_starts, taken};
  for (const void* p : all)
    if (!palu::aligned4(p)) return PALU_ERR_ALIGNMENT;
  palu::PlanArgs a{batch, page_size, max_pages, num_pages, n_rows, palu::divisor_of(page_size), num_new, seq_lens,
                   page_table, free_pages, num_free, slot_mapping, positions, row_starts, taken,
                   static_cast<palu::DevStatus*>(workspace),
                   reinterpret_cast<unsigned*>(static_cast<char*>(workspace) + 256)};
  const cudaError_t e = n_rows <= palu::kSmall ? palu::launch<1>(a, reinterpret_cast<cudaStream_t>(stream))
                                               : palu::launch<4>(a, reinterpret_cast<cudaStream_t>(stream));
  return palu::cuda_status(e);
}
