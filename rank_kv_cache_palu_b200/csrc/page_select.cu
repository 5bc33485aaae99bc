// Page selection: for each query and head group, the pages whose bound on the
// query's scores is largest.
//
//   score(page) = max_h Σ_c max(q'_h,c lo_c, q'_h,c hi_c),   q' = R(q_pos) q,
// the larger product being q'·hi for q' >= 0 and q'·lo below.
//
// One CTA scores a run of pages of one (sequence, group): a warp per page, 16
// bytes of lo and of hi per lane and pass, coalesced over the page's 2·W entries;
// bounds are read once per query (from L1 / L2 after the first).  Which pages win
// is a whole number, so the sums are float64: the 16- or 32-bit entries are exact
// there, and at one query per pass the float64 pipes keep up with HBM (16
// conversions a clock and SM against the ~12 entries HBM delivers).
//
// The last CTA of a (sequence, group) (a ticket) then keeps the best pages of each
// query: scores become order-preserving 64-bit keys; a histogram over the 8 bits
// below the highest bit in which the keys differ finds the bin of the last kept
// page, and is repeated inside that bin until it is kept whole or holds one key.
// Pages are compacted in index order, so the list ascends and equal scores go to
// the lower page.
#include "palu_common.cuh"
#include "palu_internal.h"

namespace palu {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxChunk = 128;   // pages one CTA scores
constexpr int kVec = 8;          // channels per lane and pass
constexpr int kHeads = 2;        // passes (groups of 32 / (d_h / kVec) heads) taken per page visit
constexpr int kAhead = 2;        // pages a warp has in flight
static_assert(kHeads == 2 && kAhead == 2, "the sums of a visit are folded by two");
constexpr int kKeys = 4096;      // scores of a list kept in shared memory while it is cut

struct SelectArgs {
  int batch, Q, H, G, gs, d_h, W, P;
  int max_pages, num_pages, n_first, n_last, K, chunk, chunks;
  int rope, causal;
  int key_room;          // keys the dynamic shared memory holds
  const void* q;
  const int32_t* q_pos;
  const void* bounds;
  const int32_t* page_table;
  const int32_t* seq_lens;
  int32_t* list;
  int32_t* counts;
  float* scores_out;
  DevStatus* st;
  unsigned* tickets;     // [batch·G]
  double* scores;        // [batch][G][Q][max_pages]
  uint64_t omega[kMaxHalfDim];
};

// cos and sin of the RoPE angle in float64: the turn is the exact 64-bit
// fixed-point product of position and frequency.
__device__ __forceinline__ void rope_cs_double(int32_t pos, uint64_t omega, double& c, double& s) {
  const long long turn = (long long)((uint64_t)(long long)pos * omega);
  sincospi((double)turn * 0x1p-63, &s, &c);   // 2·(turn / 2^64)
}

// Pages the query sees.
__device__ __forceinline__ int pages_seen(const SelectArgs& a, int T, int qpos) {
  long long t = T;
  if (a.causal && (long long)qpos + 1 < t) t = max(0LL, (long long)qpos + 1);
  return (int)((t + a.P - 1) / a.P);
}

// Order-preserving key of a score (no NaN); all keys lie strictly between 0 and the maximum.
__device__ __forceinline__ unsigned long long key_of(double v) {
  const long long b = __double_as_longlong(v);
  return b < 0 ? ~(unsigned long long)b : (unsigned long long)b | 0x8000000000000000ull;
}

// The lo and hi entries of one lane's channels.  The larger of q·lo and q·hi is the
// product with hi where q >= 0, else with lo: a bit select under masks that follow
// the signs of q, so one entry per channel is unpacked and converted.
template <int DT>
struct Box {
  using T = typename Dt<DT>::T;
  static constexpr int kWords = kVec * sizeof(T) / 4;      // 32-bit words per side
  uint4 lo[kWords / 4], hi[kWords / 4];
  __device__ __forceinline__ void load(const T* p, int W) {
#pragma unroll
    for (int w = 0; w < kWords / 4; ++w) {
      lo[w] = __ldg(reinterpret_cast<const uint4*>(p) + w);
      hi[w] = __ldg(reinterpret_cast<const uint4*>(p + W) + w);
    }
  }
  __device__ __forceinline__ static void masks(const double* q, uint32_t* m) {
    T ones[kVec];
#pragma unroll
    for (int k = 0; k < kVec; ++k) {
      if constexpr (sizeof(T) == 4) ones[k] = __uint_as_float(q[k] >= 0.0 ? 0xffffffffu : 0u);
      else {
        const uint16_t b = q[k] >= 0.0 ? 0xffffu : 0u;
        ones[k] = *reinterpret_cast<const T*>(&b);
      }
    }
#pragma unroll
    for (int w = 0; w < kWords; ++w) m[w] = reinterpret_cast<const uint32_t*>(ones)[w];
  }
  __device__ __forceinline__ double dot(const double* q, const uint32_t* m) const {
    uint32_t e[kWords];
#pragma unroll
    for (int w = 0; w < kWords; ++w)
      e[w] = (reinterpret_cast<const uint32_t*>(hi)[w] & m[w]) | (reinterpret_cast<const uint32_t*>(lo)[w] & ~m[w]);
    const T* v = reinterpret_cast<const T*>(e);
    double s = 0.0;
#pragma unroll
    for (int k = 0; k < kVec; ++k) s = fma(q[k], (double)Dt<DT>::to_f(v[k]), s);
    return s;
  }
};

// x of the lanes whose `bit` is clear and y of the others, each summed over the
// lane pair that differs in that bit.
__device__ __forceinline__ double fold(double x, double y, int bit, int lane) {
  const bool up = lane & bit;
  const double mine = up ? y : x, other = up ? x : y;
  return mine + __shfl_xor_sync(0xffffffffu, other, bit);
}

template <int DT, bool VEC>
__global__ void __launch_bounds__(kThreads, 2) select_kernel(const __grid_constant__ SelectArgs a) {
  using T = typename Dt<DT>::T;
  extern __shared__ double qr[];               // [gs][d_h] rotated query, [d_h] cosines and sines; later the keys
  __shared__ double best[kMaxChunk];           // this CTA's page scores
  __shared__ int pages[kMaxChunk];             // physical pages (-1: outside the pool)
  __shared__ int is_last;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = blockIdx.y, b = blockIdx.z;
  const int cap = a.max_pages * a.P;
  int T_ = a.seq_lens[b];
  if (T_ < 0 || T_ > cap) {
    if (blockIdx.x == 0 && g == 0 && tid == 0) report(a.st, PALU_ERR_DEVICE_BOUNDS, 1000000 + b);
    T_ = T_ < 0 ? 0 : cap;
  }
  const int npg = (T_ + a.P - 1) / a.P;
  const int p0 = blockIdx.x * a.chunk, p1 = min(npg, p0 + a.chunk);
  const T* bounds = static_cast<const T*>(a.bounds);
  double* out = a.scores + ((size_t)b * a.G + g) * a.Q * a.max_pages;

  for (int i = tid; p0 + i < p1; i += kThreads) {
    int pg = a.page_table[(size_t)b * a.max_pages + p0 + i];
    if (pg < 0 || pg >= a.num_pages) {
      report(a.st, PALU_ERR_DEVICE_BOUNDS, 2000000 + b);
      pg = -1;
    }
    pages[i] = pg;
  }
  const int half = a.d_h / 2;
  for (int j = 0; j < a.Q && p0 < p1; ++j) {
    __syncthreads();   // the previous query is done with qr and best
    const int qpos = a.q_pos[(size_t)b * a.Q + j];
    const T* q = static_cast<const T*>(a.q) + (((size_t)b * a.Q + j) * a.H + (size_t)g * a.gs) * a.d_h;
    double* cs = qr + a.gs * a.d_h;
    for (int f = tid; f < half; f += kThreads) {   // one angle serves every head
      double c = 1.0, s = 0.0;
      if (a.rope) rope_cs_double(qpos, a.omega[f], c, s);
      cs[f] = c;
      cs[half + f] = s;
    }
    __syncthreads();
    for (int i = tid; i < a.gs * half; i += kThreads) {
      const int h = i / half, f = i - h * half;
      const double x1 = (double)Dt<DT>::to_f(q[h * a.d_h + f]), x2 = (double)Dt<DT>::to_f(q[h * a.d_h + half + f]);
      const double c = cs[f], s = cs[half + f];
      qr[h * a.d_h + f] = x1 * c - x2 * s;
      qr[h * a.d_h + half + f] = x2 * c + x1 * s;
    }
    __syncthreads();
    const int n = p1 - p0;
    if constexpr (VEC) {
      // lanes_h lanes per head (4, 8 or 16), heads_w heads per pass
      const int lanes_h = a.d_h / kVec, heads_w = 32 / lanes_h;
      const int hl = lane / lanes_h, c0 = (lane % lanes_h) * kVec;
      for (int h0 = 0; h0 < a.gs; h0 += kHeads * heads_w) {
        double qv[kHeads][kVec];
        uint32_t mask[kHeads][Box<DT>::kWords];
        bool on[kHeads];
#pragma unroll
        for (int u = 0; u < kHeads; ++u) {
          const int h = h0 + u * heads_w + hl;
          on[u] = h < a.gs;
#pragma unroll
          for (int k = 0; k < kVec; ++k) qv[u][k] = on[u] ? qr[h * a.d_h + c0 + k] : 0.0;
          Box<DT>::masks(qv[u], mask[u]);
        }
        const T* mine = bounds + (size_t)g * 2 * a.W + (h0 + hl) * a.d_h + c0;
        // two pages side by side: their loads are all in flight before the first sum
        for (int i0 = warp * kAhead; i0 < n; i0 += kWarps * kAhead) {
          Box<DT> box[kAhead][kHeads];
          bool live[kAhead];
#pragma unroll
          for (int y = 0; y < kAhead; ++y) {
            const int pg = i0 + y < n ? pages[i0 + y] : -1;
            live[y] = pg >= 0;
#pragma unroll
            for (int u = 0; u < kHeads; ++u)
              if (live[y] && on[u]) box[y][u].load(mine + (size_t)pg * a.G * 2 * a.W + u * heads_w * a.d_h, a.W);
          }
          // the four sums (two pages, two heads) of the lanes of a head: two folds leave the sum of
          // page (lane / 2) % 2 and head lane % 2 spread over every fourth lane
          double s[kAhead];
#pragma unroll
          for (int y = 0; y < kAhead; ++y)
            s[y] = fold(live[y] && on[0] ? box[y][0].dot(qv[0], mask[0]) : 0.0,
                        live[y] && on[1] ? box[y][1].dot(qv[1], mask[1]) : 0.0, 1, lane);
          double v = fold(s[0], s[1], 2, lane);
          for (int off = 4; off < lanes_h; off <<= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
          const bool is_on = (lane & 1) ? on[1] : on[0], is_live = (lane & 2) ? live[1] : live[0];
          if (!is_on || !is_live || v != v) v = -INFINITY;
          v = fmax(v, __shfl_xor_sync(0xffffffffu, v, 1));
          for (int off = lanes_h; off < 32; off <<= 1) v = fmax(v, __shfl_xor_sync(0xffffffffu, v, off));
          const int i = i0 + (lane >> 1);
          if ((lane == 0 || lane == 2) && i < n) best[i] = h0 == 0 ? v : fmax(best[i], v);
        }
      }
    } else {
      for (int i = warp; i < n; i += kWarps) {
        const int pg = pages[i];
        double m = -INFINITY;
        for (int h = 0; h < a.gs && pg >= 0; ++h) {
          const T* lo = bounds + ((size_t)pg * a.G + g) * 2 * a.W + h * a.d_h;
          double s = 0.0;
          for (int c = lane; c < a.d_h; c += 32) {
            const double x = qr[h * a.d_h + c];
            s = fma(x, (double)Dt<DT>::to_f(x >= 0.0 ? lo[a.W + c] : lo[c]), s);
          }
#pragma unroll
          for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
          if (s == s) m = fmax(m, s);
        }
        if (lane == 0) best[i] = m;
      }
    }
    __syncthreads();
    for (int i = tid; i < n; i += kThreads) out[(size_t)j * a.max_pages + p0 + i] = best[i];
  }

  if (gridDim.x > 1) {
    __syncthreads();
    if (tid == 0) {
      __threadfence();
      is_last = atomicAdd(&a.tickets[(size_t)b * a.G + g], 1u) == gridDim.x - 1;
    }
    __syncthreads();
    if (!is_last) return;
    __threadfence();
    if (tid == 0) a.tickets[(size_t)b * a.G + g] = 0;
  } else {
    __syncthreads();
  }

  // ---- keep the best pages of each query
  __shared__ unsigned hist[256];
  __shared__ unsigned long long wmin[kWarps], wmax[kWarps];
  __shared__ int wcount[kWarps];
  __shared__ int bin_s, above_s;
  for (int j = 0; j < a.Q; ++j) {
    const int seen = min(npg, pages_seen(a, T_, a.q_pos[(size_t)b * a.Q + j]));
    const int first = min(a.n_first, seen), tail = max(first, seen - a.n_last);   // kept: [0, first) and [tail, seen)
    const int m = min(a.K, seen);
    int need = m - (first + seen - tail);      // pages to keep among [first, tail)
    const double* sc = out + (size_t)j * a.max_pages;
    unsigned long long* keys = reinterpret_cast<unsigned long long*>(qr);
    const bool in_smem = seen <= a.key_room;
    auto key = [&](int i) { return in_smem ? keys[i] : key_of(__ldcg(sc + i)); };
    const size_t li = ((size_t)b * a.Q + j) * a.G + g;

    // threshold: pages with a key above thr are kept, and the lowest `ties` of those equal to it
    unsigned long long thr = ~0ull;
    int ties = 0;
    if (need > 0 && need == tail - first) {
      thr = 0;
    } else if (need > 0) {
      unsigned long long lo = ~0ull, hi = 0;
      for (int i = first + tid; i < tail; i += kThreads) {
        const unsigned long long k = key_of(__ldcg(sc + i));
        if (in_smem) keys[i] = k;
        lo = min(lo, k);
        hi = max(hi, k);
      }
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) {
        lo = min(lo, __shfl_xor_sync(0xffffffffu, lo, off));
        hi = max(hi, __shfl_xor_sync(0xffffffffu, hi, off));
      }
      if (lane == 0) {
        wmin[warp] = lo;
        wmax[warp] = hi;
      }
      __syncthreads();
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        lo = min(lo, wmin[w]);
        hi = max(hi, wmax[w]);
      }
      // keys in [base, base + 2^bits) still compete; `need` of them are kept
      int bits = lo == hi ? 0 : 64 - __clzll((long long)(lo ^ hi));
      unsigned long long base = bits >= 64 ? 0 : (lo >> bits) << bits;
      while (bits > 0) {
        const int shift = bits > 8 ? bits - 8 : 0;
        hist[tid] = 0;
        __syncthreads();
        for (int i = first + tid; i < tail; i += kThreads) {
          const unsigned long long d = key(i) - base;
          if (bits >= 64 || (d >> bits) == 0) atomicAdd(&hist[(d >> shift) & 255], 1u);
        }
        __syncthreads();
        // the bin where the count from the top reaches need
        {
          const int bin = 255 - tid;
          const int c = (int)hist[bin];
          int s = c;
#pragma unroll
          for (int off = 1; off < 32; off <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, s, off);
            if (lane >= off) s += o;
          }
          if (lane == 31) wcount[warp] = s;
          __syncthreads();
          for (int w = 0; w < warp; ++w) s += wcount[w];
          if (s >= need && s - c < need) {
            bin_s = bin;
            above_s = s - c;
          }
        }
        __syncthreads();
        const int bin = bin_s, above = above_s, count = (int)hist[bin];
        base += (unsigned long long)bin << shift;
        need -= above;
        bits = shift;
        __syncthreads();
        if (count == need) break;      // the whole bin is kept
      }
      // kept: keys at or above base + (0 if the bin is kept whole)
      if (bits > 0) {
        thr = base - 1;                // every key of the bin lies above (base > 0: keys are never 0)
      } else {
        thr = base;
        ties = need;
      }
    }
    // compaction in index order
    int32_t* list = a.list + li * a.K;
    float* so = a.scores_out != nullptr ? a.scores_out + li * a.K : nullptr;
    int done = 0, tied = 0;
    for (int i0 = 0; i0 < seen; i0 += kThreads) {
      const int i = i0 + tid;
      const bool in = i < seen;
      bool keep = in && (i < first || i >= tail);
      const bool mid = in && !keep;
      const unsigned long long k = mid && thr != ~0ull && thr != 0 ? key(i) : 1;
      if (mid && k > thr) keep = true;
      const bool tie = mid && ties > 0 && k == thr;
      const unsigned below = (1u << lane) - 1;
      if (ties > 0) {
        const unsigned tb = __ballot_sync(0xffffffffu, tie);
        if (lane == 0) wcount[warp] = __popc(tb);
        __syncthreads();
        int t = tied + __popc(tb & below), all = 0;
        for (int w = 0; w < kWarps; ++w) {
          if (w < warp) t += wcount[w];
          all += wcount[w];
        }
        if (tie && t < ties) keep = true;
        tied += all;
        __syncthreads();
      }
      const unsigned kb = __ballot_sync(0xffffffffu, keep);
      if (lane == 0) wcount[warp] = __popc(kb);
      __syncthreads();
      int at = done + __popc(kb & below), all = 0;
      for (int w = 0; w < kWarps; ++w) {
        if (w < warp) at += wcount[w];
        all += wcount[w];
      }
      if (keep && at < a.K) {
        list[at] = i;
        if (so != nullptr) so[at] = (float)__ldcg(sc + i);
      }
      done += all;
      __syncthreads();
    }
    for (int i = m + tid; i < a.K; i += kThreads) {
      list[i] = -1;
      if (so != nullptr) so[i] = -INFINITY;
    }
    if (tid == 0) a.counts[li] = m;
    __syncthreads();
  }
}

size_t align256(size_t x) { return (x + 255) / 256 * 256; }

// Pages per CTA: about 6 CTAs for each of the 148 SMs, from one visit of every warp up.
int chunk_of(long long lists, int max_pages) {
  const long long ctas = 6 * 148;
  long long c = ((long long)max_pages * lists + ctas - 1) / ctas;
  const int visit = kWarps * kAhead;
  c = (c + visit - 1) / visit * visit;
  return (int)(c < visit ? visit : c > kMaxChunk ? kMaxChunk : c);
}

template <int DT>
cudaError_t launch(SelectArgs a, cudaStream_t st) {
  const dim3 grid(a.chunks, a.G, a.batch);
  a.key_room = a.max_pages < kKeys ? a.max_pages : kKeys;
  const int room = a.gs * a.d_h + a.d_h > a.key_room ? a.gs * a.d_h + a.d_h : a.key_room;
  const size_t smem = sizeof(double) * room;
  const int lanes_h = a.d_h / kVec;   // lanes a head takes in the vector form
  const bool vec = a.d_h % kVec == 0 && (lanes_h == 4 || lanes_h == 8 || lanes_h == 16);
  auto kern = vec ? select_kernel<DT, true> : select_kernel<DT, false>;
  if (smem > 40 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  kern<<<grid, kThreads, smem, st>>>(a);
  count_launch();
  return cudaGetLastError();
}

}  // namespace

size_t select_workspace(const palu_config* c, int batch, int num_queries, int max_pages) {
  const size_t G = (size_t)(c->num_heads / c->group_size);
  return sizeof(DevStatus) + sizeof(unsigned) * PALU_SELECT_MAX_LISTS +
         align256(sizeof(double) * batch * G * num_queries * max_pages);
}

cudaError_t launch_select(const palu_config* c, int batch, int num_queries, const void* q, const int32_t* q_pos,
                          const void* bounds, bool explicit_pos, const int32_t* page_table, int max_pages,
                          const int32_t* seq_lens, int num_pages, int num_first, int num_last, int list_len,
                          int32_t* page_list, int32_t* page_counts, float* page_scores, const uint64_t* omega,
                          void* workspace, cudaStream_t st) {
  SelectArgs a{};
  a.batch = batch;
  a.Q = num_queries;
  a.H = c->num_heads;
  a.gs = c->group_size;
  a.G = c->num_heads / c->group_size;
  a.d_h = c->head_dim;
  a.W = c->group_size * c->head_dim;
  a.P = c->page_size;
  a.max_pages = max_pages;
  a.num_pages = num_pages;
  a.n_first = num_first;
  a.n_last = num_last;
  a.K = list_len;
  a.chunk = chunk_of((long long)batch * a.G, max_pages);
  a.chunks = (max_pages + a.chunk - 1) / a.chunk;
  a.rope = c->rope_base != 0.f;
  a.causal = num_queries > 1 && !explicit_pos;
  a.q = q;
  a.q_pos = q_pos;
  a.bounds = bounds;
  a.page_table = page_table;
  a.seq_lens = seq_lens;
  a.list = page_list;
  a.counts = page_counts;
  a.scores_out = page_scores;
  char* ws = static_cast<char*>(workspace);
  a.st = reinterpret_cast<DevStatus*>(ws);
  a.tickets = reinterpret_cast<unsigned*>(ws + sizeof(DevStatus));
  a.scores = reinterpret_cast<double*>(ws + sizeof(DevStatus) + sizeof(unsigned) * PALU_SELECT_MAX_LISTS);
  for (int i = 0; i < kMaxHalfDim; ++i) a.omega[i] = omega[i];
  if (c->act_dtype == PALU_F32) return launch<PALU_F32>(a, st);
  if (c->act_dtype == PALU_F16) return launch<PALU_F16>(a, st);
  return launch<PALU_BF16>(a, st);
}

}  // namespace palu
