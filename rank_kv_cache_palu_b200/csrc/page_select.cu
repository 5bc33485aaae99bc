// Page selection: for each query and head group, the pages whose bound on the
// query's scores is largest.
//
//   score(page) = max_h Σ_c q'_h,c v_c,   v_c = hi_c where q'_h,c >= 0 and lo_c below,
// the larger product, q' = R(q_pos) q.
//
// One CTA scores a run of pages for one list (sequence, group, query).  A page's 2·W
// entries of a group are contiguous (2 KB in the 7B shape): every warp streams its
// pages through four slots of shared memory with bulk copies and sums two pages side
// by side.  The CTAs of a step's other queries read the same bounds from L2.
//
// Which pages win is a whole number, so the order is that of the float64 scores.
// Float64 sums for every page are bound by their conversions (16 a clock and SM) and
// long latencies; so pages are scored in float32 with a bound E on the error,
//   |ŝ - s| <= E = 2^-20 Σ_c (|q_c| + |q_pair(c)|) |v_c|  (|v_c|: the largest of the list's pages):
// 9 roundings of a sum of up to 9 steps, 9·2^-24 Σ|q'_c v_c|, and 2^-21.5 (|q_c| +
// |q_pair(c)|) for the rotated query (angle 2^-23, sine and cosine 2^-23, two products).
// Where |q'_c| is no more than that error its sign, and so the side of the box, may be
// another in float64: |v_c| is the larger of the two sides there.
// With T̂ the float32 threshold the float64 one lies within E of it, so a page more
// than 2 E above T̂ is in, one more than 2 E below it is out, and only where pages
// inside that band have to be told apart are their float64 scores taken (about one
// list in a hundred with random boxes; every page where E is not finite).
//
// Bound by the stream of bounds for many lists and by latency for few.  Measured in the 7B
// shape (8 groups, width 512, bf16, one query): 14 sequences x 410 to 512 pages 30.0 us (0.1 GB,
// 3.5 TB/s with start and cut, which take 10 us of it), one sequence x 512 pages 11.1 us.
//
// The last CTA of a list (a ticket) cuts it: scores become
// order-preserving keys; a histogram over the 8 bits below the highest bit in which
// the keys differ finds the bin of the last kept page, and is repeated inside that
// bin until at most 32 keys are left, which one warp ranks.  Pages are compacted in
// index order, so the list ascends and equal scores go to the lower page.
#include "palu_common.cuh"
#include "palu_internal.h"
#include "tc_ptx.cuh"

namespace palu {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxChunk = 256;   // pages one CTA scores: at most 32 a warp
constexpr int kVec = 8;          // channels per lane and pass
constexpr int kHeads = 2;        // passes (groups of 32 / (d_h / kVec) heads) summed side by side
constexpr int kVisit = 2;        // pages a warp sums side by side
static_assert(kHeads == 2 && kVisit == 2, "the sums of a visit are folded by two");
constexpr int kSlots = 4;        // pages a warp has in shared memory or on their way there
constexpr int kRing = 72 * 1024; // shared memory of the warps' slots, at most
constexpr int kStatic = 4 * 1024;// room for the kernel's static shared memory
constexpr float kErr = 0x1p-20f; // E over Σ (|q_c| + |q_pair(c)|) |v_c|

struct SelectArgs {
  int batch, Q, H, G, gs, d_h, W, P;
  int max_pages, num_pages, n_first, n_last, K, chunk, chunks;
  int rope, causal;
  const void* q;
  const int32_t* q_pos;
  const void* bounds;
  const int32_t* page_table;
  const int32_t* seq_lens;
  int32_t* list;
  int32_t* counts;
  float* scores_out;
  DevStatus* st;
  unsigned* tickets;     // [batch·G·Q]
  double* exact;         // [batch][G][Q][max_pages]: float64 scores where they are needed
  float* scores;         // [batch][G][Q][max_pages]
  float* errs;           // [batch][G][Q][chunks]: what E is taken from
  uint64_t omega[kMaxHalfDim];
};

// cos or sin of the RoPE angle in float64: the turn is the exact 64-bit
// fixed-point product of position and frequency.
__device__ __forceinline__ double rope_double(int32_t pos, uint64_t omega, bool sine) {
  const long long turn = (long long)((uint64_t)(long long)pos * omega);
  const double x = (double)turn * 0x1p-63;   // 2·(turn / 2^64)
  return sine ? sinpi(x) : cospi(x);
}

// Pages the query sees.
__device__ __forceinline__ int pages_seen(const SelectArgs& a, int T, int qpos) {
  long long t = T;
  if (a.causal && (long long)qpos + 1 < t) t = max(0LL, (long long)qpos + 1);
  return (int)((t + a.P - 1) / a.P);
}

// Whether a float32 rotated query entry q of |q_c| + |q_pair(c)| = n may have the other sign in float64.
__device__ __forceinline__ bool unsure(float q, float n) { return n > 0.f && !(fabsf(q) > 0x1p-21f * n); }

// Order-preserving keys of scores (no NaN), never 0, and back.
__device__ __forceinline__ unsigned long long key_of(double v) {
  const long long b = __double_as_longlong(v);
  return b < 0 ? ~(unsigned long long)b : (unsigned long long)b | 0x8000000000000000ull;
}
__device__ __forceinline__ unsigned key_of(float v) {
  const int b = __float_as_int(v);
  return b < 0 ? ~(unsigned)b : (unsigned)b | 0x80000000u;
}
__device__ __forceinline__ float score_of(unsigned k) {
  return __uint_as_float((k & 0x80000000u) ? k & 0x7fffffffu : ~k);
}

// One lane's 8 channels of a page in shared memory (p: its lo entries, the hi entries
// W further on).  The larger of q·lo and q·hi is the product with hi where q >= 0,
// else with lo: a bit select under masks that follow the signs of q.  Sums run on
// packed float32 pairs; `top` keeps the largest |entry| taken of each channel.
template <int DT>
struct Box {
  using T = typename Dt<DT>::T;
  static constexpr int kWords = kVec * sizeof(T) / 4;      // 32-bit words per side
  __device__ __forceinline__ static void masks(const float* q, uint32_t* m) {
    T ones[kVec];
#pragma unroll
    for (int k = 0; k < kVec; ++k) {
      if constexpr (sizeof(T) == 4) ones[k] = __uint_as_float(q[k] >= 0.f ? 0xffffffffu : 0u);
      else {
        const uint16_t b = q[k] >= 0.f ? 0xffffu : 0u;
        ones[k] = *reinterpret_cast<const T*>(&b);
      }
    }
#pragma unroll
    for (int w = 0; w < kWords; ++w) m[w] = reinterpret_cast<const uint32_t*>(ones)[w];
  }
  // channels 2·pair, 2·pair + 1 of the selected words as float32
  __device__ __forceinline__ static tc::f2 pair(const uint32_t* x, int i) {
    if constexpr (DT == PALU_F32) {
      return tc::f2_pack(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1]));
    } else if constexpr (DT == PALU_BF16) {
      return tc::f2_pack(__uint_as_float(x[i] << 16), __uint_as_float(x[i] & 0xffff0000u));
    } else {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&x[i]));
      return tc::f2_pack(f.x, f.y);
    }
  }
  __device__ __forceinline__ static uint32_t larger(uint32_t a, uint32_t b) {   // |entries|, NaN left out
    if constexpr (DT == PALU_F32) {
      return __float_as_uint(fmaxf(__uint_as_float(a), fabsf(__uint_as_float(b))));
    } else if constexpr (DT == PALU_BF16) {
      const __nv_bfloat162 r = __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&a),
                                       __habs2(*reinterpret_cast<const __nv_bfloat162*>(&b)));
      return *reinterpret_cast<const uint32_t*>(&r);
    } else {
      const __half2 r =
          __hmax2(*reinterpret_cast<const __half2*>(&a), __habs2(*reinterpret_cast<const __half2*>(&b)));
      return *reinterpret_cast<const uint32_t*>(&r);
    }
  }
  __device__ __forceinline__ static float dot(const T* p, int W, const tc::f2* q, const uint32_t* m, uint32_t* top) {
    uint32_t x[kWords];
#pragma unroll
    for (int w = 0; w < kWords; w += 4) {
      const uint4 l = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint32_t*>(p) + w);
      const uint4 h = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint32_t*>(p + W) + w);
      x[w] = (h.x & m[w]) | (l.x & ~m[w]);
      x[w + 1] = (h.y & m[w + 1]) | (l.y & ~m[w + 1]);
      x[w + 2] = (h.z & m[w + 2]) | (l.z & ~m[w + 2]);
      x[w + 3] = (h.w & m[w + 3]) | (l.w & ~m[w + 3]);
    }
#pragma unroll
    for (int w = 0; w < kWords; ++w) top[w] = larger(top[w], x[w]);
    tc::f2 s = tc::f2_mul(q[0], pair(x, 0));
#pragma unroll
    for (int i = 1; i < kVec / 2; ++i) s = tc::f2_fma(q[i], pair(x, i), s);
    float a, b;
    tc::f2_unpack(s, a, b);
    return a + b;
  }
};

// x of the lanes whose `bit` is clear and y of the others, each summed over the
// lane pair that differs in that bit.
__device__ __forceinline__ float fold(float x, float y, int bit, int lane) {
  const bool up = lane & bit;
  const float mine = up ? y : x, other = up ? x : y;
  return mine + __shfl_xor_sync(0xffffffffu, other, bit);
}

template <int DT, bool VEC>
__global__ void __launch_bounds__(kThreads, 3) select_kernel(const __grid_constant__ SelectArgs a) {
  using T = typename Dt<DT>::T;
  // [gs][d_h] rotated query and [gs][d_h] |q_c| + |q_pair(c)| (float32; the slow path: the rotated
  // query in float64), then the warps' slots, later the keys
  extern __shared__ __align__(16) float smem[];
  __shared__ __align__(8) uint64_t bars[kWarps][kSlots];
  __shared__ int is_last;
  __shared__ float werr[kWarps];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = blockIdx.y / a.Q, j = blockIdx.y % a.Q, b = blockIdx.z;   // one (sequence, group, query): a list
  const int cap = a.max_pages * a.P;
  const int width = a.gs * a.d_h;
  float* qr = smem;
  float* qn = smem + width;
  char* region = reinterpret_cast<char*>(smem + 2 * width);
  // the loads that do not wait for one another go out first: length, table entries, the first query
  int T_ = a.seq_lens[b];
  const int p0 = blockIdx.x * a.chunk;
  const int my_lp = p0 + lane * kWarps + warp;      // lane k: the warp's k-th page of the chunk
  int my_page = lane < a.chunk / kWarps && my_lp < a.max_pages ? a.page_table[(size_t)b * a.max_pages + my_lp] : -1;
  const int half = a.d_h / 2;
  const int qpos = a.q_pos[(size_t)b * a.Q + j];
  const T* q = static_cast<const T*>(a.q) + (((size_t)b * a.Q + j) * a.H + (size_t)g * a.gs) * a.d_h;
  const int h_first = tid / half, f_first = tid - h_first * half;
  T x1{}, x2{};
  if (h_first < a.gs) {
    x1 = q[h_first * a.d_h + f_first];
    x2 = q[h_first * a.d_h + half + f_first];
  }
  if (T_ < 0 || T_ > cap) {
    if (blockIdx.x == 0 && blockIdx.y == 0 && tid == 0) report(a.st, PALU_ERR_DEVICE_BOUNDS, 1000000 + b);
    T_ = T_ < 0 ? 0 : cap;
  }
  const int npg = page_count(T_, a.P);
  const int p1 = min(npg, p0 + a.chunk);
  const T* bounds = static_cast<const T*>(a.bounds);
  const size_t unit = ((size_t)b * a.G + g) * a.Q + j;
  float* out = a.scores + unit * a.max_pages;
  float* errs = a.errs + unit * gridDim.x;

  // this warp's pages: lane k holds the number of page p0 + k·kWarps + warp (-1: outside the pool)
  const int nk = p0 + warp < p1 ? (p1 - 1 - p0 - warp) / kWarps + 1 : 0;
  if (lane < nk && (my_page < 0 || my_page >= a.num_pages)) {
    report(a.st, PALU_ERR_DEVICE_BOUNDS, 2000000 + b);
    my_page = -1;
  }
  // VEC: a page's bounds of one group are contiguous; each warp streams its pages through kSlots
  // slots of its own with bulk copies, lane k issuing the copy of the warp's page k (of a bad page:
  // any page's, its score is dropped)
  const uint32_t slot_bytes = 2u * a.W * sizeof(T);
  const char* ring = region + (size_t)warp * kSlots * slot_bytes;
  const uint32_t ring_u = tc::smem_u32(ring), bar_u = tc::smem_u32(&bars[warp][0]);
  const T* my_src = bounds + ((size_t)max(my_page, 0) * a.G + g) * 2 * a.W;
  const unsigned valid = __ballot_sync(0xffffffffu, my_page >= 0);
  auto issue = [&](int k) {        // the warp's page k into slot k % kSlots
    if (lane == k && k < nk) {
      const uint32_t slot = (uint32_t)k % kSlots;
      tc::mbar_expect_tx(bar_u + 8 * slot, slot_bytes);
      tc::bulk_load(ring_u + slot * slot_bytes, my_src, slot_bytes, bar_u + 8 * slot);
    }
  };
  uint32_t phases = 0;             // bit s: the parity slot s is waited for next
  if constexpr (VEC) {
    if (lane == 0) {
      for (int s = 0; s < kSlots; ++s) tc::mbar_init(bar_u + 8 * s, 1);
      tc::fence_mbar_init();
      tc::fence_proxy_async();
    }
    __syncwarp();
#pragma unroll
    for (int s = 0; s < kSlots; ++s) issue(s);
  }

  if (p0 < p1) {
    bool doubt = false;
    for (int i = tid; i < a.gs * half; i += kThreads) {
      const int h = i / half, f = i - h * half;
      if (i >= kThreads) {
        x1 = q[h * a.d_h + f];
        x2 = q[h * a.d_h + half + f];
      }
      const float u = Dt<DT>::to_f(x1), w = Dt<DT>::to_f(x2);
      float c = 1.f, s = 0.f;
      if (a.rope) rope_cs_accurate(qpos, a.omega[f], c, s);
      const float x = u * c - w * s, y = w * c + u * s;
      float n = fabsf(u) + fabsf(w);
      if (n > 0.f) n = fmaxf(n, 0x1p-100f);     // roundings of anything less are not relative ones
      qr[h * a.d_h + f] = x;
      qr[h * a.d_h + half + f] = y;
      qn[h * a.d_h + f] = qn[h * a.d_h + half + f] = n;
      doubt = doubt || unsure(x, n) || unsure(y, n);
    }
    doubt = __syncthreads_or(doubt) && a.rope;
    float* mine = out + p0 + warp;
    float err = 0.f;   // what E is taken from, over this warp's pages
    if constexpr (VEC) {
      // lanes_h lanes per head (4, 8 or 16), heads_w heads per pass
      const int lanes_h = a.d_h / kVec, heads_w = 32 / lanes_h;
      const int hl = lane / lanes_h, c0 = (lane % lanes_h) * kVec;
      tc::f2 qv[kHeads][kVec / 2];
      uint32_t mask[kHeads][Box<DT>::kWords], top[kHeads][Box<DT>::kWords];
      int at[kHeads];                                // this lane's channels in a page's lo entries
      for (int h0 = 0; h0 < a.gs; h0 += kHeads * heads_w) {
        // a pass over the warp's pages per kHeads·heads_w heads (one pass in the 7B shape)
#pragma unroll
        for (int u = 0; u < kHeads; ++u) {
          const int h = h0 + u * heads_w + hl;
          at[u] = min(h, a.gs - 1) * a.d_h + c0;
          float f[kVec];
#pragma unroll
          for (int k = 0; k < kVec; ++k) f[k] = h < a.gs ? qr[at[u] + k] : 0.f;
          Box<DT>::masks(f, mask[u]);
#pragma unroll
          for (int k = 0; k < kVec / 2; ++k) qv[u][k] = tc::f2_pack(f[2 * k], f[2 * k + 1]);
#pragma unroll
          for (int w = 0; w < Box<DT>::kWords; ++w) top[u][w] = 0u;
        }
        if (h0 > 0) {
#pragma unroll
          for (int s = 0; s < kSlots; ++s) issue(s);
        }
        const bool is_on = h0 + (lane & 1) * heads_w + hl < a.gs;
        for (int k0 = 0; k0 < nk; k0 += kVisit) {
          const T* box[kVisit];
#pragma unroll
          for (int y = 0; y < kVisit; ++y) {
            const uint32_t slot = (uint32_t)(k0 + y) % kSlots;
            box[y] = reinterpret_cast<const T*>(ring + slot * slot_bytes);
            if (k0 + y < nk) {
              if (!tc::mbar_try_wait(bar_u + 8 * slot, (phases >> slot) & 1))
                tc::mbar_drain(bar_u + 8 * slot, (phases >> slot) & 1, a.st, 50);
              phases ^= 1u << slot;
            }
          }
          if (k0 + 1 >= nk) box[1] = box[0];   // an odd last page is summed twice, once for nothing
          // the four sums (two pages, two heads) of the lanes of a head: two folds leave the sum of
          // page (lane / 2) % 2 and head lane % 2 spread over every fourth lane
          const float s00 = Box<DT>::dot(box[0] + at[0], a.W, qv[0], mask[0], top[0]);
          const float s01 = Box<DT>::dot(box[0] + at[1], a.W, qv[1], mask[1], top[1]);
          const float s10 = Box<DT>::dot(box[1] + at[0], a.W, qv[0], mask[0], top[0]);
          const float s11 = Box<DT>::dot(box[1] + at[1], a.W, qv[1], mask[1], top[1]);
          float v = fold(fold(s00, s01, 1, lane), fold(s10, s11, 1, lane), 2, lane);
          for (int off = 4; off < lanes_h; off <<= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
          const int k = k0 + ((lane >> 1) & 1);
          if (!is_on || !(valid >> k & 1) || v != v) v = -INFINITY;
          v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
          for (int off = lanes_h; off < 32; off <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, off));
          if ((lane & ~2) == 0 && k < nk) mine[k * kWarps] = h0 == 0 ? v : fmaxf(mine[k * kWarps], v);
          __syncwarp();   // every lane has read the slots: refill them
          issue(k0 + kSlots);
          issue(k0 + 1 + kSlots);
        }
        // Σ (|q_c| + |q_pair(c)|) max |v_c| of this pass's heads over the warp's pages
#pragma unroll
        for (int u = 0; u < kHeads; ++u) {
          float e = 0.f;
#pragma unroll
          for (int i = 0; i < kVec / 2; ++i) {
            float x, y;
            tc::f2_unpack(Box<DT>::pair(top[u], i), x, y);
            const float* n = qn + at[u] + 2 * i;
            e = fmaf(n[0], x, fmaf(n[1], y, e));
          }
          for (int off = 1; off < lanes_h; off <<= 1) e += __shfl_xor_sync(0xffffffffu, e, off);
          err = e < INFINITY ? fmaxf(err, e) : INFINITY;     // a sum that is not finite says nothing
        }
      }
      for (int off = lanes_h; off < 32; off <<= 1) err = fmaxf(err, __shfl_xor_sync(0xffffffffu, err, off));
    } else {
      for (int k = 0; k < nk; ++k) {
        const int pg = __shfl_sync(0xffffffffu, my_page, k);
        float best = -INFINITY;
        for (int h = 0; h < a.gs && pg >= 0; ++h) {
          const T* lo = bounds + ((size_t)pg * a.G + g) * 2 * a.W + h * a.d_h;
          float s = 0.f, e = 0.f;
          for (int c = lane; c < a.d_h; c += 32) {
            const float x = qr[h * a.d_h + c], v = Dt<DT>::to_f(x >= 0.f ? lo[a.W + c] : lo[c]);
            s = fmaf(x, v, s);
            e = fmaf(qn[h * a.d_h + c], fabsf(v), e);
          }
#pragma unroll
          for (int off = 16; off > 0; off >>= 1) {
            s += __shfl_xor_sync(0xffffffffu, s, off);
            e += __shfl_xor_sync(0xffffffffu, e, off);
          }
          if (s == s) best = fmaxf(best, s);
          if (s == s || e == e) err = e < INFINITY ? fmaxf(err, e) : INFINITY;   // (both NaN: a NaN entry)
        }
        if (lane == 0) mine[k * kWarps] = best;
      }
    }
    if (doubt) {
      // channels where float64 may take the other side of the box: both sides count, over the warp's pages
      float most = 0.f;
      for (int k = 0; k < nk; ++k) {
        const int pg = __shfl_sync(0xffffffffu, my_page, k);
        const T* lo = bounds + ((size_t)max(pg, 0) * a.G + g) * 2 * a.W;
        float e = 0.f;
        for (int c = lane; c < width && pg >= 0; c += 32) {
          if (!unsure(qr[c], qn[c])) continue;
          const float x = fabsf(Dt<DT>::to_f(lo[c])), y = fabsf(Dt<DT>::to_f(lo[a.W + c]));
          e = fmaf(qn[c], x == x && y == y ? fmaxf(x, y) : INFINITY, e);
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) e += __shfl_xor_sync(0xffffffffu, e, off);
        most = e < INFINITY ? fmaxf(most, e) : INFINITY;
      }
      err += most;
    }
    if (lane == 0) werr[warp] = err;
    __syncthreads();
    if (tid == 0) {
      for (int w = 1; w < kWarps; ++w) err = fmaxf(err, werr[w]);
      errs[blockIdx.x] = err;
    }
  }

  __threadfence();   // every lane that wrote scores
  __syncthreads();
  if (gridDim.x > 1) {
    if (tid == 0) is_last = atomicAdd(&a.tickets[unit], 1u) == gridDim.x - 1;
    __syncthreads();
    if (!is_last) return;
    __threadfence();
    if (tid == 0) a.tickets[unit] = 0;
  }

  // ---- cut the list
  unsigned* keys = reinterpret_cast<unsigned*>(region);
  __shared__ unsigned hist[256];
  __shared__ unsigned wlo[kWarps], whi[kWarps], few[32];
  __shared__ double cs[2 * kMaxHalfDim], exact_few[32];
  __shared__ int wcount[kWarps], wband[kWarps];
  __shared__ int bin_s, above_s, few_n;
  __shared__ unsigned thr_s;
  const unsigned below = (1u << lane) - 1;
  // The bin (of 256, from the top) in which the running count of hist reaches need.
  auto find_bin = [&](int need) {
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
    __syncthreads();
  };
  // Sum over the block of up to two counts.
  auto count2 = [&](int x, int y, int& sx, int& sy) {
    x = __reduce_add_sync(0xffffffffu, x);
    y = __reduce_add_sync(0xffffffffu, y);
    if (lane == 0) {
      wcount[warp] = x;
      wband[warp] = y;
    }
    __syncthreads();
    sx = sy = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      sx += wcount[w];
      sy += wband[w];
    }
    __syncthreads();
  };
  const int seen = min(npg, pages_seen(a, T_, qpos));
  const int first = min(a.n_first, seen), tail = max(first, seen - a.n_last);   // kept: [0, first) and [tail, seen)
  const int m = min(a.K, seen);
  const int want = m - (first + seen - tail);      // pages to keep among [first, tail)
  const float* sc = out;
  double* exact = a.exact + unit * a.max_pages;
  const size_t li = ((size_t)b * a.Q + j) * a.G + g;

  // pages [first, tail) are in with a key of at least in_key; those with a key in [band_key,
  // in_key) where their float64 key lies above thr, or equals it and they are among the first `ties`
  unsigned in_key = ~0u, band_key = ~0u;
  unsigned long long thr = 0;
  int ties = 0;
  if (want > 0 && want == tail - first) {
    in_key = 0;
  } else if (want > 0) {
    unsigned lo = ~0u, hi = 0;
    float err = 0.f;
    for (int i = first + tid; i < tail; i += kThreads) {
      const unsigned k = key_of(__ldcg(sc + i));
      keys[i] = k;
      lo = min(lo, k);
      hi = max(hi, k);
    }
    for (int c = tid; c < a.chunks; c += kThreads)
      if (c * a.chunk < npg) err = fmaxf(err, __ldcg(errs + c));
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    err = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(err)));   // err >= 0
    if (lane == 0) {
      wlo[warp] = lo;
      whi[warp] = hi;
      werr[warp] = err;
    }
    hist[tid] = 0;
    if (tid == 0) few_n = 0;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      lo = min(lo, wlo[w]);
      hi = max(hi, whi[w]);
      err = fmaxf(err, werr[w]);
    }
    // the key of the want-th page from the top: keys in [base, base + 2^bits) still compete
    int need = want;
    int bits = lo == hi ? 0 : 32 - __clz((int)(lo ^ hi));
    unsigned base = bits >= 32 ? 0u : (lo >> bits) << bits;
    auto competes = [&](unsigned k) { return bits >= 32 || ((k - base) >> bits) == 0; };
    while (bits > 0) {
      const int shift = bits > 8 ? bits - 8 : 0;
      for (int i = first + tid; i < tail; i += kThreads)
        if (competes(keys[i])) atomicAdd(&hist[((keys[i] - base) >> shift) & 255], 1u);
      __syncthreads();
      find_bin(need);
      const int count = (int)hist[bin_s];
      base += (unsigned)bin_s << shift;
      need -= above_s;
      bits = shift;
      __syncthreads();
      if (bits > 0 && count <= 32) {
        // few enough for one warp: the key with fewer than need above it and at least need from it up
        for (int i = first + tid; i < tail; i += kThreads)
          if (competes(keys[i])) few[atomicAdd(&few_n, 1)] = keys[i];
        __syncthreads();
        if (warp == 0) {
          const unsigned k = lane < count ? few[lane] : 0u;
          int over = 0, from = 0;
          for (int x = 0; x < count; ++x) {
            const unsigned o = __shfl_sync(0xffffffffu, k, x);
            over += o > k;
            from += o >= k;
          }
          if (lane < count && over < need && from >= need) thr_s = k;
        }
        __syncthreads();
        base = thr_s;
        bits = 0;
      } else if (bits > 0) {
        hist[tid] = 0;
        __syncthreads();
      }
    }
    // the band of 2 E around the threshold (and the rounding of its ends, and underflow)
    const float t = score_of(base);
    const float wide = 2.f * kErr * err + 0x1p-22f * fabsf(t) + 0x1p-100f;
    if (wide < INFINITY) {
      band_key = key_of(t - wide);
      in_key = key_of(t + wide) + 1;
    } else if (t == -INFINITY && err < INFINITY) {
      band_key = key_of(t);           // pages without a score: they are equal
      in_key = band_key + 1;
    } else {
      band_key = 0;                   // E is not finite: every page's float64 score is taken
      in_key = ~0u;
    }
    int sure = 0, band = 0, n_sure, n_band;
    for (int i = first + tid; i < tail; i += kThreads) {
      sure += keys[i] >= in_key;
      band += keys[i] >= band_key && keys[i] < in_key;
    }
    count2(sure, band, n_sure, n_band);
    need = want - n_sure;
    if (n_band == need) {
      in_key = band_key;
    } else {
      // float64 scores of the band: the rotated query (its angles first: qr and qn give their place
      // to it), then a warp per page
      double* qd = reinterpret_cast<double*>(smem);
      for (int f = tid; f < a.d_h; f += kThreads)
        cs[f] = a.rope ? rope_double(qpos, a.omega[f < half ? f : f - half], f >= half) : f < half ? 1.0 : 0.0;
      if (tid == 0) few_n = 0;
      __syncthreads();
      for (int i = tid; i < a.gs * half; i += kThreads) {
        const int h = i / half, f = i - h * half;
        const double u = (double)Dt<DT>::to_f(q[h * a.d_h + f]), w = (double)Dt<DT>::to_f(q[h * a.d_h + half + f]);
        qd[h * a.d_h + f] = u * cs[f] - w * cs[half + f];
        qd[h * a.d_h + half + f] = w * cs[f] + u * cs[half + f];
      }
      if (n_band <= 32)
        for (int i = first + tid; i < tail; i += kThreads)
          if (keys[i] >= band_key && keys[i] < in_key) few[atomicAdd(&few_n, 1)] = (unsigned)i;
      __syncthreads();
      auto page_score = [&](int i) {     // float64 score of page i (the whole warp)
        const int pg = a.page_table[(size_t)b * a.max_pages + i];
        double best = -INFINITY;
        for (int h = 0; h < a.gs && pg >= 0 && pg < a.num_pages; ++h) {
          const T* box = bounds + ((size_t)pg * a.G + g) * 2 * a.W + h * a.d_h;
          double s = 0.0;
#pragma unroll 4
          for (int c = lane; c < a.d_h; c += 32) {
            const double x = qd[h * a.d_h + c];
            s = fma(x, (double)Dt<DT>::to_f(x >= 0.0 ? box[a.W + c] : box[c]), s);
          }
#pragma unroll
          for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
          if (s == s) best = fmax(best, s);
        }
        return best;
      };
      if (n_band <= 32) {
        // few pages: one warp ranks them and settles their keys, kept or not
        for (int x = warp; x < n_band; x += kWarps) {
          const double s = page_score((int)few[x]);
          if (lane == 0) exact_few[x] = s;
        }
        __syncthreads();
        if (warp == 0) {
          const int i = lane < n_band ? (int)few[lane] : INT32_MAX;
          const double s = lane < n_band ? exact_few[lane] : -INFINITY;
          int ahead = 0;
          for (int x = 0; x < n_band; ++x) {
            const double o = __shfl_sync(0xffffffffu, s, x);
            const int oi = __shfl_sync(0xffffffffu, i, x);
            ahead += o > s || (o == s && oi < i);
          }
          if (lane < n_band) keys[i] = ahead < need ? ~0u : 0u;
        }
        if (in_key == ~0u) in_key = ~0u - 1;
        band_key = in_key;
        __syncthreads();
      } else {
        for (int i = first + warp; i < tail; i += kWarps) {
          if (!(keys[i] >= band_key && keys[i] < in_key)) continue;
          const double s = page_score(i);
          if (lane == 0) exact[i] = s;
        }
        __threadfence();
        __syncthreads();
        int left = 64;                                 // bits not settled yet
        while (left > 0) {
          const int shift = left - 8;
          hist[tid] = 0;
          __syncthreads();
          for (int i = first + tid; i < tail; i += kThreads)
            if (keys[i] >= band_key && keys[i] < in_key) {
              const unsigned long long k = key_of(__ldcg(exact + i));
              if (left == 64 || (k >> left) == (thr >> left)) atomicAdd(&hist[(k >> shift) & 255], 1u);
            }
          __syncthreads();
          find_bin(need);
          thr |= (unsigned long long)bin_s << shift;
          need -= above_s;
          left = shift;
          __syncthreads();
        }
        ties = need;
      }
    }
  }
  // compaction in index order
  const bool exact_band = ties > 0;
  int32_t* list = a.list + li * a.K;
  float* so = a.scores_out != nullptr ? a.scores_out + li * a.K : nullptr;
  int done = 0, tied = 0;
  for (int i0 = 0; i0 < seen; i0 += kThreads) {
    const int i = i0 + tid;
    const bool mid = i >= first && i < tail;
    bool keep = i < seen && !mid, in_band = false, tie = false;
    if (mid && in_key != ~0u) {
      const unsigned k = in_key != 0 ? keys[i] : ~0u;
      keep = k >= in_key;
      in_band = exact_band && !keep && k >= band_key;
    } else if (mid && exact_band) {
      in_band = keys[i] >= band_key;
    }
    if (in_band) {
      const unsigned long long k = key_of(__ldcg(exact + i));
      keep = k > thr;
      tie = k == thr;
    }
    if (exact_band) {
      const unsigned tb = __ballot_sync(0xffffffffu, tie);
      if (lane == 0) wband[warp] = __popc(tb);
      __syncthreads();
      int t = tied + __popc(tb & below);
      for (int w = 0; w < kWarps; ++w) {
        if (w < warp) t += wband[w];
        tied += wband[w];
      }
      if (tie && t < ties) keep = true;
      __syncthreads();
    }
    const unsigned kb = __ballot_sync(0xffffffffu, keep);
    if (lane == 0) wcount[warp] = __popc(kb);
    __syncthreads();
    int at = done + __popc(kb & below);
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) at += wcount[w];
      done += wcount[w];
    }
    if (keep && at < a.K) {
      list[at] = i;
      if (so != nullptr)
        so[at] = in_band ? (float)__ldcg(exact + i) : __ldcg(sc + i);
    }
    __syncthreads();
  }
  for (int i = m + tid; i < a.K; i += kThreads) {
    list[i] = -1;
    if (so != nullptr) so[i] = -INFINITY;
  }
  if (tid == 0) a.counts[li] = m;
}

size_t align256(size_t x) { return (x + 255) / 256 * 256; }

// Pages per CTA: as many CTAs as fit the GPU at once (three on each of the 148 SMs), so
// that each pays for its start and its query once; at least two visits of every warp
// (8 lists of 512 pages: 11.3 us against 12.3 at one and 12.9 at four), at most 32 pages
// a warp (128 lists: 31 us at 144 to 192 pages a CTA, 35 at 64, 33 at 256).
int chunk_of(long long lists, int max_pages) {
  const long long per_list = 3 * 148 / lists > 0 ? 3 * 148 / lists : 1;
  long long c = (max_pages + per_list - 1) / per_list;
  const int visit = kWarps * kVisit;
  c = (c + visit - 1) / visit * visit;
  return (int)(c < 2 * visit ? 2 * visit : c > kMaxChunk ? kMaxChunk : c);
}

template <int DT>
cudaError_t launch(SelectArgs a, cudaStream_t st) {
  const dim3 grid(a.chunks, a.G * a.Q, a.batch);
  const int lanes_h = a.d_h / kVec;   // lanes a head takes in the vector form
  const size_t slots = (size_t)2 * a.W * Dt<DT>::bytes * kWarps * kSlots;
  const bool vec =
      a.d_h % kVec == 0 && (lanes_h == 4 || lanes_h == 8 || lanes_h == 16) && slots <= kRing;
  const size_t cut = sizeof(unsigned) * a.max_pages;
  const size_t smem = sizeof(float) * 2 * a.W + (vec && slots > cut ? slots : cut);
  auto kern = vec ? select_kernel<DT, true> : select_kernel<DT, false>;
  const cudaError_t e = allow_shared(kern, smem, kStatic);
  if (e != cudaSuccess) return e;
  kern<<<grid, kThreads, smem, st>>>(a);
  count_launch();
  return cudaGetLastError();
}

}  // namespace

size_t select_workspace(const palu_config* c, int batch, int num_queries, int max_pages) {
  const size_t G = (size_t)(c->num_heads / c->group_size);
  return sizeof(DevStatus) + sizeof(unsigned) * PALU_SELECT_MAX_LISTS +
         align256(sizeof(double) * batch * G * num_queries * max_pages) +
         align256(2 * sizeof(float) * batch * G * num_queries * max_pages);   // scores, and no more errs than pages
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
  a.chunk = chunk_of((long long)batch * a.G * num_queries, max_pages);
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
  const size_t n = (size_t)batch * a.G * num_queries * max_pages;
  a.exact = reinterpret_cast<double*>(ws + sizeof(DevStatus) + sizeof(unsigned) * PALU_SELECT_MAX_LISTS);
  a.scores = reinterpret_cast<float*>(reinterpret_cast<char*>(a.exact) + align256(sizeof(double) * n));
  a.errs = a.scores + n;
  for (int i = 0; i < kMaxHalfDim; ++i) a.omega[i] = omega[i];
  if (c->act_dtype == PALU_F32) return launch<PALU_F32>(a, st);
  if (c->act_dtype == PALU_F16) return launch<PALU_F16>(a, st);
  return launch<PALU_BF16>(a, st);
}

}  // namespace palu
