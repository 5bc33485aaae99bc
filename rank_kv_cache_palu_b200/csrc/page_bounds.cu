// Page bounds: the least and largest rebuilt, rotated key entry of every page,
// group and channel, from the cached latents.
//
//   k_t = R(pos_t)(z_k,t · B_k),  lo_c = min_t k_t,c,  hi_c = max_t k_t,c,
// rounded outwards into the compute dtype.
//
// Tensor-core kernel (16-bit or int4 latents, 128-token pages, head_dim 128): the
// product is taken transposed, Dᵀ[channel × token] = B_kᵀ · z_kᵀ, so that a thread
// owns a channel and meets its tokens in consecutive TMEM columns: the minimum
// over the page then needs no exchange between lanes (with tokens on the lanes it
// would take a 5-step shuffle for each of 512 channels).  A rotation pairs channel
// i with i + 64, so the two halves of a head pair go into two 128-lane tiles
// (lanes 0-63 the first head, 64-127 the second) and the same lane of both holds
// the pair.  Tokens of a page have consecutive positions: the key is rotated by the
// token's offset within 16 (16 angles a thread keeps in registers), then by the
// angle of the 16-token run's start.  At explicit positions every token has its own angle,
// from Taylor sums: the hardware's sine is off by up to 2^-21, and a key outside its box
// could drop a page that matters (64 pages 33.6 us, 27.3 with the hardware's, in packed
// pairs 32.4).
//
// One CTA keeps the B_k of a head pair (128 KB) and walks pages: a bulk-copy
// producer streams the page's column blocks through a ring (int4: four warps
// convert codes into it), one thread issues the MMAs into one of two TMEM slots,
// two warpgroups take half of the tokens each.  Bound by the MMAs at large sizes
// (2·128·r_k·W flops per page and group), by the B_k load and one page's latency
// at a decode step's one page per sequence.  Measured in the 7B shape (8 groups of 4
// heads, r_k 256, bf16): 64 pages 18.9 us (0.91 PFLOP/s with the start-up; 8 tiles a CTA
// of ~2.2k cycles, 2.05k of them MMA), one page of each of 16 sequences 9.7 us.
//
// Every other shape, and float32, takes the CUDA-core kernel, bound by its FMAs and, for
// a page or two, by latency (two float32 heads of 64, r_k 64, 2 pages: 18 us).
#include "decode_tc_kernel.cuh"
#include "simt_keys.cuh"

namespace palu {
namespace {
namespace pb {

using namespace tc;

constexpr int kNZ = 5;            // ring stages of 16 KB
constexpr int kMaxSeqs = 2048;    // sequences one launch enumerates
constexpr int kSlotCols = 256;    // TMEM columns per item: two 128-token tiles

struct BoundsArgs {
  int batch, d_h, gs, G, W, P, max_pages, num_pages;
  int rope, act, lat;
  const int32_t* first;
  const int32_t* pos_pool;
  const int32_t* page_table;
  const int32_t* seq_lens;
  const void* Bk;
  int bk_rows, bk_box, max_rk;
  void* bounds;
  DevStatus* st;
  GroupMap gm;
  uint64_t omega[kMaxHalfDim];
  long long wait_cycles;
  int stall_test;
};

// Cached tokens of sequence b (checked) and its first page to rebuild.
__device__ __forceinline__ int tokens_of(const BoundsArgs& a, int b, bool say) {
  int T = a.seq_lens[b];
  const int cap = a.max_pages * a.P;
  if (T < 0 || T > cap) {
    if (say) report(a.st, PALU_ERR_DEVICE_BOUNDS, 1000000 + b);
    T = T < 0 ? 0 : cap;
  }
  return T;
}
__device__ __forceinline__ int first_page(const BoundsArgs& a, int b) {
  return a.first == nullptr ? 0 : max(0, a.first[b]) / a.P;
}

// Rounded down (least entry) and up (largest).
template <int DT> struct Out;
template <> struct Out<PALU_F32> {
  __device__ __forceinline__ static float down(float v) { return v; }
  __device__ __forceinline__ static float up(float v) { return v; }
};
template <> struct Out<PALU_F16> {
  __device__ __forceinline__ static __half down(float v) { return __float2half_rd(v); }
  __device__ __forceinline__ static __half up(float v) { return __float2half_ru(v); }
};
template <> struct Out<PALU_BF16> {
  __device__ __forceinline__ static __nv_bfloat16 down(float v) { return __float2bfloat16_rd(v); }
  __device__ __forceinline__ static __nv_bfloat16 up(float v) { return __float2bfloat16_ru(v); }
};

// ---------------------------------------------------------------- CUDA cores
// One CTA per (page, head): the keys of the page's tokens in passes of 128 (64 for
// heads wider than 64; simt_keys.cuh), rotated and reduced in the threads, then over
// the token runs.
template <int ACT, int LAT>
__global__ void __launch_bounds__(kKeyThreads) bounds_simt_kernel(const __grid_constant__ BoundsArgs a) {
  using TA = typename Dt<ACT>::T;
  extern __shared__ __align__(16) float zt[];
  const int h = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
  const int g = h / a.gs, jh = h % a.gs;
  const int r_k = a.gm.rk[g], half = a.d_h / 2;
  const int lanes = key_lanes(half), tokens = key_tokens(half);
  const int i = tid % lanes, run = tid / lanes;
  const int T = tokens_of(a, b, tid == 0 && blockIdx.x == 0 && h == 0);
  const int npg = page_count(T, a.P);
  const TA* Bk = reinterpret_cast<const TA*>(a.Bk) + (size_t)a.gm.k_row0[g] * a.W + jh * a.d_h;
  for (int lp = first_page(a, b) + blockIdx.x; lp < npg; lp += gridDim.x) {
    const int page = a.page_table[(size_t)b * a.max_pages + lp];
    if (page < 0 || page >= a.num_pages) {
      if (tid == 0) report(a.st, PALU_ERR_DEVICE_BOUNDS, 2000000 + b);
      continue;
    }
    const int rows = min(a.P, T - lp * a.P);
    const uint8_t* blk = a.gm.zk[g] + (size_t)page * a.gm.k_page;
    const uint8_t* sblk = LAT == PALU_INT4 ? a.gm.zks[g] + (size_t)page * a.gm.ks_page : nullptr;
    float lo1 = INFINITY, hi1 = -INFINITY, lo2 = INFINITY, hi2 = -INFINITY;   // channels i, i + half
    for (int t0 = 0; t0 < rows; t0 += tokens) {
      const int nt = min(tokens, rows - t0);
      float k1[kKeyRun], k2[kKeyRun];
      rebuild_keys<ACT, LAT>(blk, sblk, a.P, t0, nt, r_k, Bk, a.W, half, zt, k1, k2);
#pragma unroll
      for (int t = 0; t < kKeyRun; ++t) {
        const int tt = run * kKeyRun + t;
        if (tt >= nt || i >= half) continue;
        float v1 = k1[t], v2 = k2[t];
        if (a.rope) {
          const int pos = a.pos_pool != nullptr ? a.pos_pool[(size_t)page * a.P + t0 + tt] : lp * a.P + t0 + tt;
          float c, s;
          rope_cs_accurate(pos, a.omega[i], c, s);
          v1 = k1[t] * c - k2[t] * s;
          v2 = k2[t] * c + k1[t] * s;
        }
        lo1 = fminf(lo1, v1);
        hi1 = fmaxf(hi1, v1);
        lo2 = fminf(lo2, v2);
        hi2 = fmaxf(hi2, v2);
      }
    }
    __syncthreads();   // the staging buffer takes the runs' results: [run][lo1, hi1, lo2, hi2][pair]
    float* x = zt + run * 4 * lanes + i;
    x[0] = lo1;
    x[lanes] = hi1;
    x[2 * lanes] = lo2;
    x[3 * lanes] = hi2;
    __syncthreads();
    if (tid < half) {
      for (int w = 1; w < kKeyThreads / lanes; ++w) {
        const float* y = zt + w * 4 * lanes + tid;
        lo1 = fminf(lo1, y[0]);
        hi1 = fmaxf(hi1, y[lanes]);
        lo2 = fminf(lo2, y[2 * lanes]);
        hi2 = fmaxf(hi2, y[3 * lanes]);
      }
      TA* o = reinterpret_cast<TA*>(a.bounds) + ((size_t)page * a.G + g) * 2 * a.W + jh * a.d_h + tid;
      o[0] = Out<ACT>::down(lo1);
      o[half] = Out<ACT>::down(lo2);
      o[a.W] = Out<ACT>::up(hi1);
      o[a.W + half] = Out<ACT>::up(hi2);
    }
  }
}

template <int ACT, int LAT>
cudaError_t launch_simt(const BoundsArgs& a, cudaStream_t st) {
  const size_t smem = sizeof(float) * key_stage_floats(a.d_h / 2);
  // pages of a sequence: enough CTAs for ~16 per SM, each stepping over the rest
  const long long rows = (long long)a.G * a.gs * a.batch;
  long long x = (16LL * 148 + rows - 1) / rows;
  x = x < 1 ? 1 : x > a.max_pages ? a.max_pages : x;
  bounds_simt_kernel<ACT, LAT><<<dim3((int)x, a.G * a.gs, a.batch), kKeyThreads, smem, st>>>(a);
  count_launch();
  return cudaGetLastError();
}

// ---------------------------------------------------------------- tensor cores
struct Layout {
  uint32_t zk, xch, prefix, bars, tmem_slot, abort, b, total;
};
__host__ __device__ inline Layout layout(int r_k) {
  Layout s{};
  uint32_t o = 0;
  s.zk = o;       o += kNZ * kZkBytes;
  s.xch = o;      o += 2 * 4 * 128 * 4;           // [slot][lo1, hi1, lo2, hi2][row] of warpgroup 1
  s.prefix = o;   o += (kMaxSeqs + 1) * 4 + 12;
  s.bars = o;     o += 24 * 8;
  s.tmem_slot = o; o += 16;
  s.abort = o;    o += 16;
  o = (o + 1023u) & ~1023u;
  s.b = o;        o += (uint32_t)r_k * 256 * 2;
  s.total = o;
  return s;
}
enum {
  B_BK = 0,
  B_ZK_FULL = 1,
  B_ZK_EMPTY = B_ZK_FULL + kNZ,
  B_D_FULL = B_ZK_EMPTY + kNZ,   // 2
  B_D_EMPTY = B_D_FULL + 2,      // 2
  B_XCH = B_D_EMPTY + 2,         // 2: warpgroup 1 posted its half of the tokens
  B_TEARDOWN = B_XCH + 2,
  B_COUNT
};
static_assert(B_COUNT <= 24, "barrier space");

struct Item {
  int b, lp, page, nv;   // page -1: outside the pool
};

// Item `idx` of the launch's enumeration of (sequence, page), all lanes of a warp together.
__device__ __forceinline__ Item item_of(const BoundsArgs& a, const int* prefix, int idx) {
  const int lane = threadIdx.x & 31;
  int lo = 0;   // sequences whose prefix end is <= idx, 32 at a time
  int b = 0;
  while (true) {
    const int i = lo + lane;
    const bool passed = i < a.batch && prefix[i + 1] <= idx;
    const unsigned m = __ballot_sync(0xffffffffu, passed);
    if (m != 0xffffffffu) {
      b = lo + __popc(m);
      break;
    }
    lo += 32;
  }
  Item it;
  it.b = b;
  it.lp = first_page(a, b) + idx - prefix[b];
  const int cap = a.max_pages * a.P;
  int T = a.seq_lens[b];
  T = T < 0 ? 0 : T > cap ? cap : T;
  it.nv = min(a.P, T - it.lp * a.P);
  const int pg = a.page_table[(size_t)b * a.max_pages + it.lp];
  it.page = (pg < 0 || pg >= a.num_pages) ? -1 : pg;
  return it;
}

template <int ACT, int LAT, bool CONTIG>
__global__ void __launch_bounds__(LAT == PALU_INT4 ? 512 : 384, 1)
    bounds_tc_kernel(const __grid_constant__ CUtensorMap tm_bk, const __grid_constant__ BoundsArgs a) {
  constexpr bool kInt4 = LAT == PALU_INT4;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* sbase = smem_raw + (base - raw);
  const int gi = blockIdx.y / (a.gs / 2), hp = blockIdx.y % (a.gs / 2);
  const int r_k = a.gm.rk[gi];
  const int nkc = r_k / kChunk;
  const Layout L = layout(r_k);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sbase + L.abort);
  int* prefix = reinterpret_cast<int*>(sbase + L.prefix);
  auto bar = [&](int i) { return base + L.bars + 8u * i; };

  if (threadIdx.x == 0) {
    abort_init(abort_flag, a.wait_cycles);
    mbar_init(bar(B_BK), 1);
    for (int i = 0; i < kNZ; ++i) {
      mbar_init(bar(B_ZK_FULL + i), kInt4 ? 4 : 1);
      mbar_init(bar(B_ZK_EMPTY + i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(B_D_FULL + i), 1);
      mbar_init(bar(B_D_EMPTY + i), 8);
      mbar_init(bar(B_XCH + i), 4);
    }
    mbar_init(bar(B_TEARDOWN), 1);
    fence_mbar_init();
    fence_proxy_async();
    // B_k of the head pair: four 64-column blocks, 0 and 1 the halves of the first head
    prefetch_tmap(&tm_bk);
    mbar_expect_tx(bar(B_BK), (uint32_t)r_k * 256 * 2);
    for (int nb = 0; nb < 4; ++nb)
      for (int rb = 0; rb < r_k; rb += a.bk_box)
        tma_load_2d(base + L.b + (uint32_t)nb * r_k * 128 + rb * 128, &tm_bk, hp * 256 + nb * 64,
                    a.gm.k_row0[gi] + rb, bar(B_BK));
  }
  if (warp == 1) {
    tmem_alloc(base + L.tmem_slot, 512);
    tmem_relinquish();
  }
  // prefix[b] = pages to rebuild in the sequences before b (warp 2: 32 sequences at a time)
  if (warp == 2) {
    int run = 0;
    if (lane == 0) prefix[0] = 0;
    for (int b0 = 0; b0 < a.batch; b0 += 32) {
      const int b = b0 + lane;
      int n = 0;
      if (b < a.batch) {
        const int T = tokens_of(a, b, blockIdx.x == 0 && blockIdx.y == 0);
        n = max(0, page_count(T, a.P) - first_page(a, b));
      }
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, n, off);
        if (lane >= off) n += o;
      }
      if (b < a.batch) prefix[b + 1] = run + n;
      run += __shfl_sync(0xffffffffu, n, 31);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(sbase + L.tmem_slot);
  const int total = prefix[a.batch];
  const int n_items = (int)blockIdx.x < total ? (total - 1 - (int)blockIdx.x) / (int)gridDim.x + 1 : 0;
  auto item = [&](int k) { return item_of(a, prefix, (int)blockIdx.x + k * (int)gridDim.x); };

  if (warp >= 4 && warp < 12) {
    // ============================================================ epilogue (warps 4-11)
    const int wg = (warp - 4) >> 2, q4 = warp & 3;
    const int row = q4 * 32 + lane;               // channel: head row / 64 of the pair, frequency row % 64
    const int f = row & 63;
    const uint32_t lane_addr = (uint32_t)(q4 * 32) << 16;
    const uint64_t om = a.omega[f];
    float* xch = reinterpret_cast<float*>(sbase + L.xch);
    f2 ce[8], se[8], ne[8];                       // cos, sin, -sin of the offsets 0..15 within a run
    if (CONTIG) {
#pragma unroll
      for (int v = 0; v < 8; ++v) {
        float c0, s0, c1, s1;
        rope_cs_accurate(2 * v, om, c0, s0);
        rope_cs_accurate(2 * v + 1, om, c1, s1);
        ce[v] = f2_pack(c0, c1);
        se[v] = f2_pack(s0, s1);
        ne[v] = f2_pack(-s0, -s1);
      }
    }
    bool ok = true;
    for (int k = 0; k < n_items && ok; ++k) {
      const Item it = item(k);
      const int slot = k & 1;
      if (!mbar_wait(bar(B_D_FULL + slot), (k >> 1) & 1, abort_flag, a.st, 41)) { ok = false; break; }
      tc_fence_after();
      float lo1 = INFINITY, hi1 = -INFINITY, lo2 = INFINITY, hi2 = -INFINITY;
      const int c0 = wg * 64;
      const int c1 = min(c0 + 64, it.nv);
#pragma unroll 1
      for (int cb = c0; cb < c1; cb += 16) {
        float k1[16], k2[16];
        const uint32_t col = tmem + lane_addr + (uint32_t)slot * kSlotCols + cb;
        tmem_ld16(col, k1);
        tmem_ld16(col + 128, k2);
        float C = 1.f, S = 0.f;
        if (CONTIG && a.rope) rope_cs_accurate(it.lp * kTile + cb, om, C, S);
        tmem_wait_ld();
        if (CONTIG) {
          if (a.rope) {
            const f2 C2 = f2_pack(C, C), S2 = f2_pack(S, S), N2 = f2_pack(-S, -S);
#pragma unroll
            for (int v = 0; v < 8; ++v) {
              const f2 x = f2_pack(k1[2 * v], k1[2 * v + 1]), y = f2_pack(k2[2 * v], k2[2 * v + 1]);
              const f2 u = f2_fma(x, ce[v], f2_mul(y, ne[v])), w = f2_fma(y, ce[v], f2_mul(x, se[v]));
              f2_unpack(f2_fma(u, C2, f2_mul(w, N2)), k1[2 * v], k1[2 * v + 1]);
              f2_unpack(f2_fma(w, C2, f2_mul(u, S2)), k2[2 * v], k2[2 * v + 1]);
            }
          }
        } else if (a.rope) {
          const int32_t* pp = a.pos_pool + (size_t)max(it.page, 0) * a.P + cb;
#pragma unroll
          for (int v = 0; v < 16; ++v) {
            float c, s;
            rope_cs_taylor(pp[v], om, c, s);
            const float x = k1[v], y = k2[v];
            k1[v] = x * c - y * s;
            k2[v] = y * c + x * s;
          }
        }
        if (cb + 16 > c1) {   // the page's last run: rows past the sequence are left out
#pragma unroll
          for (int v = 0; v < 16; ++v) {
            if (cb + v < c1) {
              lo1 = fminf(lo1, k1[v]);
              hi1 = fmaxf(hi1, k1[v]);
              lo2 = fminf(lo2, k2[v]);
              hi2 = fmaxf(hi2, k2[v]);
            }
          }
        } else {
#pragma unroll
          for (int v = 0; v < 16; ++v) {
            lo1 = fminf(lo1, k1[v]);
            hi1 = fmaxf(hi1, k1[v]);
            lo2 = fminf(lo2, k2[v]);
            hi2 = fmaxf(hi2, k2[v]);
          }
        }
      }
      float* x = xch + slot * 512 + row;
      if (wg == 1) {
        x[0] = lo1;
        x[128] = hi1;
        x[256] = lo2;
        x[384] = hi2;
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_XCH + slot));
      } else {
        if (!mbar_wait(bar(B_XCH + slot), (k >> 1) & 1, abort_flag, a.st, 42)) { ok = false; break; }
        lo1 = fminf(lo1, x[0]);
        hi1 = fmaxf(hi1, x[128]);
        lo2 = fminf(lo2, x[256]);
        hi2 = fmaxf(hi2, x[384]);
      }
      // the exchange buffer of this slot is read before the slot is released, so the
      // next item in it cannot overwrite what warpgroup 0 still needs
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(B_D_EMPTY + slot));
      if (wg == 0 && it.page >= 0) {
        using TA = typename Dt<ACT>::T;
        TA* o = reinterpret_cast<TA*>(a.bounds) + ((size_t)it.page * a.G + a.gm.g[gi]) * 2 * a.W +
                (hp * 2 + (row >> 6)) * 128 + f;
        o[0] = Out<ACT>::down(lo1);
        o[64] = Out<ACT>::down(lo2);
        o[a.W] = Out<ACT>::up(hi1);
        o[a.W + 64] = Out<ACT>::up(hi2);
      }
    }
  } else if (warp == 0 && !kInt4) {
    // ============================================================ z_k producer (bulk copies)
    int stage = 0;
    uint32_t phase = 0;
    long long issued = 0;
    for (int k = 0; k < n_items && !*abort_flag; ++k) {
      const Item it = item(k);
      __syncwarp();
      if (lane == 0) {
        int pg = it.page;
        if (pg < 0) {
          report(a.st, PALU_ERR_DEVICE_BOUNDS, 2000000 + it.b);
          pg = 0;   // keep the pipeline fed from a valid page; nothing is written for this item
        }
        const uint8_t* src = a.gm.zk[gi] + (size_t)pg * a.gm.k_page;
        for (int c = 0; c < nkc; ++c) {
          if (!mbar_wait(bar(B_ZK_EMPTY + stage), phase ^ 1, abort_flag, a.st, 43)) break;
          mbar_expect_tx(bar(B_ZK_FULL + stage), kZkBytes);
          bulk_load(base + L.zk + stage * kZkBytes, src + (size_t)c * kZkBytes, kZkBytes, bar(B_ZK_FULL + stage));
          ++issued;
          if (++stage == kNZ) { stage = 0; phase ^= 1; }
        }
      }
      __syncwarp();
    }
    if (lane == 0) drain_ring(bar(B_ZK_FULL), kNZ, issued, a.st, 43);
  } else if (kInt4 && warp >= 12) {
    // ============================================================ int4 key codes (warps 12-15)
    // One token per thread: its row of codes (r_k / 2 = 128 bytes) and scales, loaded
    // an item ahead of the conversion.
    const int t = threadIdx.x - 384;
    uint4 cur[8], nxt[8], csc, nsc;
    auto load = [&](int k, uint4* raw, uint4& sc) {
      const Item it = item(k);
      int pg = it.page;
      if (pg < 0) {
        if (t == 0) report(a.st, PALU_ERR_DEVICE_BOUNDS, 2000000 + it.b);
        pg = 0;
      }
      const uint8_t* rowp = a.gm.zk[gi] + (size_t)pg * a.gm.k_page + t * 128;
#pragma unroll
      for (int u = 0; u < 8; ++u) raw[u] = __ldg(reinterpret_cast<const uint4*>(rowp + ((u ^ (t & 7)) << 4)));
      sc = __ldg(reinterpret_cast<const uint4*>(a.gm.zks[gi] + (size_t)pg * a.gm.ks_page + (size_t)t * 16));
    };
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    if (n_items > 0) load(0, nxt, nsc);
    for (int k = 0; k < n_items && ok && !*abort_flag; ++k) {
#pragma unroll
      for (int u = 0; u < 8; ++u) cur[u] = nxt[u];
      csc = nsc;
      if (k + 1 < n_items) load(k + 1, nxt, nsc);
      const uint16_t* s16 = reinterpret_cast<const uint16_t*>(&csc);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        if (!mbar_wait(bar(B_ZK_EMPTY + stage), phase ^ 1, abort_flag, a.st, 44)) { ok = false; break; }
        const uint32_t dst = base + L.zk + stage * kZkBytes + t * 128;
#pragma unroll
        for (int ub = 0; ub < 2; ++ub) {
          const uint4 r = cur[2 * c + ub];
          const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
          for (int m = 0; m < 4; ++m)
            st_shared_v4(dst + (((4 * ub + m) ^ (t & 7)) << 4), dequant8<ACT, false>(w[m], s16[2 * c + ub]));
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_ZK_FULL + stage));
        if (++stage == kNZ) { stage = 0; phase ^= 1; }
      }
    }
  } else if (warp == 1) {
    // ============================================================ MMA issuer
    // The whole warp goes through the loop, one lane issues: what the loop computes is then known to
    // be the same on every lane and stays in the registers the MMAs take their operands from.
    const bool leader = elect_one();
    constexpr int kBf = ACT == PALU_BF16 ? 1 : 0;
    const uint32_t idesc = idesc_f16(kBf, 1, 0, 128, 128);   // B_kᵀ MN-major, z_kᵀ K-major
    // operand descriptors at the first stage and chunk: the same half of the second head lies two blocks on
    const uint64_t z0 = sdesc(base + L.zk, 16, kZkSbo, kZkSwz);
    const uint64_t b0 = sdesc(base + L.b, 2u * (uint32_t)r_k * 128, 1024, kSw128);
    auto wait = [&](int i, uint32_t parity, int where) {
      return __all_sync(0xffffffffu, mbar_wait(bar(i), parity, abort_flag, a.st, where)) != 0;
    };
    int zs = 0;
    uint32_t zph = 0;
    // timeout-path test hook: first wait on a phase nothing completes before the teardown commit
    bool ok = a.stall_test == 0 || wait(B_TEARDOWN, 0, 45);
    ok = ok && wait(B_BK, 0, 46);
    for (int k = 0; k < n_items && ok; ++k) {
      const int slot = k & 1;
      if (!wait(B_D_EMPTY + slot, ((k >> 1) & 1) ^ 1, 47)) break;
      tc_fence_after();
      const uint32_t d = tmem + (uint32_t)slot * kSlotCols;
      for (int c = 0; c < nkc; ++c) {
        if (!wait(B_ZK_FULL + zs, zph, 48)) { ok = false; break; }
        tc_fence_after();
        const uint64_t z = desc_at(z0, (uint32_t)zs * kZkBytes), b = desc_at(b0, (uint32_t)c * kChunk * 128);
        const uint64_t b_hi = desc_at(b, (uint32_t)r_k * 128);
        if (leader) {
#pragma unroll
          for (int kk = 0; kk < kChunk / 16; ++kk) {
            umma_f16(d, desc_at(b, kk * 16 * 128), desc_at(z, kk * 32), idesc, (c | kk) != 0);
            umma_f16(d + 128, desc_at(b_hi, kk * 16 * 128), desc_at(z, kk * 32), idesc, (c | kk) != 0);
          }
          umma_commit(bar(B_ZK_EMPTY + zs));
        }
        if (++zs == kNZ) { zs = 0; zph ^= 1; }
      }
      if (!ok) break;
      if (leader) umma_commit(bar(B_D_FULL + slot));
    }
    // drain, also after an abort: MMAs complete before TMEM is released, the B_k load before the CTA exits
    if (leader) umma_commit(bar(B_TEARDOWN));
    __syncwarp();
    mbar_drain(bar(B_TEARDOWN), 0, a.st, 45);
    mbar_drain(bar(B_BK), 0, a.st, 46);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int ACT, int LAT>
cudaError_t launch_tc(const BoundsArgs& all, cudaStream_t st) {
  const CUtensorMapDataType dt = ACT == PALU_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  CUtensorMap tm;
  if (!make_map_2d(&tm, all.Bk, dt, 2, all.W, (uint64_t)all.bk_rows, (uint64_t)all.W * 2, 64, all.bk_box,
                   CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  const size_t smem = layout(all.max_rk).total + 1024;
  auto kern = all.pos_pool == nullptr ? bounds_tc_kernel<ACT, LAT, true> : bounds_tc_kernel<ACT, LAT, false>;
  cudaError_t e = allow_shared(kern, smem);
  if (e != cudaSuccess) return e;
  // one CTA per SM, the same number for every (group, head pair), each with its B_k resident
  const int combos = all.gm.n * (all.gs / 2);
  // sequences of one launch: their pages, and a step of the grid past them, are counted in 32 bits
  const int most_seqs = (INT32_MAX - 256) / all.max_pages < kMaxSeqs ? (INT32_MAX - 256) / all.max_pages : kMaxSeqs;
  for (int b0 = 0; b0 < all.batch; b0 += most_seqs) {
    BoundsArgs a = all;
    a.batch = all.batch - b0 < most_seqs ? all.batch - b0 : most_seqs;
    a.page_table += (size_t)b0 * a.max_pages;
    a.seq_lens += b0;
    if (a.first != nullptr) a.first += b0;
    long long per = 148 / combos;
    const long long most = (long long)a.batch * a.max_pages;   // pages there can be
    per = per < 1 ? 1 : per > most ? most : per;
    kern<<<dim3((int)per, combos), LAT == PALU_INT4 ? 512 : 384, smem, st>>>(tm, a);
    count_launch();
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

// The tensor-core kernel takes a layer when it takes each of its groups.
bool tc_ok(const palu_config* c, const GroupMap& gm) {
  if (c->head_dim != 128 || c->page_size != kTile || c->group_size % 2 != 0) return false;
  if (c->act_dtype != PALU_F16 && c->act_dtype != PALU_BF16) return false;
  for (int i = 0; i < gm.n; ++i) {
    if (c->latent_dtype == PALU_INT4 ? gm.rk[i] != 256 : gm.rk[i] % 64 != 0 || gm.rk[i] > 256) return false;
  }
  return true;
}

}  // namespace pb
}  // namespace

cudaError_t launch_page_bounds(const palu_config* c, const GroupMap& gm, int bk_rows, int batch, const int32_t* first,
                               const int32_t* pos_pool, const int32_t* page_table, int max_pages,
                               const int32_t* seq_lens, int num_pages, const void* B_k, void* bounds,
                               const uint64_t* omega, void* workspace, cudaStream_t st) {
  pb::BoundsArgs a{};
  a.batch = batch;
  a.d_h = c->head_dim;
  a.gs = c->group_size;
  a.G = c->num_heads / c->group_size;
  a.W = c->group_size * c->head_dim;
  a.P = c->page_size;
  a.max_pages = max_pages;
  a.num_pages = num_pages;
  a.rope = c->rope_base != 0.f;
  a.act = c->act_dtype;
  a.lat = c->latent_dtype;
  a.first = first;
  a.pos_pool = pos_pool;
  a.page_table = page_table;
  a.seq_lens = seq_lens;
  a.Bk = B_k;
  a.bk_rows = bk_rows;
  a.bounds = bounds;
  a.st = static_cast<DevStatus*>(workspace);
  a.gm = gm;
  for (int i = 0; i < gm.n; ++i) a.max_rk = gm.rk[i] > a.max_rk ? gm.rk[i] : a.max_rk;
  a.bk_box = a.max_rk;
  for (int i = 0; i < gm.n; ++i)
    if (gm.rk[i] != a.max_rk) a.bk_box = 64;   // mixed key ranks: boxes of 64 rows
  for (int i = 0; i < kMaxHalfDim; ++i) a.omega[i] = omega[i];
  a.wait_cycles = timeout_test_setting().wait_cycles;
  a.stall_test = timeout_test_setting().stall;
  const bool int4 = c->latent_dtype == PALU_INT4, bf = c->act_dtype == PALU_BF16;
  if (pb::tc_ok(c, gm)) {
    if (int4)
      return bf ? pb::launch_tc<PALU_BF16, PALU_INT4>(a, st) : pb::launch_tc<PALU_F16, PALU_INT4>(a, st);
    return bf ? pb::launch_tc<PALU_BF16, PALU_BF16>(a, st) : pb::launch_tc<PALU_F16, PALU_F16>(a, st);
  }
  if (c->act_dtype == PALU_F32) return pb::launch_simt<PALU_F32, PALU_F32>(a, st);
  if (int4)
    return bf ? pb::launch_simt<PALU_BF16, PALU_INT4>(a, st) : pb::launch_simt<PALU_F16, PALU_INT4>(a, st);
  return bf ? pb::launch_simt<PALU_BF16, PALU_BF16>(a, st) : pb::launch_simt<PALU_F16, PALU_F16>(a, st);
}

}  // namespace palu
