// Tensor-core split kernel of the sparse decode step (palu_decode_attn_pages):
// sm_100a, TMA + tcgen05 + TMEM.
//
// Method: "PALU 论文低秩投影分解" §把它放进一次真实推理流程里看, Decode 阶段 (keys
// rebuilt from the cached latents tile by tile, rotated at their positions; values
// kept in latent space), over the pages of a list per query and head group.
//
// The tile pipeline is that of decode_tc_kernel.cuh (roles of the warps, rings, TMEM
// slots, RoPE by angle addition, value sums into the next tile's slot).  What differs:
//   - A CTA walks an equal share of all lists of its head pair (pages_walk.cuh), not a
//     page range of one sequence: lists are short (16 pages and 2 of start-up for each
//     CTA of its own left the tensor pipe idle a third of the time), so B_k is loaded
//     once and the pipeline runs on from list to list.  A segment's last value sums are
//     folded in the next segment's first tile, where its partial is written.
//   - The rotated query changes with the segment: three buffers, filled two tiles ahead.
//   - The softmax weights reach the value MMA as sums of three 16-bit numbers (split_weight).
//   - The MMA warp runs its loop converged and one lane issues.  With the loop on one lane
//     its operands went through lane registers and every group of MMAs took 700 to 850 cycles
//     to issue, which set the tile period (16 queries x 32 pages bf16: 170 us; with descriptors
//     made by one addition 163; converged 143.  int4, 32 queries x 16 pages: 266, 258, 245).
// Measured in the 7B shape, r 256/128 bf16, 16 queries x 32 pages in each of 8 groups: 139 to 149 us by the GPU
// with the merge (0.93 PFLOP/s of key and value products or more, 0.56 of the burst peak), bound as the dense kernel by
// the coupling of the operand rings to the TMEM slots; one query x 16 pages 18.1 us.  int4, r 256/256, 8 sequences x 4 queries x
// 16 pages: 231 to 236 us, bound by the conversion of codes.
#pragma once

#include "decode_tc_kernel.cuh"
#include "pages_walk.cuh"

namespace palu {
namespace {

struct PagesSmem {
  uint32_t zk, zv, p, qr, psc, tb, red, bars, tmem_slot, abort, tiles, b, total;
};

// As smem_layout, with three query buffers and the walk's tiles; the base is
// 1024-aligned by declaration, so that everything fits 227 KB at r_k = 256.
__host__ __device__ inline PagesSmem pages_smem(int r_k, bool int4) {
  PagesSmem s{};
  uint32_t o = 0;
  s.zk = o;     o += zk_stages(int4) * kZkBytes;
  s.zv = o;     o += zv_stages(int4) * kZvBytes;
  s.p = o;      o += 2 * kPBytes;
  s.qr = o;     o += 3 * 2 * 128 * 4;
  s.psc = o;    o += 2 * 2 * 128 * 4;
  s.tb = o;     o += 2 * 2 * 2 * 3 * 32 * 4;             // [warpgroup][tile parity][head][A|B|-A][32 freq]
  s.red = o;    o += 2 * 4 * 2 * 4;
  s.bars = o;   o += 32 * 8;
  s.tmem_slot = o; o += 16;
  s.abort = o;  o += 16;
  s.tiles = o;  o += kWalkTiles * sizeof(Tile);
  o = (o + 1023u) & ~1023u;                              // 128-byte-swizzle atoms: 1024-byte aligned
  s.b = o;      o += (uint32_t)r_k * 256 * 2;            // B_k for 2 heads
  s.total = o;
  return s;
}
static_assert((kWalkUnits + 1) * 4 <= 2 * kZkBytes, "the walk's prefix sums fit the z_k ring");

template <int ACT, int NRV, int LAT, bool CONTIG>
__global__ void __launch_bounds__(threads_of(LAT == PALU_INT4), 1)
    decode_pages_kernel(const __grid_constant__ CUtensorMap tm_bk, const __grid_constant__ DecodeArgs a) {
  extern __shared__ __align__(1024) uint8_t sbase[];
  const uint32_t base = smem_u32(sbase);
  // blockIdx.y: entry gi of the group map and head pair hp; the entry's key rank sets the layout
  const int gi = blockIdx.y / (a.gs / 2), hp = blockIdx.y % (a.gs / 2);
  const int r_k = a.gm.rk[gi];
  const PagesSmem L = pages_smem(r_k, LAT == PALU_INT4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr bool kInt4 = LAT == PALU_INT4;
  constexpr int kNZK = zk_stages(kInt4);
  constexpr int kNVS = zv_stages(kInt4);
  constexpr int BAR_ZK_FULL = BAR_RINGS, BAR_ZK_EMPTY = BAR_ZK_FULL + kNZK;
  constexpr int BAR_ZV_FULL = BAR_ZK_EMPTY + kNZK, BAR_ZV_EMPTY = BAR_ZV_FULL + kNVS;
  constexpr int kThreads = threads_of(kInt4);
  static_assert(!kInt4 || NRV == 2, "int4 latents: r_v = 256");
  DevStatus* st = reinterpret_cast<DevStatus*>(a.status);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sbase + L.abort);
  auto bar = [&](int i) { return base + L.bars + 8u * i; };

  const GroupMap& gm = a.gm;
  const int nkc = r_k / kChunk;
  const uint32_t k_blk_bytes = (uint32_t)a.P * (kInt4 ? r_k / 2 : 2 * r_k);   // this entry's block of a page
  const Tile* tiles = reinterpret_cast<const Tile*>(sbase + L.tiles);

  start_next();      // the merge; its CTAs find room as this launch's leave
  // ---------------------------------------------------------------- setup
  if (threadIdx.x == 0) {
    abort_init(abort_flag, a.wait_cycles);
    mbar_init(bar(BAR_B), 1);
    for (int i = 0; i < kNZK; ++i) {
      mbar_init(bar(BAR_ZK_FULL + i), kInt4 ? 4 : 1);   // int4: one arrival per converting warp
      mbar_init(bar(BAR_ZK_EMPTY + i), 1);
    }
    for (int i = 0; i < kNVS; ++i) {
      mbar_init(bar(BAR_ZV_FULL + i), kInt4 ? 3 : 1);
      mbar_init(bar(BAR_ZV_EMPTY + i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(BAR_D_FULL + i), 1);
      mbar_init(bar(BAR_D_EMPTY + i), 8);
      mbar_init(bar(BAR_P_FULL + i), 8);
    }
    mbar_init(bar(BAR_AT_FULL), 1);
    mbar_init(bar(BAR_TEARDOWN), 1);
    mbar_init(bar(BAR_QR), 4);
    mbar_init(bar(BAR_MID), 8);
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(BAR_EPI + i), 4);
      mbar_init(bar(BAR_XCH + i), 8);
    }
    fence_mbar_init();
    fence_proxy_async();
    // B_k of the head pair: on its way while the walk is laid out
    prefetch_tmap(&tm_bk);
    mbar_expect_tx(bar(BAR_B), (uint32_t)r_k * 256 * 2);
    // 64-column blocks of B_k (MN-major, 128-byte swizzle), each in boxes of bk_box rows
    // int4 latents: the rows (latent entries) in the key converters' paired order, row
    // 8g + 2a + b of shared memory = row 8g + 4b + a of B_k (a 4-D view of B_k, see the launcher)
    for (int nb = 0; nb < 4; ++nb)
      for (int rb = 0; rb < r_k; rb += a.bk_box) {
        if constexpr (kInt4)
          tma_load_4d(base + L.b + (uint32_t)nb * r_k * 128 + rb * 128, &tm_bk, hp * 256 + nb * 64, 0, 0,
                      (gm.k_row0[gi] + rb) / 8, bar(BAR_B));
        else
          tma_load_2d(base + L.b + (uint32_t)nb * r_k * 128 + rb * 128, &tm_bk, hp * 256 + nb * 64,
                      gm.k_row0[gi] + rb, bar(BAR_B));
      }
  }
  if (warp == 1) {
    tmem_alloc(base + L.tmem_slot, 512);
    tmem_relinquish();
  }
  // zero the P buffers (padding rows stay zero)
  for (int i = threadIdx.x; i < 2 * kPBytes / 4; i += kThreads)
    reinterpret_cast<uint32_t*>(sbase + L.p)[i] = 0u;
  // this CTA's tiles; the prefix sums borrow the z_k ring, which nothing fills before the barrier below
  const int N = walk_tiles(a, gm.g[gi], gi, hp == 0, reinterpret_cast<Tile*>(sbase + L.tiles),
                           reinterpret_cast<int*>(sbase + L.zk), st);
  fence_proxy_async();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(sbase + L.tmem_slot);

  // Roles.  int4 latents: each warpgroup first sets its share of the register file
  // (setmaxnreg, see kRegsLaunch), inside the branch whose code uses it.
  if (kInt4 && warp >= 12) {
    if constexpr (kInt4) setmaxnreg_dec<kRegsKey>();
    // ============================================================ int4 key codes (warps 12-15)
    // Chunk c of a tile = entries [64c, 64c + 64) of all 128 tokens, i.e. scale
    // blocks 2c and 2c+1 = 16-byte units 2c and 2c+1 of each token's row of codes.
    // Thread t takes both units of token t, loaded straight into registers two
    // chunks ahead of the conversion, while later pages are pulled into L2.  Entries
    // are written PAIRED (K position p of the operand holds entry paired_row(p)), which
    // saves byte permutes; B_k's rows are loaded in the same order, so the key MMA sums
    // the same products.
    const int t = threadIdx.x - 384;
    const int NC = N * 4;
    struct Slot {
      uint4 raw[2];
      uint16_t sc[2];
    };
    auto prefetch_tile = [&](int k) {
      if (t != 0 || k >= N) return;
      const int ppg = max(tiles[k].page, 0);
      prefetch_l2(gm.zk[gi] + (size_t)ppg * gm.k_page, k_blk_bytes);
      prefetch_l2(gm.zks[gi] + (size_t)ppg * gm.ks_page, (uint32_t)(a.P * a.ks_row));
      prefetch_l2(gm.zv[gi] + (size_t)ppg * gm.v_page, (uint32_t)(a.P * a.v_row));
      prefetch_l2(gm.zvs[gi] + (size_t)ppg * gm.vs_page, (uint32_t)(a.P * a.vs_row));
    };
    // The issue slots of the SM are what this kernel runs out of, so addresses take few of them: unit u
    // of a token's 128-byte row lies at (row + 16 (t mod 8)) XOR 16 u, in a page as in a ring stage
    // (rows start on 128 bytes), and a page's pointers are made once per tile.
    const uint32_t row0 = (uint32_t)t * 128 + ((uint32_t)(t & 7) << 4);
    const uint8_t* codes = nullptr;
    const uint8_t* scales = nullptr;
    // Loads past the last chunk repeat the last tile's: a condition on them would let the slot take its
    // values through other registers, at the end of the iteration, when they have not come yet
    // (32 queries x 16 pages: 234 us so, 230 without).
    auto issue = [&](int n, Slot& sl) {
      const int c = n & 3;
      if (c == 0 && n < NC) {
        const size_t pg = (size_t)max(tiles[n >> 2].page, 0);   // of a bad page (reported): any page's, the result is void
        codes = gm.zk[gi] + pg * gm.k_page;
        scales = gm.zks[gi] + pg * gm.ks_page + (size_t)t * a.ks_row;
      }
#pragma unroll
      for (int ub = 0; ub < 2; ++ub) {
        sl.raw[ub] = __ldg(reinterpret_cast<const uint4*>(codes + (row0 ^ (uint32_t)(32 * c + 16 * ub))));
        sl.sc[ub] = __ldg(reinterpret_cast<const unsigned short*>(scales + 4 * c + 2 * ub));
      }
    };
    int stage = 0;
    uint32_t phase = 0;
    Slot s0, s1;                                       // chunks n and n + 1
    for (int kk = 1; kk <= kPrefetch; ++kk) prefetch_tile(kk);
    if (N > 0) {
      issue(0, s0);
      issue(1, s1);
    }
    // One load batch and one conversion per chunk: a single copy of the conversion
    // code keeps the kernel's instruction footprint small.  A slot is copied an iteration after
    // its loads went out (copied at once it would wait for them).
#pragma unroll 1
    for (int n = 0; n < NC; ++n) {
      if (!mbar_wait(bar(BAR_ZK_EMPTY + stage), phase ^ 1, abort_flag, st, 12)) break;
      const uint32_t dst = base + L.zk + stage * kZkBytes + row0;
#pragma unroll
      for (int ub = 0; ub < 2; ++ub) {
        const uint32_t w[4] = {s0.raw[ub].x, s0.raw[ub].y, s0.raw[ub].z, s0.raw[ub].w};
#pragma unroll
        for (int m = 0; m < 4; ++m) st_shared_v4(dst ^ (uint32_t)(64 * ub + 16 * m), dequant8<ACT, true>(w[m], s0.sc[ub]));
      }
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(BAR_ZK_FULL + stage));
      if (++stage == kNZK) { stage = 0; phase ^= 1; }
      s0 = s1;
      issue(n + 2, s1);
      if ((n & 3) == 0) prefetch_tile((n >> 2) + 1 + kPrefetch);
    }
  } else if (warp >= 4) {
    if constexpr (kInt4) setmaxnreg_inc<kRegsEpi>();
    // ============================================================ epilogue (warps 4-11)
    // Two warpgroups split the 64 RoPE frequency pairs of every key (wg 0:
    // pairs [0, 32), wg 1: [32, 64)) for both heads, then each finishes one head.
    const int wg = (warp - 4) >> 2;
    const int q4 = warp & 3;                 // TMEM lane quarter this warp may access
    const int row = q4 * 32 + lane;          // token row of the tile / latent row of aᵀ
    const uint32_t lane_addr = (uint32_t)(q4 * 32) << 16;
    float* qr = reinterpret_cast<float*>(sbase + L.qr);     // [segment mod 3][head][q'_i | q'_{i+64}]
    float* psc = reinterpret_cast<float*>(sbase + L.psc);   // [slot][head][128]
    const int head0 = gm.g[gi] * a.gs + hp * 2;   // model head of the pair's first head
    const int hl0 = gi * a.gs + hp * 2;           // the same head among this launch's heads
    constexpr float kLog2e = 1.4426950408889634f;
    // the 4 warps of one warpgroup meet here; a bounded wait (unlike bar.sync), so a thread that gave
    // up on a timed-out wait cannot strand the others.
    uint32_t epi_phase = 0;
    auto ep_sync = [&](int where) -> bool {
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(BAR_EPI + wg));
      const bool r = mbar_wait(bar(BAR_EPI + wg), epi_phase, abort_flag, st, where);
      epi_phase ^= 1;
      return r;
    };
    // The rotated query of both heads, scaled by log2(e)/sqrt(d_h) for exp2, a buffer
    // per segment: warpgroup 0 loads a segment's query two tiles ahead of its first tile
    // and stores it the same tile; three segments can be live then (the tile's own, the
    // next tile's, whose query is rotated to its first token, and the one being stored).
    const int qh = row >> 6, qi = row & 63;
    const uint64_t q_om = a.omega[qi];
    using TA = typename Dt<ACT>::T;
    TA qx1{}, qx2{};
    int qx_pos = 0;
    auto load_query = [&](int unit) {
      const TA* q = reinterpret_cast<const TA*>(a.q) + (size_t)unit * a.q_bstride + (size_t)(head0 + qh) * 128;
      qx1 = q[qi];
      qx2 = q[qi + 64];
      qx_pos = a.q_pos[unit];
    };
    auto store_query = [&](int seg) {
      const float x1 = Dt<ACT>::to_f(qx1), x2 = Dt<ACT>::to_f(qx2);
      float c = 1.f, s = 0.f;
      if (a.rope) rope_cs_taylor(qx_pos, q_om, c, s);
      const float sc = a.sm_scale * kLog2e;
      float* o = qr + (seg % 3) * 256 + qh * 128 + qi;
      o[0] = (x1 * c - x2 * s) * sc;
      o[64] = (x2 * c + x1 * s) * sc;
    };
    if (wg == 0) {
      if (N > 0) {
        load_query(tiles[0].unit);
        store_query(0);
      }
      if (N > 1 && (tiles[1].info & kTileFirst)) {
        load_query(tiles[1].unit);
        store_query(1);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(BAR_QR));
    }
    bool ok = mbar_wait(bar(BAR_QR), 0, abort_flag, st, 32);

    // Partial scores of both heads over this warpgroup's 32 frequency pairs i:
    //   score += c_i (q'_i k_i + q'_{i+64} k_{i+64}) + s_i (q'_{i+64} k_i - q'_i k_{i+64})
    // which is q'·k' with k' the key rotated by the token's angle (rotate-half).
    // Explicit positions take a sincos per token.  Contiguous positions (pos = t0 +
    // row): with (C, S) the cosine and sine at the tile start t0 and (c_r, s_r) those
    // at this thread's fixed offset `row`, angle addition turns the sum into
    //   score += c_r (k_i A_i + k_{i+64} B_i) + s_r (k_i B_i - k_{i+64} A_i),
    //   A_i = C q'_i + S q'_{i+64},  B_i = C q'_{i+64} - S q'_i,
    // i.e. the query rotated by the tile start, computed once per tile for the whole
    // warpgroup (double-buffered, published by the tile's softmax sync).  Math runs
    // on packed fp32 pairs (two frequencies at a time).
    constexpr bool contig = CONTIG;
    float* abuf = reinterpret_cast<float*>(sbase + L.tb) + wg * 384;   // [tile parity][head][A|B|-A][32]
    // Query and tile start take their angles from Taylor sums, 2^-23.5.  The row's, and a token's at
    // explicit positions, are the hardware's approximations, off by at most 2^-21: Taylor sums took one
    // query x 16 pages from 18.1 to 18.7 us (they delay the first tile), and 16 queries x 32 pages at
    // explicit positions from 165 to 201 us; the outputs came no nearer to float32's (5e-5 of them in
    // bf16, 2.2e-5 in f16, both by their last rounding).
    f2 crow[16], srow[16];
    if (contig) {
#pragma unroll
      for (int v = 0; v < 16; ++v) {
        float c0, s0, c1, s1;
        rope_cs_fast(row, a.omega[wg * 32 + 2 * v], c0, s0);
        rope_cs_fast(row, a.omega[wg * 32 + 2 * v + 1], c1, s1);
        crow[v] = f2_pack(c0, c1);
        srow[v] = f2_pack(s0, s1);
      }
    }
    // the query of segment seg rotated by the start t0 of a tile, for this warpgroup's
    // frequencies: thread row < 64 takes frequency row mod 32 of head row / 32
    const uint64_t t_om = a.omega[wg * 32 + (row & 31)];
    auto post_rotated_query = [&](int t0, int seg, int parity) {
      if (row >= 64) return;
      const int f = row & 31, hh = row >> 5;
      float c, sn;
      rope_cs_taylor(t0, t_om, c, sn);
      const float* q = qr + (seg % 3) * 256 + hh * 128 + wg * 32 + f;
      const float qa = q[0], qb = q[64];
      const float A = c * qa + sn * qb, B = c * qb - sn * qa;
      float* o = abuf + parity * 192 + hh * 96 + f;
      o[0] = A;
      o[32] = B;
      o[64] = -A;
    };
    auto half_scores = [&](int slot, int seg, int pos, float* part, auto&& mid) {
      const float* ab = abuf + slot * 192;
      f2 acc[2][2];
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) acc[hh][0] = acc[hh][1] = 0ull;
#pragma unroll
      for (int jj = 0; jj < kNB; ++jj) {
        mid(jj);   // halfway: signal that the first batches' columns are read
        const int i0 = wg * 32 + jj * kBatch;
        const uint32_t col = tmem + lane_addr + (uint32_t)slot * 256 + i0;
        // both heads' keys of these kBatch frequency pairs in one TMEM round trip
        float lo[2][kBatch], hi[2][kBatch];
        if constexpr (kBatch == 16) {
          tmem_ld16(col, lo[0]);
          tmem_ld16(col + 64, hi[0]);
          tmem_ld16(col + 128, lo[1]);
          tmem_ld16(col + 192, hi[1]);
        } else {
          tmem_ld8(col, lo[0]);
          tmem_ld8(col + 64, hi[0]);
          tmem_ld8(col + 128, lo[1]);
          tmem_ld8(col + 192, hi[1]);
        }
        tmem_wait_ld();
        if (contig) {
#pragma unroll
          for (int v4 = 0; v4 < kBatch / 4; ++v4) {
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
              const float* q = ab + hh * 96 + jj * kBatch + 4 * v4;
              const float4 A4 = *reinterpret_cast<const float4*>(q);
              const float4 B4 = *reinterpret_cast<const float4*>(q + 32);
              const float4 N4 = *reinterpret_cast<const float4*>(q + 64);
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int v = v4 * 2 + e, vr = jj * (kBatch / 2) + v;
                const f2 A2 = e ? f2_pack(A4.z, A4.w) : f2_pack(A4.x, A4.y);
                const f2 B2 = e ? f2_pack(B4.z, B4.w) : f2_pack(B4.x, B4.y);
                const f2 N2 = e ? f2_pack(N4.z, N4.w) : f2_pack(N4.x, N4.y);
                const f2 lo2 = f2_pack(lo[hh][2 * v], lo[hh][2 * v + 1]);
                const f2 hi2 = f2_pack(hi[hh][2 * v], hi[hh][2 * v + 1]);
                const f2 u = f2_fma(hi2, B2, f2_mul(lo2, A2));   // k_i A_i + k_{i+64} B_i
                const f2 w = f2_fma(lo2, B2, f2_mul(hi2, N2));   // k_i B_i - k_{i+64} A_i
                acc[hh][e] = f2_fma(crow[vr], u, acc[hh][e]);
                acc[hh][e] = f2_fma(srow[vr], w, acc[hh][e]);
              }
            }
          }
          continue;
        }
#pragma unroll
        for (int v4 = 0; v4 < kBatch / 4; ++v4) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int v = v4 * 2 + e;
            f2 cs, sn;
            {
              // explicit positions: a sincos per token
              float c0, s0, c1, s1;
              rope_cs_fast(pos, a.omega[i0 + 2 * v], c0, s0);
              rope_cs_fast(pos, a.omega[i0 + 2 * v + 1], c1, s1);
              cs = f2_pack(c0, c1);
              sn = f2_pack(s0, s1);
            }
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
              const float* q = qr + (seg % 3) * 256 + hh * 128 + i0 + 4 * v4 + 2 * e;
              const f2 a2 = *reinterpret_cast<const f2*>(q);
              const f2 b2 = *reinterpret_cast<const f2*>(q + 64);
              const f2 n2 = f2_pack(-q[0], -q[1]);
              const f2 lo2 = f2_pack(lo[hh][2 * v], lo[hh][2 * v + 1]);
              const f2 hi2 = f2_pack(hi[hh][2 * v], hi[hh][2 * v + 1]);
              const f2 x = f2_fma(b2, hi2, f2_mul(a2, lo2));     // q'_i k_i + q'_{i+64} k_{i+64}
              const f2 y = f2_fma(b2, lo2, f2_mul(n2, hi2));     // q'_{i+64} k_i - q'_i k_{i+64}
              acc[hh][e] = f2_fma(cs, x, acc[hh][e]);
              acc[hh][e] = f2_fma(sn, y, acc[hh][e]);
            }
          }
        }
      }
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        float a0, a1, a2, a3;
        f2_unpack(acc[hh][0], a0, a1);
        f2_unpack(acc[hh][1], a2, a3);
        part[hh] = (a0 + a1) + (a2 + a3);
      }
    };

    {
      // Each warpgroup owns one head of the pair (hw = wg) for the softmax, P,
      // the latent value sums and the output; the partial scores of the other
      // head go across in shared memory.
      const int hw = wg;
      // latent entry of TMEM lane `row` of aᵀ (int4: the value operand's units are PAIRED)
      const int vrow = kInt4 ? paired_row(row) : row;
      float m_run = -INFINITY, l_part = 0.f, prev_scale = 0.f;
      float m_prev = -INFINITY, l_prev = 0.f;      // of the segment whose last value sums are still to be folded
      float acc[NRV];
#pragma unroll
      for (int mb = 0; mb < NRV; ++mb) acc[mb] = 0.f;
      float* red = reinterpret_cast<float*>(sbase + L.red);
      constexpr float kLn2 = 0.6931471805599453f;

      // The value sums of tile j sit in the TMEM slot of tile j + 1 (columns [32·mb, +16); columns
      // hw, hw + 2 and hw + 4 of each block for the terms of this head's weights); fold them into
      // the running sums.
      auto fold_at = [&](int j) -> bool {
        if (!mbar_wait(bar(BAR_AT_FULL), j & 1, abort_flag, st, 30)) return false;
        tc_fence_after();
        const uint32_t sb = (uint32_t)((j + 1) & 1) * 256;
#pragma unroll
        for (int mb = 0; mb < NRV; ++mb) {
          const float v = tmem_ld1(tmem + lane_addr + sb + mb * 32 + hw);
          const float w = tmem_ld1(tmem + lane_addr + sb + mb * 32 + hw + 2);
          const float x = tmem_ld1(tmem + lane_addr + sb + mb * 32 + hw + 4);
          tmem_wait_ld();
          acc[mb] = fmaf(acc[mb], prev_scale, v + (w + x));
        }
        return true;
      };
      // The partial of the segment that tile t ends; the running value sums start over.
      auto finish = [&](const Tile& t, float m, float l) {
        float* out = segment_part(a, t, hl0 + hw);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
        if (!*abort_flag) {
          if (row == 0) out[0] = m * kLn2;
          if (lane == 0) out[1 + q4] = l;
#pragma unroll
          for (int mb = 0; mb < NRV; ++mb) out[kPartHead + mb * 128 + vrow] = acc[mb] * (1.f / kWeightScale<ACT>);
        }
#pragma unroll
        for (int mb = 0; mb < NRV; ++mb) acc[mb] = 0.f;
      };

      int seg = 0, qlim = 0;
      if (contig && N > 0) {
        post_rotated_query(tiles[0].lp * kTile, 0, 0);
        ok = ep_sync(37) && ok;
      }
      for (int k = 0; k < N && ok; ++k) {
        const Tile t = tiles[k];
        const int t0 = t.lp * kTile, rows = tile_rows(t.info);
        const int slot = k & 1;
        if (t.info & kTileFirst) {
          if (k > 0) ++seg;
          m_prev = m_run;
          l_prev = l_part;
          m_run = -INFINITY;
          l_part = 0.f;
          // causal bound (several queries per step): tokens after the query's position are masked
          if (a.causal) qlim = a.q_pos[t.unit];
        }
        const bool next_first = k + 1 < N && (tiles[k + 1].info & kTileFirst);
        const bool stage_query = wg == 0 && k + 2 < N && (tiles[k + 2].info & kTileFirst);
        if (stage_query) load_query(tiles[k + 2].unit);
        int pos = t0 + row;
        if (a.pos_pool != nullptr) pos = t.page >= 0 ? a.pos_pool[(size_t)t.page * a.P + row] : 0;
        const bool valid = row < rows && (!a.causal || pos <= qlim);
        if (!mbar_wait(bar(BAR_D_FULL + slot), (k >> 1) & 1, abort_flag, st, 31)) { ok = false; break; }
        tc_fence_after();
        float part[2];
        // Halfway through the pass (score batches 0 and 1 read) the columns where the
        // previous tile's value MMA writes are dead: tell the MMA thread.
        half_scores(slot, seg, pos, part, [&](int jj) {
          if (jj != kNB / 2) return;
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(BAR_MID));
        });
        // the next tile's rotated query; the tile-max sync below publishes it
        if (contig && k + 1 < N) post_rotated_query(tiles[k + 1].lp * kTile, seg + next_first, slot ^ 1);
        if (stage_query) store_query(seg + next_first + 1);
        psc[(slot * 2 + (1 - hw)) * 128 + row] = part[1 - hw];
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(BAR_XCH + slot));
        if (!mbar_wait(bar(BAR_XCH + slot), (k >> 1) & 1, abort_flag, st, 36)) { ok = false; break; }
        const float sfull = part[hw] + psc[(slot * 2 + hw) * 128 + row];
        // tile max of this head across the 128 tokens
        const float sc = valid ? sfull : -INFINITY;
        float m = sc;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
        if (lane == 0) red[(k & 1) * 8 + wg * 4 + q4] = m;
        if (!ep_sync(33)) { ok = false; break; }
        const float* rr = red + (k & 1) * 8 + wg * 4;
        const float mt = fmaxf(fmaxf(rr[0], rr[1]), fmaxf(rr[2], rr[3]));
        const float m_new = fmaxf(m_run, mt);
        // 0 on a segment's first tile; 1 while every token so far is masked
        const float scale = m_new == -INFINITY ? 1.f : exp2f(m_run - m_new);
        // the weight's three terms, rows hw, hw + 2 and hw + 4 of the value MMA's 16
        const float pf = valid ? exp2f(sc - m_new) : 0.f;
        uint16_t term[kWeightTerms];
        split_weight<ACT>(pf, term);
        uint8_t* pbuf = sbase + L.p + slot * kPBytes;
#pragma unroll
        for (int i = 0; i < kWeightTerms; ++i)
          *reinterpret_cast<uint16_t*>(pbuf + p_offset(hw + 2 * i, row)) = term[i];
        l_part = fmaf(l_part, scale, pf);
        m_run = m_new;
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(BAR_P_FULL + slot));
        // the previous tile's value sums (written into this slot), then release the slot
        if (k >= 1) {
          if (!fold_at(k - 1)) { ok = false; break; }
          if (t.info & kTileFirst) finish(tiles[k - 1], m_prev, l_prev);
        }
        prev_scale = scale;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(BAR_D_EMPTY + slot));
      }
      if (ok && N > 0 && fold_at(N - 1)) finish(tiles[N - 1], m_run, l_part);
    }
  } else {
    // warps 0-3
    if constexpr (kInt4) setmaxnreg_dec<kRegsW0>();
    if (kInt4 && warp != 1) {
      // ============================================================ int4 value codes (warps 0, 2, 3)
      // Ring stage s of a tile (s = 2mb + th) = entries [128mb, +128) of tokens
      // [64th, +64) = 16-byte units 4mb .. 4mb+3 of those tokens' rows of codes: 256
      // (token, unit) items, dealt to the 96 threads round-robin (item i: token
      // 64th + i mod 64, unit 4mb + i / 64) and loaded straight into registers two
      // stages ahead of the conversion.  Unit j = i / 64 lands in the stage's 64-entry
      // block j / 2 (8 KB apart), its 32 entries written PAIRED: row r of the value
      // operand holds entry paired_row(r).
      const int vt = (warp == 0 ? 0 : warp == 2 ? 32 : 64) + lane;
      constexpr int kSPT = 2 * NRV;                      // ring stages per tile
      struct Slot {
        uint4 raw[3];
        uint16_t sc[3];
        int rows;        // rows the query sees of the stage's 64
      };
      // item j of this thread: offsets of its unit in a page (stage 0 of the tile: unit i / 64 of token
      // i mod 64) and in a ring stage, of its scale in the page's scales
      uint32_t from[3], to[3], sfrom[3];
#pragma unroll
      for (int j = 0; j < 3; ++j) {
        const uint32_t i = vt + 96 * j < 256 ? vt + 96 * j : vt + 96, t = i & 63, u = i >> 6;   // (96 threads, 2.67 items each)
        from[j] = t * 128 + ((u ^ (t & 7)) << 4);
        to[j] = (i >> 7) * (kZvBytes / 2) + t * 128 + (((4 * (u & 1)) ^ (t & 7)) << 4);
        sfrom[j] = t * (uint32_t)a.vs_row + 2 * u;
      }
      const int last = vt + 192 < 256 ? 3 : 2;           // items of this thread
      const uint8_t* codes = nullptr;
      const uint8_t* scales = nullptr;
      int rows = 0;
      // stage s of tile k (past the last: the last tile's again, as for the keys)
      auto issue = [&](int k, int s, Slot& sl) {
        if (s == 0 && k < N) {
          const size_t pg = (size_t)max(tiles[k].page, 0);
          codes = gm.zv[gi] + pg * gm.v_page;
          scales = gm.zvs[gi] + pg * gm.vs_page;
          rows = tile_rows(tiles[k].info);
        }
        const uint32_t mb = s >> 1, th = s & 1;
        const uint32_t srow = th * 64 * (uint32_t)a.vs_row + 8 * mb;
        sl.rows = rows - 64 * (int)th;
#pragma unroll
        for (int j = 0; j < 3; ++j) {
          sl.raw[j] = __ldg(reinterpret_cast<const uint4*>(codes + (from[j] ^ (64 * mb)) + th * 8192));
          sl.sc[j] = __ldg(reinterpret_cast<const unsigned short*>(scales + sfrom[j] + srow));
        }
      };
      int stage = 0;
      uint32_t phase = 0;
      Slot s0, s1;                                       // this stage and the next
      if (N > 0) {
        issue(0, 0, s0);
        issue(0, 1, s1);
      }
#pragma unroll 1
      for (int n = 0; n < N * kSPT; ++n) {
        if (!mbar_wait(bar(BAR_ZV_EMPTY + stage), phase ^ 1, abort_flag, st, 13)) break;
        const uint32_t dst = base + L.zv + stage * kZvBytes;
#pragma unroll
        for (int j = 0; j < 3; ++j) {
          if (j < last) {
            const uint32_t w[4] = {s0.raw[j].x, s0.raw[j].y, s0.raw[j].z, s0.raw[j].w};
            // rows past the sequence become zeros, whatever the page holds there: codes are finite
            const uint16_t sc = ((vt + 96 * j) & 63) < s0.rows ? s0.sc[j] : (uint16_t)0;
#pragma unroll
            for (int m = 0; m < 4; ++m) st_shared_v4((dst + to[j]) ^ (uint32_t)(16 * m), dequant8<ACT, true>(w[m], sc));
          }
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(BAR_ZV_FULL + stage));
        if (++stage == kNVS) { stage = 0; phase ^= 1; }
        s0 = s1;
        issue((n + 2) / kSPT, (n + 2) % kSPT, s1);
      }
    } else if (warp == 0) {
      // ============================================================ z_k producer (bulk copies)
      if (lane == 0) {
        int stage = 0;
        uint32_t phase = 0;
        // No bulk L2 prefetch of later pages here: with the bulk copies of the two
        // head-pair CTAs of a group in flight, a prefetch 3 or 6 pages ahead left the
        // copy latency unchanged and the call 2-3 % slower.
        long long issued = 0;
        for (int k = 0; k < N && !*abort_flag; ++k) {
          const int pg = max(tiles[k].page, 0);   // of a bad page (reported): any page's, the result is void
          // one (page, group) block is the shared-memory image of the tile: each
          // 128-byte column block (64 latent entries of all 128 tokens) is one copy
          const uint8_t* src = gm.zk[gi] + (size_t)pg * gm.k_page;
          for (int c = 0; c < nkc; ++c) {
            if (!mbar_wait(bar(BAR_ZK_EMPTY + stage), phase ^ 1, abort_flag, st, 10)) break;
            mbar_expect_tx(bar(BAR_ZK_FULL + stage), kZkBytes);
            bulk_load(base + L.zk + stage * kZkBytes, src + (size_t)c * kZkBytes, kZkBytes, bar(BAR_ZK_FULL + stage));
            ++issued;
            if (++stage == kNZK) { stage = 0; phase ^= 1; }
          }
        }
        drain_ring(bar(BAR_ZK_FULL), kNZK, issued, st, 10);
      }
    } else if (warp == 2) {
      // ============================================================ z_v producer (bulk copies)
      if (lane == 0) {
        int stage = 0;
        uint32_t phase = 0;
        long long issued = 0;
        for (int k = 0; k < N && !*abort_flag; ++k) {
          const uint32_t valid = (uint32_t)tile_rows(tiles[k].info) * 128;   // bytes of a column block
          const uint8_t* src = gm.zv[gi] + (size_t)max(tiles[k].page, 0) * gm.v_page;
          // one 16 KB copy per 128-byte column block of the page (64 latent entries of all
          // 128 tokens); the two stages of the ring are the two 64-entry halves of one
          // value-MMA operand (whole blocks copied faster than token halves of 8 KB)
          for (int cb = 0; cb < 2 * NRV; ++cb) {
            if (!mbar_wait(bar(BAR_ZV_EMPTY + stage), phase ^ 1, abort_flag, st, 11)) break;
            mbar_expect_tx(bar(BAR_ZV_FULL + stage), kZvBytes);
            const uint32_t dst = base + L.zv + stage * kZvBytes;
            if (valid > 0) bulk_load(dst, src + (size_t)cb * a.P * 128, valid, bar(BAR_ZV_FULL + stage));
            if (valid < kZvBytes) bulk_load(dst + valid, g_zero_rows, kZvBytes - valid, bar(BAR_ZV_FULL + stage));
            ++issued;
            if (++stage == kNVS) { stage = 0; phase ^= 1; }
          }
        }
        drain_ring(bar(BAR_ZV_FULL), kNVS, issued, st, 11);
      }
    } else if (warp == 1) {
      // ============================================================ MMA issuer
      // The whole warp goes through the loop, one lane issues: what the loop computes is then known to
      // be the same on every lane and stays in the registers the MMAs take their operands from.
      {
        const bool leader = elect_one();
        auto ready = [&](uint32_t b, uint32_t parity) { return __all_sync(0xffffffffu, mbar_test_wait(b, parity)) != 0; };
        auto gave_up = [&]() { return __any_sync(0xffffffffu, *abort_flag != 0) != 0; };
        constexpr int kBf = ACT == PALU_BF16 ? 1 : 0;
        const uint32_t idesc_d = idesc_f16(kBf, 0, 1, 256, 128);    // z_k K-major, B_k MN-major
        const uint32_t idesc_pv = idesc_f16(kBf, 1, 0, 16, 128);    // z_vᵀ MN-major, Pᵀ K-major
        // operand descriptors at the first stage, chunk or buffer: the others lie a multiple of 16 bytes on
        const uint64_t zk0 = sdesc(base + L.zk, 16, kZkSbo, kZkSwz);
        const uint64_t b0 = sdesc(base + L.b, (uint32_t)r_k * 128, 1024, kSw128);   // 64-column blocks of B
        const uint64_t zv0 = sdesc(base + L.zv, kInt4 ? kZvBytes / 2 : kZvBytes, 1024, kSw128);
        const uint64_t p0 = sdesc(base + L.p, 16, 1024, kSw128);
        int zs = 0;
        uint32_t zph = 0, vph = 0;
        // timeout-path test hook: first wait on a phase nothing completes before the teardown commit
        bool ok = a.stall_test == 0 || mbar_wait(bar(BAR_TEARDOWN), 0, abort_flag, st, 26);
        ok = ok && mbar_wait(bar(BAR_B), 0, abort_flag, st, 20);
        ok = __all_sync(0xffffffffu, ok);
        int pv_next = 0;       // next tile whose value MMA is not issued yet
        int pv_s = 0;          // next operand of that value MMA: block mb = pv_s / 2 (int4: token half pv_s % 2)
        int vs = 0;            // int4: z_v ring stage of that operand

        // The value MMA of tile j, aᵀ[128 entries × 16] per block mb = z_vᵀ · Pᵀ, goes into
        // columns [32·mb, +16) of the TMEM slot of tile j + 1: columns whose keys that
        // tile's epilogue has read by the middle of its score pass (BAR_MID), so the value
        // round trip never holds a slot back from the next key MMA.  The last tile's value
        // MMA goes into the other slot once it is free.  Its gate (besides P and z_v):
        auto pv_gate = [&](int j) -> bool {
          if (j + 1 < N) return ready(bar(BAR_MID), (uint32_t)((j + 1) & 1));
          const int u = j + 1;
          return ready(bar(BAR_D_EMPTY + (u & 1)), (uint32_t)(((u >> 1) & 1) ^ 1));
        };
        // The next stage of the pending value MMA can go?  (Phases cannot alias: the epilogue
        // cannot pass tile j + 1 before the value sums of tile j are folded.)  int4: one ring
        // stage per operand (mb, th); 16-bit latents: the two stages of the ring hold the two
        // 64-entry halves of operand mb over all 128 tokens.
        auto pv_ready = [&]() -> bool {
          if constexpr (kInt4) {
            if (!ready(bar(BAR_ZV_FULL + vs), vph)) return false;
          } else {
            if (!(ready(bar(BAR_ZV_FULL + 0), vph) && ready(bar(BAR_ZV_FULL + 1), vph)))
              return false;
          }
          return pv_s > 0 || (ready(bar(BAR_P_FULL + (pv_next & 1)), (uint32_t)((pv_next >> 1) & 1)) &&
                              pv_gate(pv_next));
        };
        // One value-MMA operand into block mb of the value sums.  int4: stage (mb, th) =
        // latent entries [128mb, +128) (two 64-entry blocks 8 KB apart) × tokens [64th, +64),
        // against the matching half of Pᵀ.  16-bit latents: the two ring stages (64 entries
        // of all 128 tokens each) against all of Pᵀ.
        auto issue_pv_block = [&]() {
          const int j = pv_next;
          tc_fence_after();
          const uint64_t p = desc_at(p0, (uint32_t)(j & 1) * kPBytes);
          if constexpr (kInt4) {
            const int mb = pv_s >> 1, th = pv_s & 1;
            const uint32_t a_tmem = tmem + (uint32_t)((j + 1) & 1) * 256 + (uint32_t)mb * 32;
            const uint64_t z = desc_at(zv0, (uint32_t)vs * kZvBytes), ph = desc_at(p, th * 2048);
            if (leader) {
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)    // rows = latent entries, K = 16 tokens of the half
                umma_f16(a_tmem, desc_at(z, kk * 16 * 128), desc_at(ph, kk * 32), idesc_pv, (th | kk) != 0);
              umma_commit(bar(BAR_ZV_EMPTY + vs));
            }
            if (++vs == kNVS) { vs = 0; vph ^= 1; }
            ++pv_s;
          } else {
            static_assert(kInt4 || zv_stages(false) == 2, "one value MMA operand = the two ring stages");
            const uint32_t a_tmem = tmem + (uint32_t)((j + 1) & 1) * 256 + (uint32_t)(pv_s >> 1) * 32;
            if (leader) {
#pragma unroll
              for (int kk = 0; kk < kTile / 16; ++kk)    // rows = latent entries (two 64-entry blocks, one per stage), K = tokens
                umma_f16(a_tmem, desc_at(zv0, kk * 16 * 128), desc_at(p, (kk >> 2) * 2048 + (kk & 3) * 32), idesc_pv,
                         kk != 0);
              umma_commit(bar(BAR_ZV_EMPTY + 0));
              umma_commit(bar(BAR_ZV_EMPTY + 1));
            }
            vph ^= 1;
            pv_s += 2;
          }
          if (pv_s == 2 * NRV) {
            if (leader) umma_commit(bar(BAR_AT_FULL));
            ++pv_next;
            pv_s = 0;
          }
        };
        auto pv_step = [&]() -> bool {      // one step of the value MMAs, if one can be taken
          if (pv_next >= N || !pv_ready()) return false;
          issue_pv_block();
          return true;
        };
        // Wait for a barrier phase; meanwhile issue every value-MMA block whose operands
        // and gate are in (the epilogue's slot releases depend on them).  Bounded.
        auto poll_wait = [&](uint32_t b, uint32_t parity, int where) -> bool {
          const long long t0 = clock64();
          while (true) {
            if (ready(b, parity)) return true;
            if (pv_step()) continue;
            if (gave_up()) return false;
            __nanosleep(64);   // leave the issue slots of this SM partition to the epilogue warps
            if (__any_sync(0xffffffffu, clock64() - t0 > wait_limit(abort_flag))) {
              if (leader) report(st, PALU_ERR_DEVICE_TIMEOUT, where);
              *abort_flag = 1;
              return false;
            }
          }
        };

        for (int k = 0; k < N && ok; ++k) {
          const int slot = k & 1;
          if (!poll_wait(bar(BAR_D_EMPTY + slot), ((k >> 1) & 1) ^ 1, 23)) { ok = false; break; }
          tc_fence_after();
          const uint32_t d_tmem = tmem + (uint32_t)slot * 256;
          for (int c = 0; c < nkc; ++c) {
            if (!poll_wait(bar(BAR_ZK_FULL + zs), zph, 24)) { ok = false; break; }
            tc_fence_after();
            const uint64_t z = desc_at(zk0, (uint32_t)zs * kZkBytes), b = desc_at(b0, (uint32_t)c * kChunk * 128);
            if (leader) {
#pragma unroll
              for (int kk = 0; kk < kChunk / 16; ++kk)
                umma_f16(d_tmem, desc_at(z, kk * 32), desc_at(b, kk * 16 * 128), idesc_d, (c | kk) != 0);
              umma_commit(bar(BAR_ZK_EMPTY + zs));
            }
            if (++zs == kNZK) { zs = 0; zph ^= 1; }
          }
          if (!ok) break;
          if (leader) umma_commit(bar(BAR_D_FULL + slot));
        }
        // the value MMAs still pending (the last tiles'), each once its operands are in
        if (ok) {
          const long long t0 = clock64();
          while (pv_next < N) {
            if (pv_step()) continue;
            if (gave_up()) break;
            __nanosleep(64);
            if (__any_sync(0xffffffffu, clock64() - t0 > wait_limit(abort_flag))) {
              if (leader) report(st, PALU_ERR_DEVICE_TIMEOUT, 21);
              *abort_flag = 1;
              break;
            }
          }
        }
        // drain, also after an abort: every MMA issued above has completed before
        // TMEM is released, and the B_k load has landed before the CTA exits
        if (leader) umma_commit(bar(BAR_TEARDOWN));
        __syncwarp();
        mbar_drain(bar(BAR_TEARDOWN), 0, st, 25);
        mbar_drain(bar(BAR_B), 0, st, 20);
      }
    }
  }

  // ---------------------------------------------------------------- teardown
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}


template <int ACT, int NRV, int LAT>
cudaError_t launch_pages_t(const DecodeArgs& a, cudaStream_t st) {
  const CUtensorMapDataType dt = ACT == PALU_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  CUtensorMap tm_bk;
  if (a.bk_box <= 0 || a.bk_box > 256 || a.bk_box % 64 != 0 || a.batch > kWalkUnits) return cudaErrorInvalidValue;
  if constexpr (LAT == PALU_INT4) {
    if (a.bk_rows % 8 != 0 || !make_map_bk_paired(&tm_bk, a.Bk, dt, a.W, (uint64_t)a.bk_rows, a.bk_box))
      return cudaErrorInvalidValue;
  } else if (!make_map_2d(&tm_bk, a.Bk, dt, 2, a.W, (uint64_t)a.bk_rows, (uint64_t)a.W * 2, 64, a.bk_box,
                          CU_TENSOR_MAP_SWIZZLE_128B)) {
    return cudaErrorInvalidValue;
  }
  const size_t smem = pages_smem(a.r_k, LAT == PALU_INT4).total;
  auto kern =
      a.pos_pool == nullptr ? decode_pages_kernel<ACT, NRV, LAT, true> : decode_pages_kernel<ACT, NRV, LAT, false>;
  cudaError_t e = allow_shared(kern, smem);
  if (e != cudaSuccess) return e;
  if constexpr (LAT == PALU_INT4) {
    // the setmaxnreg split needs a launch at kRegsLaunch registers a thread (see decode_tc_kernel.cuh)
    cudaFuncAttributes fa;
    e = cudaFuncGetAttributes(&fa, kern);
    if (e != cudaSuccess) return e;
    if (fa.numRegs != (int)kRegsLaunch) return cudaErrorInvalidConfiguration;
  }
  kern<<<dim3(a.walk_ctas, a.gm.n * (a.gs / 2)), threads_of(LAT == PALU_INT4), smem, st>>>(tm_bk, a);
  count_launch();
  return cudaGetLastError();
}

}  // namespace
}  // namespace palu
