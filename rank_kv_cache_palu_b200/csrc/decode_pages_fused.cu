// Sparse decode step without rotary embedding (palu_decode_attn_pages, rope_base 0):
// the fused kernel over page lists (sm_100a: tcgen05 + TMEM).
//
// Method: "PALU 论文低秩投影分解" §低秩投影分解 and §把它放进一次真实推理流程里看,
// Decode 阶段 (attention fused with the up-projection): scores z_k · (B_k,h q_h) come
// straight from the cached latents, values stay in latent space, as in
// decode_fused.cu.  What differs here:
//   - a CTA walks an equal share of all lists of its group (pages_walk.cuh) with its
//     copies running on from list to list, where CTAs of their own for each list spent
//     a third of the time starting up;
//   - the folded queries change with the segment: the producer brings each segment's
//     (a 128-byte-swizzled image, fold_query.cuh) into one of three buffers;
//   - the softmax weights reach the value MMA as sums of three 16-bit numbers
//     (split_weight), rows p, 4 + p and 8 + p of its 16.
// Bound by the latents' bytes from HBM: 14 queries x 64 pages in each of 8 groups (r 256/128,
// f16, 0.71 GB) 128 us with the fold and the merge, 0.84 of the measured copy bandwidth; this
// kernel alone 114 us, 0.95.
#include <cuda.h>
#include <math.h>

#include "fold_query.cuh"
#include "pages_walk.cuh"
#include "palu_tc.h"
#include "tc_ptx.cuh"

namespace palu {
namespace {

using namespace tc;

constexpr int kTile = 128;          // tokens per tile = page size
constexpr int kChunk = 64;          // K chunk (latent entries) = one 128-byte column block
constexpr int kThreads = 192;       // producer, MMA, four epilogue warps
constexpr int kNZK = 6;             // z_k ring stages
constexpr int kNZV = 4;             // z_v ring stages (pairs of column blocks)
constexpr int kNQ = 3;              // folded-query buffers
constexpr int kStageBytes = kTile * kChunk * 2;   // 16 KB: one column block of a page
constexpr int kN = 16;              // score MMA columns: the terms of q̃, heads in rows 0-3, 4-7, 8-11, padding
constexpr int kQRows = kFoldTerms * kMaxG;
static_assert(kQRows <= kN, "a row for each term of each head's query");
constexpr int kNP = 16;             // value MMA columns: the weights' terms, heads in rows 0-3, 4-7, 8-11, padding
static_assert(kWeightTerms * kMaxG <= kNP, "a row for each term of each head's weights");
constexpr int kPBytes = kNP * kTile * 2;
constexpr int kTmemCols = 128;      // 2 score slots × kN, 2 value buffers × r_v / 128 × kNP
constexpr int kAt = 2 * kN;         // first value column

struct FusedSmem {
  uint32_t zk, zv, p, red, tiles, bars, tmem_slot, abort, qt, total;
};

enum {
  F_ZK_FULL = 0,
  F_ZK_EMPTY = F_ZK_FULL + kNZK,
  F_ZV_FULL = F_ZK_EMPTY + kNZK,
  F_ZV_EMPTY = F_ZV_FULL + kNZV,
  F_QT_FULL = F_ZV_EMPTY + kNZV,
  F_QT_EMPTY = F_QT_FULL + kNQ,
  F_D_FULL = F_QT_EMPTY + kNQ,       // 2
  F_D_EMPTY = F_D_FULL + 2,          // 2
  F_P_FULL = F_D_EMPTY + 2,          // 2
  F_AT_FULL = F_P_FULL + 2,          // 2
  F_AT_EMPTY = F_AT_FULL + 2,        // 2
  F_EPI = F_AT_EMPTY + 2,            // epilogue warps meet (bounded)
  F_TEARDOWN = F_EPI + 1,
  F_COUNT
};
static_assert(F_COUNT <= 48, "barrier space");

__host__ __device__ inline FusedSmem fused_smem(int r_k) {
  FusedSmem s{};
  uint32_t o = 0;
  s.zk = o;   o += kNZK * kStageBytes;
  s.zv = o;   o += kNZV * kStageBytes;
  s.p = o;    o += 2 * kPBytes;
  s.red = o;  o += 2 * 4 * kMaxG * 4;                    // [tile parity][warp][head] maxima
  s.tiles = o; o += kWalkTiles * sizeof(Tile);
  s.bars = o; o += 48 * 8;
  s.tmem_slot = o; o += 16;
  s.abort = o;     o += 16;
  o = (o + 1023u) & ~1023u;                             // 128-byte-swizzle atoms: 1024-byte aligned
  s.qt = o;   o += kNQ * (uint32_t)(r_k / kChunk) * kN * 128;   // [buffer][K chunk][16 rows][128 B]
  s.total = o;
  return s;
}

// P tile, K-major with the 128-byte swizzle: row n, token k; tokens 0-63 and
// 64-127 sit in two atoms of kNP rows.
__device__ __forceinline__ uint32_t p_offset(int n, int k) {
  const int region = k >> 6, kin = k & 63;
  return (uint32_t)(region * kNP * 128 + n * 128 + (((kin >> 3) ^ (n & 7)) << 4) + (kin & 7) * 2);
}

template <int ACT, int NRV>
__global__ void __launch_bounds__(kThreads, 1)
    decode_pages_fused_kernel(const __grid_constant__ DecodeArgs a, const void* qt) {
  extern __shared__ __align__(1024) uint8_t sbase[];
  const uint32_t base = smem_u32(sbase);
  // blockIdx.y: entry gi of the group map (model group gm.g[gi]); its key rank sets the layout
  const int gi = blockIdx.y;
  const GroupMap& gm = a.gm;
  const int r_k = gm.rk[gi];
  const FusedSmem L = fused_smem(r_k);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  DevStatus* st = reinterpret_cast<DevStatus*>(a.status);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sbase + L.abort);
  auto bar = [&](int i) { return base + L.bars + 8u * i; };
  const Tile* tiles = reinterpret_cast<const Tile*>(sbase + L.tiles);
  const int gs = a.gs;
  const int nkc = r_k / kChunk;
  const uint32_t qt_bytes = (uint32_t)nkc * kN * 128;    // of one buffer

  start_next();      // the merge; its CTAs find room as this launch's leave
  if (threadIdx.x == 0) {
    abort_init(abort_flag, a.wait_cycles);
    for (int i = 0; i < kNZK; ++i) {
      mbar_init(bar(F_ZK_FULL + i), 1);
      mbar_init(bar(F_ZK_EMPTY + i), 1);
    }
    for (int i = 0; i < kNZV; ++i) {
      mbar_init(bar(F_ZV_FULL + i), 1);
      mbar_init(bar(F_ZV_EMPTY + i), 1);
    }
    for (int i = 0; i < kNQ; ++i) {
      mbar_init(bar(F_QT_FULL + i), 1);
      mbar_init(bar(F_QT_EMPTY + i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(F_D_FULL + i), 1);
      mbar_init(bar(F_D_EMPTY + i), 4);
      mbar_init(bar(F_P_FULL + i), 4);
      mbar_init(bar(F_AT_FULL + i), 1);
      mbar_init(bar(F_AT_EMPTY + i), 4);
    }
    mbar_init(bar(F_EPI), 4);
    mbar_init(bar(F_TEARDOWN), 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(base + L.tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  // padding rows of P and of the folded queries stay zero
  for (int i = threadIdx.x; i < 2 * kPBytes / 4; i += kThreads) reinterpret_cast<uint32_t*>(sbase + L.p)[i] = 0u;
  for (int i = threadIdx.x; i < (int)(kNQ * qt_bytes / 4); i += kThreads)
    reinterpret_cast<uint32_t*>(sbase + L.qt)[i] = 0u;
  // this CTA's tiles; the prefix sums borrow the z_k ring, which nothing fills before the barrier below
  const int N = walk_tiles(a, gm.g[gi], gi, true, reinterpret_cast<Tile*>(sbase + L.tiles),
                           reinterpret_cast<int*>(sbase + L.zk), st);
  fence_proxy_async();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(sbase + L.tmem_slot);

  if (warp == 0) {
    // ============================================================ producer (bulk copies)
    if (lane == 0) {
      int zs = 0, vs = 0, seg = -1;
      uint32_t zph = 0, vph = 0;
      long long zk_issued = 0, zv_issued = 0, q_issued = 0;
      // z_v of a tile is needed only after its scores: stream it one tile behind
      // z_k, so the two rings fill in the order the MMAs consume them
      auto push_zv = [&](int k) -> bool {
        const uint32_t valid = (uint32_t)tile_rows(tiles[k].info) * 128;   // bytes of a column block
        const uint8_t* src = gm.zv[gi] + (size_t)max(tiles[k].page, 0) * gm.v_page;
        for (int cb = 0; cb < 2 * NRV; ++cb) {
          if (!mbar_wait(bar(F_ZV_EMPTY + vs), vph ^ 1, abort_flag, st, 11)) return false;
          mbar_expect_tx(bar(F_ZV_FULL + vs), kStageBytes);
          const uint32_t dst = base + L.zv + vs * kStageBytes;
          if (valid > 0) bulk_load(dst, src + (size_t)cb * a.P * 128, valid, bar(F_ZV_FULL + vs));
          if (valid < kStageBytes) bulk_load(dst + valid, g_zero_rows, kStageBytes - valid, bar(F_ZV_FULL + vs));
          ++zv_issued;
          if (++vs == kNZV) { vs = 0; vph ^= 1; }
        }
        return true;
      };
      // the folded query of the segment that tile k begins: the first kQRows of each chunk's 16 rows
      auto push_q = [&](int k) -> bool {
        ++seg;
        const int qb = seg % kNQ;
        if (!mbar_wait(bar(F_QT_EMPTY + qb), ((seg / kNQ) & 1) ^ 1, abort_flag, st, 12)) return false;
        mbar_expect_tx(bar(F_QT_FULL + qb), (uint32_t)nkc * kQRows * 128);
        const uint8_t* src = static_cast<const uint8_t*>(qt) + ((size_t)tiles[k].unit * gm.n + gi) * kQRows * a.r_k * 2;
        for (int c = 0; c < nkc; ++c)
          bulk_load(base + L.qt + qb * qt_bytes + c * kN * 128, src + (size_t)c * kQRows * 128, kQRows * 128,
                    bar(F_QT_FULL + qb));
        ++q_issued;
        return true;
      };
      // The first tile's latents go out ahead of its query, which waits for the fold: as many chunks as
      // the ring holds, for a further one waits for an MMA, and the MMAs wait for the query.
      auto first_query = [&]() -> bool {
        await_previous();
        return push_q(0);
      };
      bool ok = true;
      for (int k = 0; k < N && ok && !*abort_flag; ++k) {
        if (k > 0 && (tiles[k].info & kTileFirst) && !push_q(k)) break;
        const uint8_t* src = gm.zk[gi] + (size_t)max(tiles[k].page, 0) * gm.k_page;
        for (int c = 0; c < nkc; ++c) {
          if (k == 0 && c == kNZK && !first_query()) { ok = false; break; }
          if (!mbar_wait(bar(F_ZK_EMPTY + zs), zph ^ 1, abort_flag, st, 10)) { ok = false; break; }
          mbar_expect_tx(bar(F_ZK_FULL + zs), kStageBytes);
          bulk_load(base + L.zk + zs * kStageBytes, src + (size_t)c * kStageBytes, kStageBytes, bar(F_ZK_FULL + zs));
          ++zk_issued;
          if (++zs == kNZK) { zs = 0; zph ^= 1; }
        }
        if (k == 0 && nkc <= kNZK) ok = ok && first_query();
        if (ok && k >= 1) ok = push_zv(k - 1);
      }
      if (ok && N >= 1 && !*abort_flag) push_zv(N - 1);
      await_previous();   // with no tile too: no launch of the step ends before the one it follows
      // after an abort, copies already issued still land in shared memory: wait for them
      drain_ring(bar(F_ZK_FULL), kNZK, zk_issued, st, 10);
      drain_ring(bar(F_ZV_FULL), kNZV, zv_issued, st, 11);
      drain_ring(bar(F_QT_FULL), kNQ, q_issued, st, 12);
    }
  } else if (warp == 1) {
    // ============================================================ MMA issuer
    // The whole warp goes through the loop, one lane issues: what the loop computes is then known to
    // be the same on every lane and stays in the registers the MMAs take their operands from.
    const bool leader = elect_one();
    constexpr int kBf = ACT == PALU_BF16 ? 1 : 0;
    const uint32_t idesc_s = idesc_f16(kBf, 0, 0, kN, 128);    // z_k K-major, q̃ K-major
    const uint32_t idesc_pv = idesc_f16(kBf, 1, 0, kNP, 128);  // z_vᵀ MN-major, Pᵀ K-major
    // operand descriptors at the first stage or buffer: the others lie a multiple of 16 bytes on
    const uint64_t zk0 = sdesc(base + L.zk, 16, 1024, kSw128), q0 = sdesc(base + L.qt, 16, 1024, kSw128);
    const uint64_t zv0 = sdesc(base + L.zv, kStageBytes, 1024, kSw128), p0 = sdesc(base + L.p, 16, 1024, kSw128);
    auto wait = [&](int i, uint32_t parity, int where) {
      return __all_sync(0xffffffffu, mbar_wait(bar(i), parity, abort_flag, st, where)) != 0;
    };
    int zs = 0, vs = 0, seg = -1;
    uint32_t zph = 0, vph = 0;
    // timeout-path test hook: first wait on a phase nothing completes before the teardown commit
    bool ok = a.stall_test == 0 || wait(F_TEARDOWN, 0, 27);
    auto issue_pv = [&](int j) -> bool {
      const int vb = j & 1;
      const uint32_t a_tmem = tmem + kAt + (uint32_t)vb * NRV * kNP;
      const uint64_t p = desc_at(p0, (uint32_t)vb * kPBytes);
      if (!wait(F_P_FULL + vb, (j >> 1) & 1, 21)) return false;
      if (!wait(F_AT_EMPTY + vb, ((j >> 1) & 1) ^ 1, 22)) return false;
      for (int mb = 0; mb < NRV; ++mb) {
        for (int cb = 0; cb < 2; ++cb)
          if (!wait(F_ZV_FULL + vs + cb, vph, 23)) return false;
        tc_fence_after();
        const uint64_t z = desc_at(zv0, (uint32_t)vs * kStageBytes);
        if (leader) {
#pragma unroll
          for (int kk = 0; kk < kTile / 16; ++kk)
            umma_f16(a_tmem + mb * kNP, desc_at(z, kk * 16 * 128), desc_at(p, (kk >> 2) * kNP * 128 + (kk & 3) * 32),
                     idesc_pv, kk != 0);
          umma_commit(bar(F_ZV_EMPTY + vs));
          umma_commit(bar(F_ZV_EMPTY + vs + 1));
        }
        vs += 2;
        if (vs == kNZV) { vs = 0; vph ^= 1; }
      }
      if (leader) umma_commit(bar(F_AT_FULL + vb));
      return true;
    };
    for (int k = 0; k < N && ok; ++k) {
      const int slot = k & 1;
      const int info = __shfl_sync(0xffffffffu, tiles[k].info, 0);
      if (info & kTileFirst) {
        ++seg;
        if (!wait(F_QT_FULL + seg % kNQ, (seg / kNQ) & 1, 28)) { ok = false; break; }
      }
      if (!wait(F_D_EMPTY + slot, ((k >> 1) & 1) ^ 1, 24)) { ok = false; break; }
      tc_fence_after();
      const uint32_t d_tmem = tmem + (uint32_t)slot * kN;
      const uint64_t q = desc_at(q0, (uint32_t)(seg % kNQ) * qt_bytes);
      for (int c = 0; c < nkc; ++c) {
        if (!wait(F_ZK_FULL + zs, zph, 25)) { ok = false; break; }
        tc_fence_after();
        const uint64_t z = desc_at(zk0, (uint32_t)zs * kStageBytes), qc = desc_at(q, (uint32_t)c * kN * 128);
        if (leader) {
#pragma unroll
          for (int kk = 0; kk < kChunk / 16; ++kk)
            umma_f16(d_tmem, desc_at(z, kk * 32), desc_at(qc, kk * 32), idesc_s, (c | kk) != 0);
          umma_commit(bar(F_ZK_EMPTY + zs));
        }
        if (++zs == kNZK) { zs = 0; zph ^= 1; }
      }
      if (!ok) break;
      if (leader) {
        umma_commit(bar(F_D_FULL + slot));
        if (info & kTileLast) umma_commit(bar(F_QT_EMPTY + seg % kNQ));
      }
      // the previous tile's value MMA, once its P is written
      if (k >= 1 && !issue_pv(k - 1)) { ok = false; break; }
    }
    if (ok && N >= 1) issue_pv(N - 1);
    // drain, also after an abort: every MMA issued above completes before TMEM is released
    if (leader) umma_commit(bar(F_TEARDOWN));
    __syncwarp();
    mbar_drain(bar(F_TEARDOWN), 0, st, 26);
  } else {
    // ============================================================ epilogue (warps 2-5)
    // One thread per token row (scores) and per latent row (value sums).
    const int q4 = warp & 3;                 // TMEM lane quarter this warp may access
    const int row = q4 * 32 + lane;          // token row of the tile / latent row of aᵀ
    const uint32_t lane_addr = (uint32_t)(q4 * 32) << 16;
    float* red = reinterpret_cast<float*>(sbase + L.red);
    uint32_t epi_phase = 0;
    auto ep_sync = [&](int where) -> bool {
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(F_EPI));
      const bool r = mbar_wait(bar(F_EPI), epi_phase, abort_flag, st, where);
      epi_phase ^= 1;
      return r;
    };
    float m_run[kMaxG], l_part[kMaxG], prev_scale[kMaxG];
    float acc[NRV][kMaxG];
    auto restart = [&]() {
#pragma unroll
      for (int p = 0; p < kMaxG; ++p) {
        m_run[p] = -INFINITY;
        l_part[p] = 0.f;
        prev_scale[p] = 0.f;
#pragma unroll
        for (int mb = 0; mb < NRV; ++mb) acc[mb][p] = 0.f;
      }
    };
    restart();
    auto fold_at = [&](int j) -> bool {
      const int vb = j & 1;
      if (!mbar_wait(bar(F_AT_FULL + vb), (j >> 1) & 1, abort_flag, st, 30)) return false;
      tc_fence_after();
#pragma unroll
      for (int mb = 0; mb < NRV; ++mb) {
        float v[kNP];                        // sums of the weights' first terms, of the second, of the third
        tmem_ld16(tmem + lane_addr + kAt + (uint32_t)vb * NRV * kNP + mb * kNP, v);
        tmem_wait_ld();
#pragma unroll
        for (int p = 0; p < kMaxG; ++p)
          acc[mb][p] = fmaf(acc[mb][p], prev_scale[p], v[p] + (v[kMaxG + p] + v[2 * kMaxG + p]));
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(F_AT_EMPTY + vb));
      return true;
    };
    // The partials of the segment that tile t ends; the running sums start over.
    auto finish = [&](const Tile& t) {
      constexpr float kLn2 = 0.6931471805599453f;
#pragma unroll
      for (int p = 0; p < kMaxG; ++p) {
        float l = l_part[p];
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
        if (p >= gs || *abort_flag) continue;
        float* out = segment_part(a, t, gi * gs + p);
        if (row == 0) out[0] = m_run[p] * kLn2;
        if (lane == 0) out[1 + q4] = l;
#pragma unroll
        for (int mb = 0; mb < NRV; ++mb) out[kPartHead + mb * 128 + row] = acc[mb][p] * (1.f / kWeightScale<ACT>);
      }
      restart();
    };
    bool ok = true;
    int qlim = 0;
    for (int k = 0; k < N && ok; ++k) {
      const Tile t = tiles[k];
      const int slot = k & 1, rows = tile_rows(t.info);
      if (a.causal && (t.info & kTileFirst)) qlim = a.q_pos[t.unit];   // tokens after it are masked
      int pos = t.lp * kTile + row;
      if (a.causal && a.pos_pool != nullptr) pos = t.page >= 0 ? a.pos_pool[(size_t)t.page * a.P + row] : 0;
      if (!mbar_wait(bar(F_D_FULL + slot), (k >> 1) & 1, abort_flag, st, 31)) { ok = false; break; }
      tc_fence_after();
      float d[kN];
      tmem_ld16(tmem + lane_addr + slot * kN, d);
      tmem_wait_ld();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(F_D_EMPTY + slot));
      // the previous tile's latent sums are ready by now (its value MMA went in behind this
      // tile's scores); they may end a segment
      if (k >= 1) {
        if (!fold_at(k - 1)) { ok = false; break; }
        if (t.info & kTileFirst) finish(tiles[k - 1]);
      }
      const bool valid = row < rows && (!a.causal || pos <= qlim);
      float sc[kMaxG];
#pragma unroll
      for (int p = 0; p < kMaxG; ++p) {
        sc[p] = valid && p < gs ? d[p] + (d[kMaxG + p] + d[2 * kMaxG + p]) : -INFINITY;   // the terms of q̃
        float m = sc[p];
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
        if (lane == 0) red[(slot * 4 + q4) * kMaxG + p] = m;
      }
      if (!ep_sync(33)) { ok = false; break; }
      uint8_t* pbuf = sbase + L.p + slot * kPBytes;
#pragma unroll
      for (int p = 0; p < kMaxG; ++p) {
        if (p >= gs) continue;
        const float* rr = red + slot * 4 * kMaxG + p;
        const float mt = fmaxf(fmaxf(rr[0], rr[kMaxG]), fmaxf(rr[2 * kMaxG], rr[3 * kMaxG]));
        const float m_new = fmaxf(m_run[p], mt);
        const float scale = m_new == -INFINITY ? 1.f : exp2f(m_run[p] - m_new);   // 1 while all masked
        const float pf = sc[p] != -INFINITY ? exp2f(sc[p] - m_new) : 0.f;
        uint16_t term[kWeightTerms];
        split_weight<ACT>(pf, term);
#pragma unroll
        for (int i = 0; i < kWeightTerms; ++i)
          *reinterpret_cast<uint16_t*>(pbuf + p_offset(i * kMaxG + p, row)) = term[i];
        l_part[p] = fmaf(l_part[p], scale, pf);
        m_run[p] = m_new;
        prev_scale[p] = scale;
      }
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(F_P_FULL + slot));
    }
    if (ok && N > 0 && fold_at(N - 1)) finish(tiles[N - 1]);
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <int ACT, int NRV>
cudaError_t launch_t(const DecodeArgs& a, cudaStream_t st) {
  if (a.batch > kWalkUnits) return cudaErrorInvalidValue;
  fold_query_kernel<ACT, true>
      <<<dim3(a.gm.n, (a.r_k + 63) / 64, (a.batch + kFoldSeqs - 1) / kFoldSeqs), 256, 0, st>>>(a, 1, a.fused_q);
  count_launch();
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const size_t smem = fused_smem(a.r_k).total;
  auto kern = decode_pages_fused_kernel<ACT, NRV>;
  e = allow_shared(kern, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute at = dependent_launch();
  cudaLaunchConfig_t c{};
  c.gridDim = dim3(a.walk_ctas, a.gm.n);
  c.blockDim = dim3(kThreads);
  c.dynamicSmemBytes = smem;
  c.stream = st;
  c.attrs = &at;
  c.numAttrs = 1;
  count_launch();
  return cudaLaunchKernelEx(&c, kern, a, (const void*)a.fused_q);
}

}  // namespace

size_t pages_query_bytes(const palu_config* c, int units) {
  return (size_t)units * (c->num_heads / c->group_size) * kQRows * c->rank_k * 2;
}

cudaError_t launch_decode_pages_fused(const DecodeArgs& a, cudaStream_t st) {
  if (a.act == PALU_BF16) return a.r_v == 256 ? launch_t<PALU_BF16, 2>(a, st) : launch_t<PALU_BF16, 1>(a, st);
  return a.r_v == 256 ? launch_t<PALU_F16, 2>(a, st) : launch_t<PALU_F16, 1>(a, st);
}

}  // namespace palu
