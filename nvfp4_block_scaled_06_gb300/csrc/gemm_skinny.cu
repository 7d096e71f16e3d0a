// gemm_skinny.cu -- the W4A4 product for a few activation rows (decode,
// M <= 32) on tcgen05, with the operands swapped.
//
// Same product as k_gemm_fp4 (gemm.cu): Y[m, n] = g_x g_w * sum_k
// e2m1(x_mk) sx(m, k/16) e2m1(w_nk) sw(n, k/16), both operands K-major with one
// E4M3 scale per 16 elements ("vroomfondel/glm-5.2-reap-504B-v2-W4A4" card,
// "Kernel choice" and "What this variant changes": at decode the projection is
// a stream of the weights).  Here the weights are the MMA's 128-row A operand
// and the <= 32 activation rows its B operand (N = 32): the accumulator holds
// Y^T for 128 output features, and a stage carries 16 KB of weights and only
// 4 KB of activations (24 KB with both scale atoms), so nine stages -- 144 KB
// of weights -- are in flight per SM instead of the six (96 KB) of the
// 128 x 128 tile whose A side would be the padded activation rows.
//
// A persistent kernel, one CTA per SM (grouped: two), 384 threads:
//   warps 0, 10, 11  producers (one thread each): the stage's weight tile (128
//               rows x 256 codes) in two halves by TMA; the activation tile (32
//               rows x 256 codes) by TMA and the scale atoms by bulk copy.
//               (One thread for all of it was no slower with one CTA per SM.)
//   warp 1      MMA issue (one thread): kind::mxf4nvf4 scale_vec::4X, M=128,
//               N=32, K=64, four per stage.
//   warps 2..5  scales -> tensor memory for every stage.
//   warps 6..9  drain a unit's 128 x 32 accumulator (two of them, so that the
//               next unit's MMAs go on) and store Y (or the unit's fp32 split-K
//               partial) transposed: lane = feature n, one store per
//               activation row, coalesced across the warp.
// Work units are (128-feature tile, K range); K ranges are summed in order by
// the split-K pass.  Every wait is bounded.
//
// MX: the same kernel for MXFP4 operands (one E8M0 scale per 32 elements): a
// stage has two scale atoms per operand instead of four, and the MMA (kind::mxf4
// scale_vec::2X) of K step j takes half (j & 1) of atom j / 2.
//
// FUSE (MXFP4, up to eight bf16 rows with at most 768 of their blocks per CTA): no
// packing kernel in front (6144 x 16384, one row: 16.5 -> 14.3 us per call; eight
// rows are 1408 blocks there and took 17.6 us against 16.3 with the kernel).
// Warps 2..9 pack the CTA's K range of the rows before the first stage, into one
// 8-row group of the swizzled tile (1 KB) per 256-wide K tile; they stay for all
// of the CTA's units, and the stages carry weights only.  The MMA's rows 8..31
// read whatever follows: their results are not stored.
//
// GROUPED (MXFP4 experts at decode): a unit is a 128-feature tile of one
// expert's weights against 32 of its routed rows, taken from the m-tile table
// (four such row groups per 128-row tile, those without rows skipped), so the
// experts' weights, not the padding of their rows, fill the stages.  32 tokens'
// top 8 of 32 experts (27 with rows, N 6144, K 2048, 182 MB): 38 us = 4.8 TB/s,
// where the 128 x 256 tiles took 43.5 us; bound by whole units in rounds (1296
// of them on 304 CTAs).
#include "internal.h"
#include "mxfp4.cuh"
#include "ptx.cuh"

namespace nvfp4 {

namespace {

constexpr int kSkThreads = 384;
// Dense: nine stages, one CTA per SM (four and two CTAs: one to two units per
// CTA, o_proj 16.6 instead of 15.8 us).  Grouped: four, so that two CTAs fit an
// SM (and its tensor memory) and the units of one, about five, hide the other's
// starts and drains: 38 instead of 42.5 us.
constexpr int sk_stages(bool grouped) { return grouped ? 4 : 9; }
constexpr int kSkN = 32;                         // activation rows per MMA (B operand)
constexpr int kSkABytes = 128 * 128;             // 128 weight rows x 256 codes
constexpr int kSkBBytes = kSkN * 128;            // 32 activation rows x 256 codes
constexpr int kSkSfBytes = 4 * 512;              // one 128-row chunk, four 128x4 atoms
constexpr int kSkStageBytes = kSkABytes + kSkBBytes + 2 * kSkSfBytes;
constexpr int sk_smem_bytes(bool grouped) { return sk_stages(grouped) * kSkStageBytes + 512 + 1024; }
constexpr int kSkAccs = 2;                       // accumulators in flight
// TMEM: 2 x 32 accumulator columns, then per stage 16 columns of weight scales and
// 16 of activation scales (4 per K step each: lane i of every quarter holds
// line i of the atom, rows i, i+32, i+64, i+96 -- the MMA reads row r of an
// operand from lane r % 32, column r / 32 of its K step)
constexpr int kSkSfCols = 32;
constexpr int sk_tmem_cols(bool grouped) { return grouped ? 256 : 512; }
constexpr uint64_t kSkDrainNs = 200000000ull;
constexpr int kSkSfBase = kSkAccs * kSkN;         // first scale column
static_assert(kSkSfBase + sk_stages(false) * kSkSfCols <= sk_tmem_cols(false) &&
                  kSkSfBase + sk_stages(true) * kSkSfCols <= sk_tmem_cols(true),
              "TMEM budget");
static_assert(sk_smem_bytes(false) <= 232448 && 2 * (sk_smem_bytes(true) + 1024) <= 233472, "shared memory budget");

__device__ __forceinline__ void sk_abort(volatile int *abort_flag, int *status) {
  *abort_flag = 1;
  record_timeout(status);
}

}  // namespace

// p.M activation rows (<= 32), p.N features, a_* = activations, b_* = weights
// (as for k_gemm_fp4); tmX: activation codes, box 128 B x 32 rows; tmW: weight
// codes, box 128 B x 64 rows.
template <bool MX, bool GROUPED, bool FUSE>
__global__ void __launch_bounds__(kSkThreads, GROUPED ? 2 : 1)
    k_gemm_fp4_skinny(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW,
                      const GemmParams p) {
  constexpr int S = sk_stages(GROUPED);
  extern __shared__ uint8_t smem_raw[];
  uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~uintptr_t(1023));
  uint8_t *sW = base;
  uint8_t *sX = sW + S * kSkABytes;
  uint8_t *sSFW = sX + S * kSkBBytes;
  uint8_t *sSFX = sSFW + S * kSkSfBytes;
  uint64_t *bars = reinterpret_cast<uint64_t *>(sSFX + S * kSkSfBytes);
  uint64_t *full = bars, *empty = bars + S, *sfready = bars + 2 * S;
  uint64_t *acc_full = bars + 3 * S, *acc_empty = acc_full + kSkAccs, *drain = acc_empty + kSkAccs;
  uint64_t *never = drain + 1;             // test hook: a barrier nothing arrives at
  uint64_t *xready = drain + 2;            // FUSE: the rows are packed
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 3);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 3);     // the three producers
      mbar_init(&empty[s], 1);
      mbar_init(&sfready[s], 4);
    }
    for (int a = 0; a < kSkAccs; ++a) {
      mbar_init(&acc_full[a], 1);
      mbar_init(&acc_empty[a], 4);
    }
    mbar_init(drain, 1);
    mbar_init(never, 1);
    mbar_init(xready, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmX);
    tma_prefetch_desc(&tmW);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, sk_tmem_cols(GROUPED));
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  griddep_launch_dependents();
  // Inputs of this kernel come from the previous one in the stream (the
  // activation packing).  NVFP4: that kernel lets this grid start only after
  // every kernel before it has completed, so the producer issues the weight
  // tiles of its first stages before its wait.  MXFP4: the packing lets this
  // grid start at once, before what precedes it is done, so the producer only
  // asks L2 for its first unit's weights (a hint: a weight written later is
  // updated there), which then stream from HBM while the packing and the
  // previous call's last kernel run (o_proj, M = 1: 15.9 -> 15.8 us per call
  // back to back).  Grouped: the units come from the
  // previous kernels.  Every other thread waits here.
  const bool producer = warp == 0 || warp >= 10;
  if (!producer || GROUPED) griddep_wait();

  const int ksplit = p.ksplit > 1 ? p.ksplit : 1;
  // (128-feature tile, K range); grouped: (row group, m-tile, 128-feature tile),
  // the first row group of every m-tile before the second (which few have), so
  // that the units with rows spread over all CTAs
  const int group_units = GROUPED ? p.tiles_n * *p.gnum_mtiles : 0;
  const int num_units = GROUPED ? 4 * group_units : p.tiles_n * ksplit;
  struct Unit {
    int nt, w_row, x_row, out_row, rows, sub;   // rows: activation rows (0: nothing to do)
  };
  // The m-tile of unit u, fetched a unit ahead of its use (an L2 latency).
  const auto tile_of = [&](int u) {
    GroupTile g = {};
    if constexpr (GROUPED)
      if (u < num_units) g = p.gtiles[u % group_units / p.tiles_n];
    return g;
  };
  const auto unit_of = [&](int u, GroupTile g) {
    Unit t;
    if constexpr (!GROUPED) {
      t.nt = u / ksplit;
      t.w_row = t.nt * 128;
      t.x_row = t.out_row = t.sub = 0;
      t.rows = (int)p.M;
      return t;
    } else {
      t.sub = u / group_units;
      const int v = u - t.sub * group_units;
      t.nt = v % p.tiles_n;
      if (!NVFP4_GUARD(g.expert >= 0 && (int64_t)(g.expert + 1) * p.N <= p.b_sf_row_chunks * 128 && g.a_row0 >= 0 &&
                           g.a_row0 + 128 <= p.M && g.valid_rows >= 0 && g.valid_rows <= 128 && g.out_row0 >= 0 &&
                           g.out_row0 + g.valid_rows <= p.out_rows,
                       p.status))
        g.expert = g.a_row0 = g.valid_rows = g.out_row0 = 0;
      t.w_row = (int)(g.expert * p.N) + t.nt * 128;
      t.x_row = g.a_row0 + 32 * t.sub;
      t.out_row = g.out_row0 + 32 * t.sub;
      t.rows = min(32, g.valid_rows - 32 * t.sub);
      return t;
    }
  };
  const int kt_per = (p.num_kt + ksplit - 1) / ksplit;
  const int last_nk = p.nk64 - (p.num_kt - 1) * 4;   // K steps of the last 256-wide K tile
  constexpr int kAtoms = MX ? 2 : 4;                 // scale atoms of a full stage
  const auto sf_bytes = [&](int kt) {                // scale bytes of K tile kt (per 128 rows)
    const int nk = kt == p.num_kt - 1 ? last_nk : 4;
    return (uint32_t)((MX ? (nk + 1) / 2 : nk) * 512);
  };

  if (FUSE && warp >= 2 && warp < 10) {
    // ------------------------------------------------------- pack the rows --
    // (K ranges: one unit per CTA; one range: the same rows for every unit)
    if ((int)blockIdx.x < num_units) {
      const int kt0 = (blockIdx.x % ksplit) * kt_per, nblocks = (min(p.num_kt, kt0 + kt_per) - kt0) * 8;
      const int64_t nblk = p.K / 32;
      const uint32_t x_base = smem_u32(sX);
      constexpr int kPer = kFuseBlocks / 256;        // blocks per thread, every load before the first use
      uint32_t w[kPer][16];
#pragma unroll
      for (int h = 0; h < kPer; ++h) {
        const int i = threadIdx.x - 64 + 256 * h, r = i / nblocks, b = i - r * nblocks;
#pragma unroll
        for (int k = 0; k < 16; ++k) w[h][k] = 0u;
        if (r < p.M && (int64_t)kt0 * 8 + b < nblk)
          load32<false>(p.x_bf16 + r * p.x_ld + ((int64_t)kt0 * 8 + b) * 32, w[h]);
      }
#pragma unroll
      for (int h = 0; h < kPer; ++h) {
        const int i = threadIdx.x - 64 + 256 * h, r = i / nblocks, b = i - r * nblocks;
        if (r >= p.M) continue;
        uint32_t sb;
        const uint4 c = mx_encode32(w[h], sb);
        // 128-byte swizzle: 16-byte chunk c of row r sits at c ^ (r & 7)
        sts128(x_base + (b >> 3) * 1024 + r * 128 + (((b & 7) ^ r) << 4), c.x, c.y, c.z, c.w);
        sSFX[(b >> 3) * 64 + r * 8 + (b & 7)] = (uint8_t)sb;
      }
      fence_proxy_async_shared();      // the tiles are read by the MMA (async proxy)
    }
    asm volatile("bar.sync 1, 256;" ::: "memory");
    if (threadIdx.x == 64) mbar_arrive(xready);
  }
  if (producer) {
    // ----------------------------------------------------------- producers --
    // Three threads in three warps, one stream each: the weight tile's upper
    // and lower 64 rows, and the activation tile with both operands' scales.
    if (lane == 0) {
      const int role = warp == 0 ? 0 : warp - 9;
      const uint32_t w_base = smem_u32(sW) + (role == 1 ? kSkABytes / 2 : 0), x_base = smem_u32(sX);
      const uint32_t sfw_base = smem_u32(sSFW), sfx_base = smem_u32(sSFX);
      const uint32_t full_base = smem_u32(full), empty_base = smem_u32(empty);
      const int half_row = role == 1 ? 64 : 0;
      int stage = 0;
      uint32_t phase = 0, armed = 0, armed_par = 0;
      bool ok = true;
      // the first unit's weights, before the wait
      int pre = 0;
      if (!GROUPED && (int)blockIdx.x < num_units) {
        const int nt = blockIdx.x / ksplit;
        const int kt0 = (blockIdx.x % ksplit) * kt_per, kt1 = min(p.num_kt, kt0 + kt_per);
        const uint8_t *sfw_src = p.b_sf + 512 * ((int64_t)nt * p.b_sf_katoms + (int64_t)kt0 * kAtoms);
        if (MX) {
          for (int i = 0; i < kt1 - kt0; ++i) {
            if (role < 2)
              tma_prefetch_2d(&tmW, (kt0 + i) * 128, nt * 128 + half_row);
            else
              prefetch_l2_bulk(sfw_src + (int64_t)i * 512 * kAtoms, sf_bytes(kt0 + i));
          }
        } else {
          // the first stages, all free at entry
          pre = min(S, kt1 - kt0);
          for (int i = 0; i < pre; ++i) {
            const uint32_t fb = full_base + 8 * i;
            if (role < 2) {
              mbar_arrive_expect_tx_u(fb, kSkABytes / 2);
              tma_load_2d_u(w_base + i * kSkABytes, &tmW, fb, (kt0 + i) * 128, nt * 128 + half_row);
            } else {
              const uint32_t sfb = sf_bytes(kt0 + i);
              mbar_arrive_expect_tx_u(fb, kSkBBytes + 2 * sfb);
              bulk_load_u(sfw_base + i * kSkSfBytes, sfw_src + (int64_t)i * 512 * kAtoms, sfb, fb);
            }
          }
        }
      }
      griddep_wait();
      GroupTile ahead = tile_of(blockIdx.x);
      for (int u = blockIdx.x; ok && u < num_units; u += gridDim.x) {
        const Unit t = unit_of(u, ahead);
        ahead = tile_of(u + gridDim.x);
        if (t.rows <= 0) continue;
        const int kt0 = (u % ksplit) * kt_per, kt1 = min(p.num_kt, kt0 + kt_per);
        const uint8_t *sfw_src = p.b_sf + 512 * ((int64_t)(t.w_row >> 7) * p.b_sf_katoms + (int64_t)kt0 * kAtoms);
        // the rows' 128-row chunk
        const uint8_t *sfx_src = p.a_sf + 512 * ((int64_t)(t.x_row >> 7) * p.a_sf_katoms + (int64_t)kt0 * kAtoms);
        for (int kt = kt0; kt < kt1; ++kt) {
          const bool early = u == (int)blockIdx.x && kt - kt0 < pre;   // weights already in flight
          const bool got = early || (!*abort_flag && mbar_wait_u(empty_base + 8 * stage, phase ^ 1, p.timeout_ns));
          if (!got) {
            sk_abort(abort_flag, p.status);
            ok = false;
            break;
          }
          const uint32_t fb = full_base + 8 * stage;
          if (role < 2) {
            if (!early) {
              mbar_arrive_expect_tx_u(fb, kSkABytes / 2);
              tma_load_2d_u(w_base + stage * kSkABytes, &tmW, fb, kt * 128, t.w_row + half_row);
            }
          } else {
            const uint32_t sfb = sf_bytes(kt);
            if (!early) {
              mbar_arrive_expect_tx_u(fb, FUSE ? sfb : kSkBBytes + 2 * sfb);
              bulk_load_u(sfw_base + stage * kSkSfBytes, sfw_src, sfb, fb);
            }
            if constexpr (!FUSE) {
              tma_load_2d_u(x_base + stage * kSkBBytes, &tmX, fb, kt * 128, t.x_row);
              bulk_load_u(sfx_base + stage * kSkSfBytes, sfx_src, sfb, fb);
            }
            sfw_src += 512 * kAtoms;
            sfx_src += 512 * kAtoms;
          }
          armed |= 1u << stage;
          armed_par = (armed_par & ~(1u << stage)) | (phase << stage);
          if (++stage == S) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
      // every fill this thread started lands before the CTA may exit (after an
      // abort another producer may never complete a stage: one bounded wait)
      for (int s = 0; s < S; ++s)
        if ((armed & (1u << s)) && !mbar_wait(&full[s], (armed_par >> s) & 1, kSkDrainNs)) break;
    }
  } else if (warp == 1) {
    // ----------------------------------------------------------- MMA issue --
    if (lane == 0) {
      const uint32_t idesc = MX ? idesc_mxfp4(128, kSkN, 0) : idesc_nvfp4(128, kSkN);
      const uint32_t idesc_hi = idesc_mxfp4(128, kSkN, 2);   // MX: the upper half of an atom
      const uint64_t wdesc0 = sdesc_k_sw128(sW), xdesc0 = sdesc_k_sw128(sX);
      const uint32_t sfr_base = smem_u32(sfready), empty_base = smem_u32(empty);
      const uint32_t accf = smem_u32(acc_full), acce = smem_u32(acc_empty);
      int stage = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true;
      if (p.stall_probe && !mbar_wait(never, 0, p.timeout_ns)) {
        sk_abort(abort_flag, p.status);   // expected: the expiry path under test
        ok = false;
      }
      if (FUSE && ok && !mbar_wait(xready, 0, p.timeout_ns)) {
        sk_abort(abort_flag, p.status);
        ok = false;
      }
      GroupTile ahead = tile_of(blockIdx.x);
      for (int u = blockIdx.x; ok && u < num_units; u += gridDim.x) {
        const Unit t = unit_of(u, ahead);
        ahead = tile_of(u + gridDim.x);
        if (t.rows <= 0) continue;
        const int kt0 = (u % ksplit) * kt_per, kt1 = min(p.num_kt, kt0 + kt_per);
        if (*abort_flag || !mbar_wait_u(acce + 8 * acc, acc_phase ^ 1, p.timeout_ns)) {
          sk_abort(abort_flag, p.status);
          break;
        }
        tc_fence_after();
        uint32_t accumulate = 0;
        const uint32_t dcol = tmem + acc * kSkN;
        for (int kt = kt0; kt < kt1; ++kt) {
          // the stage's operands have landed and its scales are in tensor memory
          if (*abort_flag || !mbar_wait_u(sfr_base + 8 * stage, phase, p.timeout_ns)) {
            sk_abort(abort_flag, p.status);
            ok = false;
            break;
          }
          tc_fence_after();
          const int nk = kt == p.num_kt - 1 ? last_nk : 4;
          const uint64_t wdesc = wdesc0 + (uint64_t)((stage * kSkABytes) >> 4);
          const uint64_t xdesc = xdesc0 + (uint64_t)((FUSE ? (kt - kt0) * 1024 : stage * kSkBBytes) >> 4);
          const uint32_t sfw_col = tmem + kSkSfBase + stage * kSkSfCols, sfx_col = sfw_col + 16;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (j < nk) {
              if constexpr (MX)
                tc_mma_mxfp4(dcol, wdesc + 2 * j, xdesc + 2 * j, j & 1 ? idesc_hi : idesc, sfw_col + 4 * (j >> 1),
                             sfx_col + 4 * (j >> 1), accumulate);
              else
                tc_mma_nvfp4(dcol, wdesc + 2 * j, xdesc + 2 * j, idesc, sfw_col + 4 * j, sfx_col + 4 * j, accumulate);
              accumulate = 1;
            }
          }
          tc_commit_u(empty_base + 8 * stage);
          if (++stage == S) {
            stage = 0;
            phase ^= 1;
          }
        }
        if (!ok) break;
        tc_commit_u(accf + 8 * acc);
        if (++acc == kSkAccs) {
          acc = 0;
          acc_phase ^= 1;
        }
      }
      // all MMAs issued by this thread complete before TMEM is freed
      tc_commit(drain);
      mbar_wait(drain, 0, kSkDrainNs);
    }
  } else if (warp < 6) {
    // --------------------------------------------------- scales -> tensor memory --
    const int q = warp & 3;
    const uint32_t tq = tmem + ((uint32_t)(q * 32) << 16);
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    GroupTile ahead = tile_of(blockIdx.x);
    for (int u = blockIdx.x; ok && u < num_units; u += gridDim.x) {
      const Unit t = unit_of(u, ahead);
      ahead = tile_of(u + gridDim.x);
      if (t.rows <= 0) continue;
      const int kt0 = (u % ksplit) * kt_per, kt1 = min(p.num_kt, kt0 + kt_per);
      for (int kt = kt0; kt < kt1; ++kt) {
        if (!__all_sync(0xffffffffu, !*abort_flag && mbar_wait(&full[stage], phase, p.timeout_ns))) {
          if (lane == 0) sk_abort(abort_flag, p.status);
          ok = false;
          break;
        }
        const uint4 *fw = reinterpret_cast<const uint4 *>(sSFW + stage * kSkSfBytes) + lane;
        const uint4 *fx = reinterpret_cast<const uint4 *>(sSFX + stage * kSkSfBytes) + lane;
        uint32_t v[16];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint4 w = fw[32 * (j % kAtoms)];     // atom j, line `lane` (MX: columns 8..15 are not read)
          v[4 * j] = w.x; v[4 * j + 1] = w.y; v[4 * j + 2] = w.z; v[4 * j + 3] = w.w;
        }
        tmem_st_32x32b_x16(tq + kSkSfBase + stage * kSkSfCols, v);
        if constexpr (FUSE) {
          // rows 0..7, lanes 0..7: the two words of this K tile
          const uint2 w = *reinterpret_cast<const uint2 *>(sSFX + (kt - kt0) * 64 + (lane & 7) * 8);
#pragma unroll
          for (int j = 0; j < 16; ++j) v[j] = lane < 8 ? (j & 4 ? w.y : w.x) : 0u;
        }
#pragma unroll
        for (int j = 0; j < 4 && !FUSE; ++j) {
          const uint4 w = fx[32 * (j % kAtoms)];
          // the MMA's 32 activation rows take their scales from the first of
          // the four columns: the words of this unit's row group go there
          v[4 * j] = !GROUPED || t.sub == 0 ? w.x : t.sub == 1 ? w.y : t.sub == 2 ? w.z : w.w;
          v[4 * j + 1] = w.y; v[4 * j + 2] = w.z; v[4 * j + 3] = w.w;
        }
        tmem_st_32x32b_x16(tq + kSkSfBase + stage * kSkSfCols + 16, v);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sfready[stage]);
        if (++stage == S) {
          stage = 0;
          phase ^= 1;
        }
      }
    }
  } else if (warp < 10) {
    // ------------------------------------------------------------ epilogue --
    // thread = feature n0 + 32q + lane, its 32 columns = the activation rows
    const int q = warp & 3;
    const uint32_t tq = tmem + ((uint32_t)(q * 32) << 16);
    const float alpha = acc_scale_of(p.g_a ? *p.g_a : 1.0f, p.g_b ? *p.g_b : 1.0f);
    int slot = 0;
    uint32_t acc_phase = 0;
    GroupTile ahead = tile_of(blockIdx.x);
    for (int u = blockIdx.x; u < num_units; u += gridDim.x) {
      const Unit t = unit_of(u, ahead);
      ahead = tile_of(u + gridDim.x);
      if (t.rows <= 0) continue;
      const int ks = u % ksplit;
      if (!__all_sync(0xffffffffu, !*abort_flag && mbar_wait(&acc_full[slot], acc_phase, p.timeout_ns))) {
        if (lane == 0) sk_abort(abort_flag, p.status);
        break;
      }
      tc_fence_after();
      uint32_t acc[32];
      __syncwarp();
      tmem_ld_32x32b_x32(tq + slot * kSkN, acc);
      tmem_ld_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&acc_empty[slot]);
      if (++slot == kSkAccs) {
        slot = 0;
        acc_phase ^= 1;
      }
      const int row = q * 32 + lane;
      const int64_t n = (int64_t)t.nt * 128 + row;
      float f[kSkN];
#pragma unroll
      for (int m = 0; m < kSkN; ++m) f[m] = __fmul_rn(__uint_as_float(acc[m]), alpha);
      if (n < p.N) {
#pragma unroll
        for (int m = 0; m < kSkN; ++m) {
          if (m < t.rows) {
            if (p.partial)
              p.partial[((int64_t)ks * p.M + m) * p.N + n] = f[m];
            else if (p.out_fp32)
              reinterpret_cast<float *>(p.d)[(t.out_row + (int64_t)m) * p.ldd + n] = f[m];
            else
              reinterpret_cast<__nv_bfloat16 *>(p.d)[(t.out_row + (int64_t)m) * p.ldd + n] = __float2bfloat16_rn(f[m]);
          }
        }
      }
    }
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, sk_tmem_cols(GROUPED));
  }
}

cudaError_t launch_gemm_fp4_skinny(const GemmParams &p, const CUtensorMap &x, const CUtensorMap &w, int num_sms,
                                   cudaStream_t st) {
  const auto kernel = p.gtiles   ? k_gemm_fp4_skinny<true, true, false>
                      : p.x_bf16 ? k_gemm_fp4_skinny<true, false, true>
                      : p.mx     ? k_gemm_fp4_skinny<true, false, false>
                                 : k_gemm_fp4_skinny<false, false, false>;
  const int smem = sk_smem_bytes(p.gtiles != nullptr);
  if (cudaError_t e = ensure_dynamic_smem((const void *)kernel, smem); e != cudaSuccess) return e;
  // the grouped form and the rows packed by the kernel are MXFP4's
  if ((p.gtiles || p.x_bf16) && !p.mx) return cudaErrorInvalidValue;
  if (p.x_bf16 && !skinny_fuses(p.M, p.num_kt, p.ksplit)) return cudaErrorInvalidValue;
  const int64_t slots = p.gtiles ? 2 * num_sms : num_sms;
  const int64_t units = p.gtiles ? slots : (int64_t)p.tiles_n * std::max(1, p.ksplit);
  const int64_t grid = std::min<int64_t>(units, slots);
  if (grid <= 0) return cudaSuccess;
  return launch_pdl(kernel, dim3((unsigned)grid), dim3(kSkThreads), smem, st, x, w, p);
}

}  // namespace nvfp4
