// route.cu -- group (token, slot) pairs by routed expert for the grouped GEMM.
//
// 256 routed experts, 8 per token ("GLM-5.2-NVFP4" card): the pairs are
// grouped stably by expert id (rows of one expert contiguous, ordered by pair
// index token*top_k + slot).  Three small kernels, no atomics on global memory:
//   hist     per 1024-pair chunk, per-expert counts -> hist[chunk][e]
//   scan     one CTA: counts, offsets, 128-padded offsets, the m-tile table
//            and the padding rows of row_map
//   scatter  per chunk: its base per expert (offset + earlier chunks' counts),
//            then the stable rank of each pair among same-expert pairs (warp
//            match + per-warp counts) -> perm and row_map
// Expert ids outside [0, E) are dropped.
#include "internal.h"
#include "ptx.cuh"

namespace nvfp4 {

constexpr int kRouteChunk = 1024;

__global__ void __launch_bounds__(1024) k_route_hist(const RouteParams p) {
  griddep_launch_dependents();
  griddep_wait();   // inputs may come from the previous kernel in the stream
  extern __shared__ int32_t sh_hist[];   // [E]
  for (int e = threadIdx.x; e < p.num_experts; e += blockDim.x) sh_hist[e] = 0;
  __syncthreads();
  const int64_t i = (int64_t)blockIdx.x * p.chunk + threadIdx.x;
  if (threadIdx.x < p.chunk && i < p.pairs) {
    const int e = p.expert_ids[i];
    // -1 (a missing choice) is dropped, like any other id outside the experts
    if (NVFP4_NOTE(e >= -1 && e < p.num_experts, p.status) && e >= 0) atomicAdd(&sh_hist[e], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < p.num_experts; e += blockDim.x)
    p.hist[(int64_t)blockIdx.x * p.num_experts + e] = sh_hist[e];
}

// Exclusive scan of one value per thread over a 1024-thread block.
__device__ __forceinline__ int32_t block_exclusive_scan(int32_t v, int32_t *scratch, int32_t &total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  int32_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int32_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) scratch[w] = x;
  __syncthreads();
  if (w == 0) {
    int32_t s = scratch[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int32_t y = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += y;
    }
    scratch[32 + lane] = s;     // inclusive warp-sum prefix
  }
  __syncthreads();
  total = scratch[32 + 31];
  const int32_t before = w > 0 ? scratch[32 + w - 1] : 0;
  return before + x - v;
}

// The same scan with every partial sum capped at `cap` (inputs in [0, cap]):
// min(a + b, cap) is associative on such values, so the result is the exact
// prefix sum clamped to cap, and nothing overflows.
__device__ __forceinline__ int32_t block_exclusive_scan_capped(int32_t v, int32_t cap, int32_t *scratch) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  int32_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int32_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x = min(x, cap - y) + y;
  }
  __syncthreads();
  if (lane == 31) scratch[w] = x;
  __syncthreads();
  if (w == 0) {
    int32_t s = scratch[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int32_t y = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s = min(s, cap - y) + y;
    }
    scratch[32 + lane] = s;
  }
  const int32_t prev = __shfl_up_sync(0xffffffffu, x, 1);
  const int32_t in_warp = lane > 0 ? prev : 0;   // capped exclusive prefix within the warp
  __syncthreads();
  const int32_t before = w > 0 ? scratch[32 + w - 1] : 0;
  return min(in_warp, cap - before) + before;
}

// m-tiles of `rows` rows; tile_rows is 128 or 256.
__device__ __forceinline__ int32_t tiles_of(int32_t rows, int tile_rows) {
  return (rows + tile_rows - 1) >> (tile_rows == 256 ? 8 : 7);
}

// Offsets, 128-padded offsets, the m-tile table and the padding rows of row_map
// from one expert count per thread of a 1024-thread block; returns the
// thread's expert's first grouped row and first padded row.
__device__ __forceinline__ void write_layout(const RouteParams &p, int32_t count, int32_t &off, int32_t &poff) {
  __shared__ int32_t scratch[64];
  const int e = threadIdx.x;
  const bool act = e < p.num_experts;
  const int32_t padded = (count + 127) & ~127;
  const int32_t mt = tiles_of(count, p.tile_rows);
  int32_t total, ptotal, mtotal;
  off = block_exclusive_scan(count, scratch, total);
  poff = block_exclusive_scan(padded, scratch, ptotal);
  const int32_t moff = block_exclusive_scan(mt, scratch, mtotal);
  __shared__ int32_t s_cnt[1024], s_off[1024], s_poff[1024], s_moff[1024];
  if (act) {
    p.counts[e] = count;
    p.offsets[e] = off;
    p.poffsets[e] = poff;
    if (p.offsets_out) p.offsets_out[e] = off;
    s_cnt[e] = count;
    s_off[e] = off;
    s_poff[e] = poff;
    s_moff[e] = moff;
  }
  __syncthreads();
  // one warp per expert: its m-tile entries and its padding rows (up to 127)
  // written by the 32 lanes
  {
    const int lane = threadIdx.x & 31;
    for (int x = threadIdx.x >> 5; x < p.num_experts; x += blockDim.x >> 5) {
      const int32_t cnt = s_cnt[x], of = s_off[x], pf = s_poff[x], mo = s_moff[x];
      const int32_t pad = (cnt + 127) & ~127, tr = p.tile_rows;
      for (int j = lane; j * tr < cnt; j += 32) {
        GroupTile g;
        g.expert = x;
        g.a_row0 = pf + tr * j;
        g.valid_rows = min(tr, cnt - tr * j);
        g.out_row0 = of + tr * j;
        if (NVFP4_GUARD(mo + j < p.padded_rows_max / 128, p.status)) p.gtiles[mo + j] = g;
      }
      for (int32_t i = cnt + lane; i < pad; i += 32)
        if (NVFP4_GUARD(pf + i < p.padded_rows_max, p.status)) p.row_map[pf + i] = -1;
    }
  }
  if (threadIdx.x == 0) {
    p.offsets[p.num_experts] = total;
    p.poffsets[p.num_experts] = ptotal;
    if (p.offsets_out) p.offsets_out[p.num_experts] = total;
    p.gnum_mtiles[0] = ptotal / 128;
    p.gnum_mtiles[1] = mtotal;
  }
  // rows past ptotal (= 128 x the m-tile count) are never read: every user of
  // the layout is bounded by the m-tile count
}

__global__ void __launch_bounds__(1024) k_route_scan(const RouteParams p) {
  griddep_launch_dependents();
  griddep_wait();   // inputs may come from the previous kernel in the stream
  const int e = threadIdx.x;
  const bool act = e < p.num_experts;
  int32_t count = 0;
  // up to 32 chunks: every chunk count of this expert in registers at once,
  // and after the scan each chunk's first grouped position is written back
  // over its count; more chunks: eight loads in flight per step, and the
  // scatter kernel forms the chunk bases itself
  const bool few = p.nchunks <= 32;
  int32_t hv[32];
  if (act && few) {
    // unconditional loads (the last chunk repeated, its value masked): all
    // 32 are in flight together
#pragma unroll
    for (int j = 0; j < 32; ++j) hv[j] = p.hist[(int64_t)min(j, p.nchunks - 1) * p.num_experts + e];
#pragma unroll
    for (int j = 0; j < 32; ++j) hv[j] = j < p.nchunks ? hv[j] : 0;
#pragma unroll
    for (int j = 0; j < 32; ++j) count += hv[j];
  } else if (act) {
    int c = 0;
    for (; c + 8 <= p.nchunks; c += 8) {
      int32_t v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = p.hist[(int64_t)(c + j) * p.num_experts + e];
#pragma unroll
      for (int j = 0; j < 8; ++j) count += v[j];
    }
    for (; c < p.nchunks; ++c) count += p.hist[(int64_t)c * p.num_experts + e];
  }
  int32_t off, poff;
  write_layout(p, count, off, poff);
  if (act && few) {
    int32_t b = off;
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      if (j < p.nchunks) p.hist[(int64_t)j * p.num_experts + e] = b;
      b += hv[j];
    }
  }
}

// Stable rank of each of the block's pairs among those with its expert, and
// their perm and row_map entries.  sh_base: first grouped row of this block's
// pairs per expert; sh_first, sh_pfirst: the expert's first grouped and padded
// rows; sh_cnt [32 warps][E] is zero and the block synchronized.
__device__ __forceinline__ void scatter_pairs(const RouteParams &p, int64_t i, bool in, const int32_t *sh_base,
                                              uint16_t *sh_cnt, const int32_t *first, const int32_t *pfirst) {
  const int E = p.num_experts;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  int e = -1;
  if (in) {
    e = p.expert_ids[i];
    if (e < 0 || e >= E) e = -1;
    if (e < 0 && p.pair_row) p.pair_row[i] = -1;
  }
  const unsigned same = __match_any_sync(0xffffffffu, e);
  const unsigned lt = (1u << lane) - 1u;
  const int rank_w = __popc(same & lt);
  if (e >= 0 && (same & lt) == 0) sh_cnt[w * E + e] = (uint16_t)__popc(same);
  __syncthreads();
  if (e >= 0) {
    int before = 0;
    for (int v = 0; v < w; ++v) before += sh_cnt[v * E + e];
    const int32_t pos = sh_base[e] + before + rank_w;
    const int64_t prow = (int64_t)pfirst[e] + (pos - first[e]);
    if (NVFP4_GUARD(pos >= 0 && pos < p.pairs && prow >= 0 && prow < p.padded_rows_max, p.status)) {
      p.perm[pos] = (int32_t)i;
      p.row_map[prow] = (int32_t)(i / p.top_k);
      if (p.pair_row) p.pair_row[i] = (int32_t)prow;
    }
  }
}

__global__ void __launch_bounds__(1024) k_route_scatter(const RouteParams p) {
  griddep_launch_dependents();
  griddep_wait();   // inputs may come from the previous kernel in the stream
  extern __shared__ int32_t sh_base[];   // [E] first grouped position of this chunk's pairs
  const int E = p.num_experts;
  uint16_t *sh_cnt = reinterpret_cast<uint16_t *>(sh_base + E);   // [32 warps][E]
  for (int i = threadIdx.x; i < 32 * E; i += blockDim.x) sh_cnt[i] = 0;
  for (int e = threadIdx.x; e < E; e += blockDim.x) {
    if (p.nchunks <= 32) {
      sh_base[e] = p.hist[(int64_t)blockIdx.x * E + e];   // written by the scan kernel
    } else {
      int32_t b = p.offsets[e];
      for (int c = 0; c < (int)blockIdx.x; ++c) b += p.hist[(int64_t)c * E + e];
      sh_base[e] = b;
    }
  }
  __syncthreads();
  const int64_t i = (int64_t)blockIdx.x * p.chunk + threadIdx.x;
  const bool in = threadIdx.x < p.chunk && i < p.pairs;
  const int32_t total = p.offsets[E];    // (on its way while the pairs are placed)
  scatter_pairs(p, i, in, sh_base, sh_cnt, p.offsets, p.poffsets);
  if (in && i >= total) p.perm[i] = -1;   // dropped pairs leave grouped rows unused at the end
}

// Up to kRouteOnePairs pairs (decode): counts, layout and scatter by one block in one
// launch (the general path's three take 3 + 8 + 5.5 us, each alone).
__global__ void __launch_bounds__(1024) k_route_one(const RouteParams p) {
  griddep_launch_dependents();
  griddep_wait();   // inputs may come from the previous kernel in the stream
  extern __shared__ int32_t sh_one[];                             // [E] counts, [E] offsets, [E] padded offsets
  const int E = p.num_experts;
  int32_t *sh_off = sh_one + E, *sh_poff = sh_off + E;
  uint16_t *sh_cnt = reinterpret_cast<uint16_t *>(sh_poff + E);   // [32 warps][E]
  for (int i = threadIdx.x; i < 32 * E; i += blockDim.x) sh_cnt[i] = 0;
  for (int e = threadIdx.x; e < E; e += blockDim.x) sh_one[e] = 0;
  __syncthreads();
  const bool in = threadIdx.x < p.pairs;
  if (in) {
    const int e = p.expert_ids[threadIdx.x];
    if (NVFP4_NOTE(e >= -1 && e < E, p.status) && e >= 0) atomicAdd(&sh_one[e], 1);   // as above
  }
  __syncthreads();
  int32_t off, poff;
  write_layout(p, (int)threadIdx.x < E ? sh_one[threadIdx.x] : 0, off, poff);
  if ((int)threadIdx.x < E) {
    sh_off[threadIdx.x] = off;
    sh_poff[threadIdx.x] = poff;
  }
  __syncthreads();
  if (in && (int)threadIdx.x >= p.offsets[E]) p.perm[threadIdx.x] = -1;
  scatter_pairs(p, threadIdx.x, in, sh_off, sh_cnt, sh_off, sh_poff);
}

cudaError_t launch_route(const RouteParams &p, cudaStream_t st) {
  if (p.pairs <= kRouteOnePairs) {
    const size_t one = (size_t)p.num_experts * (3 * sizeof(int32_t) + 32 * sizeof(uint16_t));
    if (cudaError_t e = ensure_dynamic_smem((const void *)k_route_one, one); e != cudaSuccess) return e;
    return launch_pdl(k_route_one, dim3(1), dim3(1024), one, st, p);
  }
  cudaError_t e = launch_pdl(k_route_hist, dim3(p.nchunks), dim3(kRouteChunk), p.num_experts * sizeof(int32_t), st, p);
  if (e != cudaSuccess) return e;
  e = launch_pdl(k_route_scan, dim3(1), dim3(1024), 0, st, p);
  if (e != cudaSuccess) return e;
  const size_t sm = (size_t)p.num_experts * sizeof(int32_t) + (size_t)32 * p.num_experts * sizeof(uint16_t);
  if ((e = ensure_dynamic_smem((const void *)k_route_scatter, sm)) != cudaSuccess) return e;
  return launch_pdl(k_route_scatter, dim3(p.nchunks), dim3(kRouteChunk), sm, st, p);
}

// ------------------------------------------- layout from given expert offsets --
// The grouped operand's padded layout when the rows already arrive grouped
// (the down-projection input, in the order of the up-projection's output, or
// a caller's precomputed routing): per expert e, its rows keep their order
// and start at the 128-aligned padded offset.  The offsets are the caller's
// device data, so the counts are clamped to [0, pairs] cumulatively and the
// layout is rebuilt from the clamped counts (goffsets): consistent offsets
// give back the same offsets, inconsistent ones can never index past the
// grouped rows or the padded bound.
__global__ void __launch_bounds__(1024) k_offsets_layout(const int32_t *__restrict__ offsets, int E, int64_t pairs,
                                                         int32_t *goffsets, int32_t *poffsets, GroupTile *gtiles,
                                                         int32_t *gnum_mtiles, int64_t max_tiles, int *status,
                                                         int32_t *row_map, const int32_t *__restrict__ perm,
                                                         int top_k, int32_t *inv, int tile_rows) {
  griddep_launch_dependents();
  griddep_wait();   // inputs may come from the previous kernel in the stream
  __shared__ int32_t scratch[64];
  const int e = threadIdx.x;
  const bool act = e < E;
  if (inv)
    for (int64_t i = threadIdx.x; i < pairs; i += blockDim.x) inv[i] = -1;
  const int64_t diff = act ? (int64_t)offsets[e + 1] - (int64_t)offsets[e] : 0;
  int32_t count = (int32_t)(diff < 0 ? 0 : diff > pairs ? pairs : diff);
  const int32_t before = block_exclusive_scan_capped(count, (int32_t)pairs, scratch);
  count = min(count, (int32_t)pairs - before);
  (void)NVFP4_NOTE(!act || (int64_t)count == diff, status);   // the caller's offsets were clamped
  if (threadIdx.x == 0) (void)NVFP4_NOTE(offsets[0] == 0, status);
  const int32_t padded = (count + 127) & ~127;
  const int32_t mt = tiles_of(count, tile_rows);
  int32_t ctotal, ptotal, mtotal;
  const int32_t off = block_exclusive_scan(count, scratch, ctotal);
  const int32_t poff = block_exclusive_scan(padded, scratch, ptotal);
  const int32_t moff = block_exclusive_scan(mt, scratch, mtotal);
  if (act) {
    goffsets[e] = off;
    poffsets[e] = poff;
    for (int j = 0; j < mt; ++j) {
      GroupTile g;
      g.expert = e;
      g.a_row0 = poff + tile_rows * j;
      g.valid_rows = min(tile_rows, count - tile_rows * j);
      g.out_row0 = off + tile_rows * j;
      if (NVFP4_GUARD(moff + j < max_tiles, status)) gtiles[moff + j] = g;
    }
  }
  if (threadIdx.x == 0) {
    goffsets[E] = ctotal;
    poffsets[E] = ptotal;
    gnum_mtiles[0] = ptotal / 128;
    gnum_mtiles[1] = mtotal;
  }
  if (row_map) {
    // few rows: the row map (and the inverse of perm) by the same block, a
    // warp per expert; rows past ptotal are never read
    __shared__ int32_t s_cnt[1024], s_off[1024], s_poff[1024];
    if (act) {
      s_cnt[e] = count;
      s_off[e] = off;
      s_poff[e] = poff;
    }
    __syncthreads();   // (orders the fill of inv before its entries below, too)
    for (int x = threadIdx.x >> 5; x < E; x += blockDim.x >> 5) {
      const int32_t cnt = s_cnt[x], pad = (cnt + 127) & ~127;
      for (int32_t i = threadIdx.x & 31; i < pad; i += 32) {
        int32_t v = i < cnt ? s_off[x] + i : -1;
        if (perm && top_k && v >= 0) {
          const int32_t pr = perm[v];
          v = NVFP4_NOTE(pr >= 0 && pr < pairs, status) ? pr / top_k : -1;
        }
        if (NVFP4_GUARD(s_poff[x] + i < 128 * max_tiles, status)) row_map[s_poff[x] + i] = v;
      }
    }
    if (inv) {
      for (int64_t i = threadIdx.x; i < ctotal; i += blockDim.x) {
        const int32_t q = perm[i];
        if (NVFP4_NOTE(q >= 0 && q < pairs, status)) inv[q] = (int32_t)i;
      }
    }
  }
}

// row_map[r] = the grouped row that padded row r holds, or -1 (padding); with
// perm given, the token of that row's pair instead (perm[row] / top_k; pair
// indices outside [0, pairs) count as padding).
__global__ void k_rowmap_from_offsets(const int32_t *__restrict__ goffsets,
                                      const int32_t *__restrict__ poffsets, int E, int64_t rows,
                                      const int32_t *__restrict__ perm, int top_k, int64_t pairs,
                                      int32_t *row_map, int *status) {
  griddep_launch_dependents();
  griddep_wait();   // inputs may come from the previous kernel in the stream
  for (int64_t r = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; r < rows;
       r += (int64_t)gridDim.x * blockDim.x) {
    int32_t v = -1;
    if (r < poffsets[E]) {
      int lo = 0, hi = E - 1;            // the last e with poffsets[e] <= r
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (poffsets[mid] <= r) lo = mid;
        else hi = mid - 1;
      }
      const int64_t i = r - poffsets[lo];
      if (i < goffsets[lo + 1] - goffsets[lo]) {
        v = (int32_t)(goffsets[lo] + i);
        if (perm) {
          const int32_t pr = perm[v];
          v = NVFP4_NOTE(pr >= 0 && pr < pairs, status) ? pr / top_k : -1;
        }
      }
    }
    row_map[r] = v;
  }
}

// Up to this many pairs and padded rows the one-block kernel writes the row map
// and the inverse as well: one launch instead of four.  NVFP4 down-projection
// against four launches: 4000 pairs on 32 experts (8064 rows) 57.5 instead of
// 59.7 us, on 8 experts 63.9 instead of 65.7; 6000 pairs on 8 experts 87.2 instead
// of 85.7, 8000 on 32 (12064 rows) 75.9 instead of 74.4.
constexpr int64_t kOneBlockPairs = 4096, kOneBlockRows = 8192;

bool layout_makes_inverse(int64_t pairs, int64_t padded_rows_max) {
  return pairs <= kOneBlockPairs && padded_rows_max <= kOneBlockRows;
}

cudaError_t launch_layout_from_offsets(const int32_t *offsets, int E, int64_t pairs, int64_t padded_rows_max,
                                       int32_t *goffsets, int32_t *poffsets, GroupTile *gtiles,
                                       int32_t *gnum_mtiles, int32_t *row_map, const int32_t *perm, int top_k,
                                       int num_sms, cudaStream_t st, int *status, int32_t *inv, int tile_rows) {
  const bool one = layout_makes_inverse(pairs, padded_rows_max);
  cudaError_t e = launch_pdl(k_offsets_layout, dim3(1), dim3(1024), 0, st, offsets, E, pairs, goffsets, poffsets,
                             gtiles, gnum_mtiles, padded_rows_max / 128, status, one ? row_map : (int32_t *)nullptr,
                             perm, top_k, one ? inv : (int32_t *)nullptr, tile_rows);
  if (e != cudaSuccess || one) return e;
  const int64_t ctas = std::max<int64_t>(1, std::min<int64_t>((padded_rows_max + 255) / 256, (int64_t)num_sms * 4));
  return launch_pdl(k_rowmap_from_offsets, dim3((unsigned)ctas), dim3(256), 0, st, (const int32_t *)goffsets,
                    (const int32_t *)poffsets, E, padded_rows_max, top_k ? perm : (const int32_t *)nullptr, top_k, pairs,
                    row_map, status);
}

// ----------------------------------------------------------------- combine --
// y[t][n] = sum over slots j (in order) of w[t][j] * d[g(t, j)][n], fp32
// accumulation (one fused multiply-add per slot), rounded once to bf16, where
// g(t, j) is the grouped row of pair t*top_k + j (the inverse of perm).
// perm is the caller's device data: only its first *rows entries name grouped
// rows (the last offset: dropped pairs have none), entries outside [0, pairs)
// are skipped, and inv is first filled with -1 so that a pair no entry names
// reads nothing.
__global__ void k_invert_perm(const int32_t *__restrict__ perm, int64_t pairs, const int32_t *__restrict__ rows,
                              int32_t *inv, int *status) {
  griddep_launch_dependents();
  griddep_wait();   // inputs may come from the previous kernel in the stream
  const int32_t n = *rows;     // (read beside the entries, not before them)
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < pairs;
       i += (int64_t)gridDim.x * blockDim.x) {
    const int32_t q = perm[i];
    if (i < n && NVFP4_NOTE(q >= 0 && q < pairs, status)) inv[q] = (int32_t)i;
  }
}
__global__ void k_fill_i32(int32_t *p, int64_t n, int32_t v) {
  griddep_launch_dependents();
  griddep_wait();
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (int64_t)gridDim.x * blockDim.x)
    p[i] = v;
}

// Sixteen bytes of D as floats.
__device__ __forceinline__ void unpack16(uint4 q, float (&f)[8]) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void unpack16(uint4 q, float (&f)[4]) {
  f[0] = __uint_as_float(q.x);
  f[1] = __uint_as_float(q.y);
  f[2] = __uint_as_float(q.z);
  f[3] = __uint_as_float(q.w);
}
// The sums' one rounding to bf16.
__device__ __forceinline__ uint32_t round_pair(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ void store_sums(__nv_bfloat16 *y, const float (&f)[8]) {
  *reinterpret_cast<uint4 *>(y) = make_uint4(round_pair(f[0], f[1]), round_pair(f[2], f[3]), round_pair(f[4], f[5]),
                                             round_pair(f[6], f[7]));
}
__device__ __forceinline__ void store_sums(__nv_bfloat16 *y, const float (&f)[4]) {
  *reinterpret_cast<uint2 *>(y) = make_uint2(round_pair(f[0], f[1]), round_pair(f[2], f[3]));
}

// A warp takes a token, or with few tokens (kSplit) one of `parts` interleaved
// column ranges of it (32 tokens of 6144 bf16 columns, top 8: 4.5 us, with a warp each 22): its
// slots' row indices and weights are read once, and for top_k <= 8 the 16-byte
// loads of all slots are in flight together before the sums (which keep the
// slot order).  TD: bf16, or float (the MXFP4 experts' outputs, which are not
// rounded before the sum).
template <typename TD, bool kSplit>
__global__ void __launch_bounds__(256) k_moe_combine(const TD *__restrict__ d, const int32_t *__restrict__ inv,
                                                     const float *__restrict__ w, int64_t tokens, int top_k,
                                                     int64_t N, __nv_bfloat16 *__restrict__ y, int parts,
                                                     int *status) {
  griddep_launch_dependents();
  griddep_wait();   // inputs may come from the previous kernel in the stream
  constexpr int kMaxK = 8, V = 16 / (int)sizeof(TD);
  const int lane = threadIdx.x & 31;
  const int64_t warp = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  const int64_t nwarps = (int64_t)gridDim.x * (blockDim.x >> 5);
  const int64_t vecs = N / V;                       // 16-byte vectors of a row
  for (int64_t item = warp; item < (kSplit ? tokens * parts : tokens); item += nwarps) {
    const int64_t t = kSplit ? item / parts : item;
    const int64_t v0 = kSplit ? (item - t * parts) * 32 + lane : lane, vstep = kSplit ? 32 * (int64_t)parts : 32;
    if (top_k <= kMaxK) {
      const uint4 *rows[kMaxK];
      float wj[kMaxK];
#pragma unroll
      for (int j = 0; j < kMaxK; ++j) {
        int32_t g = j < top_k ? inv[t * top_k + j] : -1;
        if (!NVFP4_GUARD(g < tokens * top_k, status)) g = -1;
        rows[j] = g >= 0 ? reinterpret_cast<const uint4 *>(d + (int64_t)g * N) : nullptr;
        wj[j] = g >= 0 ? w[t * top_k + j] : 0.0f;
      }
      for (int64_t v = v0; v < vecs; v += vstep) {
        uint4 q[kMaxK];
#pragma unroll
        for (int j = 0; j < kMaxK; ++j) q[j] = rows[j] ? __ldg(rows[j] + v) : make_uint4(0, 0, 0, 0);
        float acc[V];
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] = 0.0f;
#pragma unroll
        for (int j = 0; j < kMaxK; ++j) {
          if (j >= top_k) break;
          float f[V];
          unpack16(q[j], f);
#pragma unroll
          for (int i = 0; i < V; ++i) acc[i] = __fmaf_rn(wj[j], f[i], acc[i]);
        }
        store_sums(y + t * N + v * V, acc);
      }
      continue;
    }
    for (int64_t v = v0; v < vecs; v += vstep) {
      float acc[V];
#pragma unroll
      for (int i = 0; i < V; ++i) acc[i] = 0.0f;
      for (int j = 0; j < top_k; ++j) {
        const int64_t g = inv[t * top_k + j];
        if (g < 0 || !NVFP4_GUARD(g < tokens * top_k, status)) continue;
        const float wv = w[t * top_k + j];
        float f[V];
        unpack16(__ldg(reinterpret_cast<const uint4 *>(d + g * N) + v), f);
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] = __fmaf_rn(wv, f[i], acc[i]);
      }
      store_sums(y + t * N + v * V, acc);
    }
  }
}

cudaError_t launch_moe_combine(const void *d, bool d_fp32, const int32_t *perm, int32_t *inv, const float *w,
                               int64_t tokens, int top_k, int64_t N, __nv_bfloat16 *y, int num_sms,
                               cudaStream_t st, int *status, bool inv_ready, const int32_t *rows) {
  const int64_t pairs = tokens * top_k;
  if (!inv_ready) {
    const int64_t c1 = std::max<int64_t>(1, std::min<int64_t>((pairs + 255) / 256, (int64_t)num_sms * 4));
    cudaError_t e = launch_pdl(k_fill_i32, dim3((unsigned)c1), dim3(256), 0, st, inv, pairs, (int32_t)-1);
    if (e != cudaSuccess) return e;
    e = launch_pdl(k_invert_perm, dim3((unsigned)c1), dim3(256), 0, st, perm, pairs, rows, inv, status);
    if (e != cudaSuccess) return e;
  }
  // column ranges until every SM has 32 warps
  const int64_t vecs = N / (d_fp32 ? 4 : 8);
  const int64_t parts = std::max<int64_t>(1, std::min<int64_t>((vecs + 31) / 32, (int64_t)num_sms * 32 / tokens));
  const int64_t c2 = std::max<int64_t>(1, std::min<int64_t>((tokens * parts + 7) / 8, (int64_t)num_sms * 8));
  const auto go = [&](auto kernel, auto rows_of_d) {
    return launch_pdl(kernel, dim3((unsigned)c2), dim3(256), 0, st, rows_of_d, (const int32_t *)inv, w, tokens, top_k,
                      N, y, (int)parts, status);
  };
  if (d_fp32) {
    const float *df = static_cast<const float *>(d);
    return parts > 1 ? go(k_moe_combine<float, true>, df) : go(k_moe_combine<float, false>, df);
  }
  const __nv_bfloat16 *db = static_cast<const __nv_bfloat16 *>(d);
  return parts > 1 ? go(k_moe_combine<__nv_bfloat16, true>, db) : go(k_moe_combine<__nv_bfloat16, false>, db);
}

}  // namespace nvfp4
