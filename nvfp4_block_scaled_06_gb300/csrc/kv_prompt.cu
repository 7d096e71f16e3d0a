// kv_prompt.cu -- attention of many query rows over the pages of the NVFP4
// cache: prompts, later chunks of them, large groups of heads.
//
// The product's rows are (new token, query head of the group) of one sequence
// and key-value head, 256 to a tile (two M = 128 halves), its keys come 128 at a
// time:  S = Q K^T (f16 operands, exact K, q scaled by a power of two per row),
// P = exp2(S - m), O += P V, m a running reference of the row: 4 below its first
// keys' maximum, to a whole number, raised, with O and l rescaled, when a step's
// numerators sum to more than 2^12, and within a step before one would leave f16,
// so that the row's largest stays 2^3 or more: keys count down to 2^-28 of it
// (f16 ends at 2^-25).
//
// Bound: the tensor cores, 4 x 128 x 256 x head_dim operations per step and 4096
// multiply-adds a cycle; next to them 32768 exponentials (32 a cycle) and the
// decode of 2 x 128 x head_dim cached values.  Roles of a CTA's warps:
//   0-3, 4-7  softmax of one half each, a thread per row: S from tensor memory,
//             P back into the same columns as f16, O's rescaling and the result
//   8-11      a thread per key: packed row -> f16 row in the swizzled K or V
//             tile (a cached value is decoded once per 256 rows)
//   12        issues the MMAs: P V of one half and S of its next step while the
//             softmax of the other half runs
// V's tile lies as K's does, a key per row; it enters as the transposed operand.
//
// Work: the steps of all (row tile, head) segments in one line, cut into equal
// spans, one per CTA, so that long contexts with few rows and causal prompts both
// fill the GPU; segments in several spans leave partial (o, m, l), joined in
// order by a second kernel.  A first kernel lists the row tiles.
//
// Measured: 2 x 1021 queries of 32 heads over 32768 keys of 4, 772 us = 1.40 PFLOP/s
// (73% of cuBLAS's burst rate; 769 to 787 over several GPUs); a prompt of 4096, 64 heads on 8, 267 us = 1.03.
// Traced when the former took 796 us, a key tile was 3470 cycles: a half's softmax
// about 1950 and its MMAs' wait and issue 1430 in turn, the other half beside it;
// the tensor pipe is busy 55%.
#include <float.h>
#include <math_constants.h>

#include <type_traits>

#include "internal.h"
#include "kv.cuh"
#include "ptx.cuh"

namespace nvfp4 {

namespace {

constexpr int kRowsTile = 256;
constexpr int kThreads = 13 * 32;
constexpr int kLift = 4;              // log2 of the numerator at the maximum of a row's first keys
constexpr float kMostF16 = 65504.0f;  // a sum of numerators up to it leaves them all in f16
constexpr float kRaiseSum = 4096.0f;  // of a tile's numerators, beyond which the next raises the reference
// References from here on are compared with products that were rounded like them (half a step of fp32 is 2^-2
// here): an unrounded product and a reference made of the rounded one differ by 2^4 and more from 2^28 on, and the
// row's largest numerator with them.
constexpr float kLarge = 4194304.0f;
constexpr int kTwo = 1 << 30;       // in an item's key tiles: it has rows in both halves
// What a segment costs beside its key tiles, in key tiles: 1, 2, 3, 4, 6 gave 424,
// 326, 272, 270, 278 us for the 4096 prompt, which takes 267 with 3 by now.
constexpr int kOver = 3;
constexpr uint64_t kKvDrainNs = 200000000ull;

template <int HD>
struct Pr {
  static constexpr int kStages = HD == 128 ? 2 : 3;   // of K and of V
  static constexpr int kHalf = 128 * HD * 2;          // 128 f16 rows: Q of one half, a K or V tile
  static constexpr int kO = 256;                      // first column of O in tensor memory (S: 0 and 128)
  static constexpr int kStaging = 16384;              // results of one half on their way out, 128 bytes a row
  static constexpr size_t kSmem = (size_t)(2 + 2 * kStages) * kHalf + 2 * kStaging + 1024;
};

// Instruction descriptor: kind::f16 with f16 A and B, fp32 D; tb: B is MN-major.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, int tb) {
  return (1u << 4) | ((uint32_t)tb << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
// MN-major operand, 128-byte swizzle: rows of 64 f16 along N, one per k, eight
// of them 1024 bytes; the next 64 of N lie `chunk` bytes on.
__device__ __forceinline__ uint64_t sdesc_mn_sw128(uint32_t a, uint32_t chunk) {
  uint64_t d = (a >> 4) & 0x3FFFull;
  d |= (uint64_t)(chunk >> 4) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}
// K-major operand, 128-byte swizzle (sdesc_k_sw128 on a shared-memory address).
__device__ __forceinline__ uint64_t sdesc_k_sw128_u(uint32_t a) { return sdesc_mn_sw128(a, 16); }
// D(tmem) (+)= A(tmem) * B(smem), f16.
__device__ __forceinline__ void tc_mma_f16_ts(uint32_t d, uint32_t a, uint64_t bdesc, uint32_t idesc,
                                              uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void tmem_st_x8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ void tmem_st_x32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
// Waits for this thread's loads from tensor memory; what x holds is used after it.
__device__ __forceinline__ void tmem_ld_wait_for(uint32_t (&x)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(x[0]), "+r"(x[1]), "+r"(x[2]), "+r"(x[3]), "+r"(x[4]), "+r"(x[5]), "+r"(x[6]), "+r"(x[7]),
                 "+r"(x[8]), "+r"(x[9]), "+r"(x[10]), "+r"(x[11]), "+r"(x[12]), "+r"(x[13]), "+r"(x[14]), "+r"(x[15]),
                 "+r"(x[16]), "+r"(x[17]), "+r"(x[18]), "+r"(x[19]), "+r"(x[20]), "+r"(x[21]), "+r"(x[22]),
                 "+r"(x[23]), "+r"(x[24]), "+r"(x[25]), "+r"(x[26]), "+r"(x[27]), "+r"(x[28]), "+r"(x[29]),
                 "+r"(x[30]), "+r"(x[31])::"memory");
}
// One lane of a converged warp, the same each time; a branch on it keeps the
// MMAs' operands in uniform registers.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r)::"memory");
  return r != 0;
}
__device__ __forceinline__ void tmem_ld_wait_for(uint32_t (&x)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(x[0]), "+r"(x[1]), "+r"(x[2]), "+r"(x[3]), "+r"(x[4]), "+r"(x[5]), "+r"(x[6]), "+r"(x[7]),
                 "+r"(x[8]), "+r"(x[9]), "+r"(x[10]), "+r"(x[11]), "+r"(x[12]), "+r"(x[13]), "+r"(x[14]),
                 "+r"(x[15])::"memory");
}
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  return ((uint64_t)__float_as_uint(hi) << 32) | __float_as_uint(lo);
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float lo2(uint64_t a) { return __uint_as_float((uint32_t)a); }
__device__ __forceinline__ float hi2(uint64_t a) { return __uint_as_float((uint32_t)(a >> 32)); }
// 2^-e of a whole number e >= 0, 0 beyond fp32's normal range.
__device__ __forceinline__ float down(float e) {
  return e < 127.0f ? __uint_as_float((uint32_t)(127 - (int)e) << 23) : 0.0f;
}
// The O of these lanes' rows times f.
template <int HD>
__device__ __forceinline__ void scale_o(uint32_t o_col, float f) {
#pragma unroll 1
  for (int c = 0; c < HD / 32; ++c) {
    uint32_t x[32];
    tmem_ld_32x32b_x32(o_col + c * 32, x);
    tmem_ld_wait_for(x);
#pragma unroll
    for (int i = 0; i < 32; ++i) x[i] = __float_as_uint(__uint_as_float(x[i]) * f);
    tmem_st_x32(o_col + c * 32, x);
  }
  tmem_st_wait();
}

// The numerators of a tile's chunks (32 keys) from c on, where a reference is large or a numerator may be beyond f16
// (2^16 times the reference's): such a row is raised to its chunk's largest score, and O (unless it starts with this
// tile), l and the numerators written before follow.  The chunks' scores are all still there: numerators take half
// their columns, from the front.  Returns (m, l, sum of the tile's numerators).  All lanes of a warp; a row's own
// chunks decide what happens to it and sums go in the loop's order, so that the rows around it change nothing.  16
// columns at a time, since the registers are the loop's around (32 spilled there: 4096 prompt 266 -> 275 us).
template <int HD>
__device__ __forceinline__ float4 finish_tile(uint32_t s_col, uint32_t o_col, int c, bool starts, float sc, float m,
                                              float l, float sum) {
#pragma unroll 1
  for (; c < 4; ++c) {
    float mx = -CUDART_INF_F, part = 0.0f;
    // first without storing, for the sum; then with the reference that it calls for
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass) {
      uint32_t x[16];
      const float ref = m == -CUDART_INF_F ? 0.0f : m;
      const bool large = fabsf(ref) >= kLarge;
      float acc[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] = 0.0f;
#pragma unroll 1
      for (int h = 0; h < 2; ++h) {
        uint32_t pk[8];
        tmem_ld_32x32b_x16(s_col + c * 32 + h * 16, x);
        tmem_ld_wait_for(x);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float e[2];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float v = __uint_as_float(x[2 * i + k]);
            mx = fmaxf(mx, v);
            e[k] = ex2(large ? __fmul_rn(v, sc) - ref : __fmaf_rn(v, sc, -ref));
            acc[2 * (i & 3) + k] += e[k];
          }
          pk[i] = pack_h2(e[0], e[1]);
        }
        if (pass == 1) tmem_st_x8(s_col + c * 16 + h * 8, pk);
      }
      part = ((acc[0] + acc[2]) + (acc[4] + acc[6])) + ((acc[1] + acc[3]) + (acc[5] + acc[7]));
      if (pass == 1 || !__any_sync(0xffffffffu, part > kMostF16)) continue;
      const float to = part > kMostF16 ? fmaxf(ceilf(__fmul_rn(mx, sc)) - kLift, m) : m;
      const float f = to > m ? down(to - m) : 1.0f;
      m = to;
      l *= f;
      sum *= f;
      if (!starts) scale_o<HD>(o_col, f);
      tmem_st_wait();                                // (the numerators' stores)
      // (in fp32: f itself may be below f16's range, where 96 numerators of up to 2^11 times f still count)
#pragma unroll 1
      for (int d = 0; d < c; ++d) {
        tmem_ld_32x32b_x16(s_col + d * 16, x);
        tmem_ld_wait_for(x);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&x[i]));
          x[i] = pack_h2(v.x * f, v.y * f);
        }
        tmem_st_32x32b_x16(s_col + d * 16, x);
      }
    }
    sum += part;
  }
  return make_float4(m, l, sum, 0.0f);
}

// ------------------------------------------------------------------- listing --
// Row tiles of the sequences with more than few_rows rows, in order: {sequence,
// tile, first key tile, key tiles}, and the key tiles before each.  One block.
__global__ void __launch_bounds__(1024) k_kv_list(const KvAttnParams p) {
  __shared__ int base[1024];
  __shared__ int64_t wsum[32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  griddep_launch_dependents();
  griddep_wait();
  // exclusive sum over the block, and the block's total
  auto scan = [&](int64_t v, int64_t &total) {
    int64_t s = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t x = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += x;
    }
    __syncthreads();
    if (lane == 31) wsum[warp] = s;
    __syncthreads();
    int64_t t = wsum[lane];                    // the warps' sums, added up by every warp
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t x = __shfl_up_sync(0xffffffffu, t, o);
      if (lane >= o) t += x;
    }
    total = __shfl_sync(0xffffffffu, t, 31);
    const int64_t before = __shfl_sync(0xffffffffu, t, max(warp - 1, 0));
    return (warp > 0 ? before : 0) + s - v;
  };
  int64_t items = 0, units = 0;
  for (int b0 = 0; b0 < p.seqs; b0 += 1024) {
    int64_t n = 0, count;
    if (b0 + tid < p.seqs) {
      const KvSeq s = kv_seq(p, b0 + tid);
      const int64_t rows = (int64_t)s.qn * p.group;
      n = rows > p.few_rows ? (rows + kRowsTile - 1) / kRowsTile : 0;
    }
    const int64_t at = scan(n, count);
    // (offsets that make sequences share rows can name more tiles than there are rows for: those are dropped)
    count = min(count, p.max_items - items);
    base[tid] = (int)min(at, (int64_t)0x7FFFFFFF);
    __syncthreads();
    for (int64_t i0 = 0; i0 < count; i0 += 1024) {
      const int64_t i = i0 + tid;
      int64_t nt = 0, sum;
      int4 it = make_int4(0, 0, 0, 0);
      if (i < count) {
        int lo = 0, hi = 1024;                 // the last sequence that starts at or before i
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (base[mid] <= i) lo = mid; else hi = mid;
        }
        const KvSeq s = kv_seq(p, b0 + lo);
        const int tile = (int)(i - base[lo]);
        const int tok0 = (int)((int64_t)tile * kRowsTile / p.group);
        const int tok1 = (int)min((int64_t)s.qn - 1, ((int64_t)(tile + 1) * kRowsTile - 1) / p.group);
        const int64_t first = p.window > 0 ? (int64_t)s.n - s.qt + tok0 + 1 - p.window : 0;
        const int64_t end = p.causal ? (int64_t)s.n - s.qt + tok1 + 1 : s.n;
        const int t0 = (int)(max(min(first, (int64_t)s.n - 1), (int64_t)0) >> 7);
        nt = max((int64_t)1, ((end + 127) >> 7) - t0);
        const bool two = (int64_t)s.qn * p.group - (int64_t)tile * kRowsTile > 128;
        it = make_int4(b0 + lo, tile, t0, (int)nt | (two ? kTwo : 0));
        nt += kOver;
      }
      const int64_t u = scan(nt, sum);
      if (i < count) {
        p.item_prefix[items + i] = units + u;
        p.items[items + i] = it;
      }
      units += sum;
    }
    items += count;
    __syncthreads();
  }
  if (tid == 0) {
    p.item_prefix[items] = units;
    *p.item_count = (int)items;
  }
}

// The last item that starts at or before unit u (of one head): a warp tries 32
// places at a time.
__device__ __forceinline__ int find_item(const int64_t *prefix, int count, int64_t u) {
  int lo = 0, n = count;
  const int lane = threadIdx.x & 31;
  while (n > 1) {
    const int step = (n + 31) / 32, at = lo + lane * step;
    const bool in = lane * step < n && prefix[at] <= u;
    const int last = 31 - __clz(__ballot_sync(0xffffffffu, in));   // lane 0 holds: prefix[lo] <= u
    n = min(step, n - last * step);
    lo += last * step;
  }
  return lo;
}

// A CTA's way through the segments of its span.  A segment counts as its key
// tiles and kOver more in front, for what it costs beside them.
struct Walk {
  int item, h, j0, j1;      // key tiles [j0, j1) of the segment's
  int seq, tile, t0, nt;    // the item: sequence, row tile, first key tile, key tiles
  int left, r;              // units of the span from the segment's place r on
  bool two;                 // rows in both halves
  __device__ __forceinline__ void load(const KvAttnParams &p) {
    const int4 it = p.items[item];
    seq = it.x;
    tile = it.y;
    t0 = it.z;
    nt = it.w & (kTwo - 1);
    two = (it.w & kTwo) != 0;
  }
  __device__ __forceinline__ void clip() {
    j0 = max(r - kOver, 0);
    j1 = max(min(nt, r + left - kOver), 0);
  }
  // On to the next segment with a key tile in the span.
  __device__ __forceinline__ bool next(const KvAttnParams &p) {
    do {
      left -= nt + kOver - r;
      if (left <= 0) return false;
      if (++h == p.kv_heads) {
        h = 0;
        ++item;
        load(p);
      }
      r = 0;
      clip();
    } while (j0 >= j1);
    return true;
  }
};

// -------------------------------------------------------------------- kernel --
template <int HD>
__global__ void __launch_bounds__(kThreads, 1) k_kv_prompt(const KvAttnParams p) {
  using T = Pr<HD>;
  constexpr int S = T::kStages;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[4 * S + 10];
  __shared__ uint32_t tmem_holder;
  __shared__ uint32_t kmask[4][4];          // keys that exist, of the last four tiles
  __shared__ volatile int abort_flag;
  __shared__ int nan_end;                   // the last tile with a NaN value scale, and one: counted over the CTA's tiles
  // barriers and buffers by their shared-memory addresses
  const uint32_t bar = smem_u32(bars);
  const uint32_t k_full = bar, k_empty = bar + 8 * S, v_full = bar + 16 * S, v_empty = bar + 24 * S;   // (empty 8 S behind full)
  const uint32_t s_ready = bar + 32 * S, p_ready = s_ready + 16, o_full = s_ready + 32, q_ready = s_ready + 48;
  const uint32_t drain = s_ready + 64, never = s_ready + 72;
  const uint32_t smem = (smem_u32(smem_raw) + 1023) & ~1023u;
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;

  if (tid == 0) {
    for (int i = 0; i < 4 * S; ++i) mbar_init(bars + i, (i / S) & 1 ? 1 : 4);   // full: four warps, empty: a commit
    for (int i = 0; i < 8; ++i) mbar_init(bars + 4 * S + i, (i >> 1) & 1 ? 128 : 1);   // p, q: a half's threads
    mbar_init(bars + 4 * S + 8, 1);
    mbar_init(bars + 4 * S + 9, 1);
    abort_flag = 0;
    nan_end = 0;
    fence_barrier_init();
  }
  if (warp == 12) {
    tmem_alloc(&tmem_holder, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_holder;
  griddep_launch_dependents();
  griddep_wait();

  auto give_up = [&] {
    abort_flag = 1;
    record_timeout(p.status);
  };
  // every lane of a warp agrees on whether the wait ended
  auto warp_wait = [&](uint32_t at, uint32_t parity) {
    const bool ok = __all_sync(0xffffffffu, !abort_flag && mbar_wait_u(at, parity, p.timeout_ns));
    if (!ok && lane == 0) give_up();
    return ok;
  };

  const int count = *p.item_count;
  const int64_t total = count > 0 ? p.item_prefix[count] * p.kv_heads : 0;
  const KvCut cut(total, gridDim.x);
  const int64_t cta = blockIdx.x;
  if (cta < cut.spans && note_bounds(tmem == 0, p.status)) {
    Walk w;
    bool any;
    {
      const int64_t u0 = cut.start(cta);
      w.left = (int)(cut.start(cta + 1) - u0);
      w.item = find_item(p.item_prefix, count, kv_div(u0, p.kv_heads));
      // (prefix counts the units of one head: item i's lie from prefix[i] * kv_heads on)
      w.load(p);
      const int64_t base = p.item_prefix[w.item] * p.kv_heads;
      w.h = (int)kv_div(u0 - base, w.nt + kOver);
      const int64_t first = base + (int64_t)w.h * (w.nt + kOver);
      w.r = (int)(u0 - first);
      w.clip();
      // the first border inside a segment stands for it in the joining kernel
      if (tid == 0) {
        const int64_t c0 = cut.owner(first + kOver);
        p.borders[cta] = make_int4(w.j0 > 0 && c0 == cta - 1 ? w.item : -1, w.h,
                                   (int)cut.owner(first + w.nt + kOver - 1),
                                   cut.start(c0) < first ? 1 : 0);
      }
      any = w.j0 < w.j1 || w.next(p);
    }
    if (!any) {
    } else if (warp < 8) {
      // -------------------------------------------------------------- softmax --
      const int half = warp >> 2, row = (warp & 3) * 32 + lane;     // of the half
      const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
      const uint32_t s_col = tmem + lane_off + half * 128, o_col = tmem + lane_off + T::kO + half * HD;
      uint32_t tiles = 0, segs = 0, steps = 0;      // key tiles passed; segments and steps of this half
      bool first_seg = true, ok = true;
      const uint32_t sq = smem + half * T::kHalf + (warp & 3) * 32 * 128;   // this warp's rows of Q
      // A segment as this thread sees it.
      KvSeq s;
      int tok, head;
      int64_t rows;
      auto open = [&] {
        s = kv_seq(p, w.seq);
        rows = (int64_t)s.qn * p.group - (int64_t)w.tile * kRowsTile - half * 128;   // of this half
        const uint32_t grp = p.group, at = (uint32_t)((int64_t)w.tile * kRowsTile % p.group) + half * 128 + row;
        tok = (int)((int64_t)w.tile * kRowsTile / p.group + at / grp);
        head = w.h * p.group + (int)(at % grp);
      };
      // Its bf16 rows of Q into the buffer, 16-byte runs of a row on consecutive lanes; rows past the last are zero.
      auto ask_q = [&] {
        if (rows > 0) {
          constexpr int kL = HD / 8, kR = 32 / kL;
          const int c = lane % kL;
          const int64_t own = (int64_t)(s.q0 + tok) * p.q_ld + (int64_t)head * p.q_head_ld;
#pragma unroll 4
          for (int i = 0; i < 32 / kR; ++i) {
            const int rw = i * kR + lane / kL;
            const int64_t at = __shfl_sync(0xffffffffu, own, rw);
            const bool in = (warp & 3) * 32 + rw < rows;
            cp_async_16(sq + rw * 128 + (c >> 3) * 16384 + (((c & 7) ^ (rw & 7)) << 4),
                        p.q + (in ? at + c * 8 : 0), in ? 16u : 0u);
          }
        }
        cp_async_commit();
      };
      open();
      ask_q();
      do {
        if (rows <= 0) {                             // nothing in this half
          tiles += w.j1 - w.j0;
        } else {
        const bool live = row < rows;
        // the keys [see_lo, see_hi) of this row; rows past the last see all and hold zeros
        int see_lo = 0, see_hi = 0x7FFFFFFF;
        if (live) {
          const int64_t pos = (int64_t)s.n - s.qt + tok;
          see_hi = p.causal ? (int)max((int64_t)0, pos + 1) : s.n;
          if (p.window > 0) see_lo = (int)max((int64_t)0, pos + 1 - p.window);
        }
        const int all_lo = __reduce_max_sync(0xffffffffu, see_lo), all_hi = __reduce_min_sync(0xffffffffu, see_hi);
        // this thread's row to f16, times a power of two that brings its maximum to [2^13, 2^14) (1 for a row with
        // an infinity or a NaN; at most 2^126, which makes f16 numbers of all that bf16 holds below 2^-113)
        cp_async_wait<0>();
        __syncwarp();
        const uint32_t mine = sq + lane * 128, xr = (lane & 7) << 4;
        uint32_t m2 = 0;
#pragma unroll 4
        for (int c = 0; c < HD / 8; ++c) {
          const uint4 v = lds128(mine + (c >> 3) * 16384 + (((c & 7) << 4) ^ xr));
          m2 = __vmaxu2(m2, __vmaxu2(__vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu),
                                     __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu)));
        }
        const int e = (int)(max(m2 & 0xFFFFu, m2 >> 16) >> 7), up = e == 255 ? 127 : min(267 - e, 253);
        const float mul = __uint_as_float((uint32_t)up << 23);
        const float sc = fmaxf(__uint_as_float((uint32_t)(254 - up) << 23) * (p.scale_log2 * p.gk[w.h]), FLT_MIN);
#pragma unroll 4
        for (int c = 0; c < HD / 8; ++c) {
          const uint32_t at = mine + (c >> 3) * 16384 + (((c & 7) << 4) ^ xr);
          const uint4 v = lds128(at);
          sts128(at, pack_h2(bf16lo(v.x) * mul, bf16hi(v.x) * mul), pack_h2(bf16lo(v.y) * mul, bf16hi(v.y) * mul),
                 pack_h2(bf16lo(v.z) * mul, bf16hi(v.z) * mul), pack_h2(bf16lo(v.w) * mul, bf16hi(v.w) * mul));
        }
        fence_proxy_async_shared();
        tc_fence_before();
        mbar_arrive_u(q_ready + 8 * half);
        float m = -CUDART_INF_F, l = 0.0f;
        float last = 0.0f;                           // the last tile's sum of numerators
        for (int j = w.j0; j < w.j1; ++j, ++tiles, ++steps) {
          if (!(ok = warp_wait(s_ready + 8 * half, steps & 1))) break;
          tc_fence_after();
          const int key0 = (w.t0 + j) * 128;
          const uint32_t *km = kmask[tiles & 3];
          const bool whole = key0 >= all_lo && key0 + 128 <= all_hi && (km[0] & km[1] & km[2] & km[3]) == 0xFFFFFFFFu;
          if (!whole) {                              // -inf where the row does not see a key
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
              // of the row's range: the bits from its first key on and below its last
              const int from = min(max(see_lo - key0 - c * 32, 0), 32), to = min(max(see_hi - key0 - c * 32, 0), 32);
              const uint32_t bits = km[c] & (uint32_t)((1ull << to) - 1) & ~(uint32_t)((1ull << from) - 1);
              uint32_t x[32];
              tmem_ld_32x32b_x32(s_col + c * 32, x);
              tmem_ld_wait_for(x);
#pragma unroll
              for (int i = 0; i < 32; ++i) x[i] = bits & (1u << i) ? x[i] : 0xFF800000u;
              tmem_st_x32(s_col + c * 32, x);
            }
            tmem_st_wait();
          }
          // O and l follow a raised reference: times f, a power of two (or 0 for a first maximum)
          auto rescale = [&](float f) {
            l *= f;
            if (j > w.j0) scale_o<HD>(o_col, f);     // (O starts with the first tile)
          };
          // numerators are not negative, so a tile's sum bounds them
          const bool fresh = m == -CUDART_INF_F, over = last > kRaiseSum;
          if (__any_sync(0xffffffffu, fresh || over)) {
            float f = 1.0f;
            if (__any_sync(0xffffffffu, fresh)) {
              float mx = -CUDART_INF_F;
#pragma unroll 1
              for (int c = 0; c < 4; ++c) {
                uint32_t x[32];
                tmem_ld_32x32b_x32(s_col + c * 32, x);
                tmem_ld_wait_for(x);
#pragma unroll
                for (int i = 0; i < 32; ++i) mx = fmaxf(mx, __uint_as_float(x[i]));
              }
              if (fresh && mx > -CUDART_INF_F) {
                m = ceilf(__fmul_rn(mx, sc)) - kLift;
                f = 0.0f;
              }
            }
            if (!fresh && over) {
              // By the last tile's sum, to a power of two: the largest of its 128 numerators, 2^-7 of the sum or
              // more, stays 2^(kLift - 1) or more, where a row's first largest may lie too.  (The sum is at most 2^18.)
              const int e = (int)(__float_as_uint(last) >> 23) - 127 - 7 - (kLift - 1);
              const float was = m;
              m += (float)e;
              f = down(m - was);                     // (by what fp32 raised it)
            }
            rescale(f);
          }
          const float ref = m == -CUDART_INF_F ? 0.0f : m;
          const uint64_t sc2 = pack2(sc, sc);
          float sum = 0.0f;
          uint32_t x[32], pk[16];
          // a chunk's numerators, two to a word, and their sum
          auto numerators = [&] {
            const uint64_t ref2 = pack2(-ref, -ref);
            uint64_t acc[4] = {0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const uint64_t y = fma2(((uint64_t)x[2 * i + 1] << 32) | x[2 * i], sc2, ref2);
              const float e0 = ex2(lo2(y)), e1 = ex2(hi2(y));
              acc[i & 3] = add2(acc[i & 3], pack2(e0, e1));
              pk[i] = pack_h2(e0, e1);
            }
            acc[0] = add2(add2(acc[0], acc[1]), add2(acc[2], acc[3]));
            return lo2(acc[0]) + hi2(acc[0]);
          };
          // (one copy of the loop: a large reference leaves it before the first chunk)
          int c = __any_sync(0xffffffffu, fabsf(ref) >= kLarge) ? 4 : 0;
          bool rest = c != 0;
#pragma unroll 1
          for (; c < 4; ++c) {
            tmem_ld_32x32b_x32(s_col + c * 32, x);
            tmem_ld_wait_for(x);
            const float part = numerators();
            if ((rest = __any_sync(0xffffffffu, part > kMostF16))) break;
            sum += part;
            tmem_st_32x32b_x16(s_col + c * 16, pk);
          }
          if (rest) {
            const float4 y = finish_tile<HD>(s_col, o_col, c & 3, j == w.j0, sc, m, l, sum);
            m = y.x;
            l = y.y;
            sum = y.z;
          }
          l += sum;
          last = sum;
          tmem_st_wait();
          tc_fence_before();
          mbar_arrive_u(p_ready + 8 * half);
        }
        if (!ok) break;
        if (!(ok = warp_wait(o_full + 8 * half, segs & 1))) break;
        tc_fence_after();
        ++segs;

        // A value row with a NaN scale entered the sums as zeros; the rows that see it get their NaN here.  The warp
        // shares the keys up to the last such tile (the copies run up to a ring ahead, so that a segment may be
        // searched for its successor's NaN, to no effect): 96 x 32 queries over 32768 keys, a NaN in one of two heads,
        // 0.61 ms, without one 0.59, and 6.8 with a row's thread reading all its keys for itself in every segment of
        // the CTA from then on.
        uint32_t nan_blocks = 0;
        const int bad = *(volatile int *)&nan_end - (int)(tiles - (w.j1 - w.j0));   // tiles of this segment up to it
        if (__any_sync(0xffffffffu, bad > 0)) {
          const int from = __reduce_min_sync(0xffffffffu, live ? see_lo : 0x7FFFFFFF);
          const int to = __reduce_max_sync(0xffffffffu, live ? see_hi : 0);
          const int tile_end = w.j0 + min(__reduce_max_sync(0xffffffffu, bad), w.j1 - w.j0);
          const int k0 = max((w.t0 + w.j0) * 128, from), k1 = min(min((w.t0 + tile_end) * 128, to), s.n);
          constexpr int kAtOnce = 4;
#pragma unroll 1
          for (int k = k0; k < k1; k += 32 * kAtOnce) {
            int id[kAtOnce];
            uint32_t found[kAtOnce];                 // NaN blocks of this lane's keys, a bit each
#pragma unroll
            for (int y = 0; y < kAtOnce; ++y) {
              const int key = k + 32 * y + lane;
              id[y] = key < k1 ? __ldg(p.table + (int64_t)w.seq * p.table_ld + (key >> p.page_shift)) : -1;
            }
#pragma unroll
            for (int y = 0; y < kAtOnce; ++y) {
              const int key = k + 32 * y + lane;
              const bool in = id[y] >= 0 && id[y] < p.num_pages;
              const uint32_t *sf = reinterpret_cast<const uint32_t *>(
                  p.v_sf + (in ? id[y] * p.sf_stride +
                                     (((int64_t)w.h << p.page_shift) + (key & ((1 << p.page_shift) - 1))) * (HD / 16)
                               : 0));
              found[y] = 0;
#pragma unroll
              for (int i = 0; i < HD / 64; ++i) {
                const uint32_t x = in ? __ldg(sf + i) : 0u;
#pragma unroll
                for (int z = 0; z < 4; ++z)
                  if (((x >> (8 * z)) & 0x7Fu) == 0x7Fu) found[y] |= 1u << (4 * i + z);
              }
            }
#pragma unroll
            for (int y = 0; y < kAtOnce; ++y)
              for (uint32_t left = __ballot_sync(0xffffffffu, found[y] != 0); left != 0; left &= left - 1) {
                const int at = __ffs(left) - 1, key = k + 32 * y + at;
                const uint32_t blocks = __shfl_sync(0xffffffffu, found[y], at);
                if (live && key >= see_lo && key < see_hi) nan_blocks |= blocks;
              }
          }
        }
        const bool full = w.j0 == 0 && w.j1 == w.nt;
        const int64_t prow = (2 * cta + (first_seg ? 0 : 1)) * kRowsTile + half * 128 + row;
        // 128 bytes of each row at a time, through shared memory, so that eight lanes write one row; base: this
        // thread's row of the destination
        const int64_t base = full ? ((int64_t)(s.q0 + tok) * p.out_ld + (int64_t)head * p.out_head_ld) * 2
                                  : prow * HD * 4;
        uint8_t *dst = full ? reinterpret_cast<uint8_t *>(p.out) : reinterpret_cast<uint8_t *>(p.pr_part_o);
        const float f = !full ? 1.0f : l == 0.0f ? 0.0f : p.gv[w.h] / l;
        const uint32_t stage = smem + (2 + 2 * S) * T::kHalf + half * T::kStaging + (warp & 3) * 32 * 128;
        const int64_t rows_now = rows;
        if (live && !full) *reinterpret_cast<float2 *>(p.pr_part_ml + prow * 2) = make_float2(m, l);
        if (live && full && p.lse)
          p.lse[(int64_t)(s.q0 + tok) * p.kv_heads * p.group + head] = kv_lse(m, l);
        // the next segment's Q meanwhile (no MMA reads this one's any more)
        first_seg = false;
        const bool more = w.next(p);
        if (more) {
          open();
          ask_q();
        }
        const int cols = full ? 64 : 32;             // of a round
        const uint32_t put = stage + lane * 128, xl = (lane & 7) << 4;
#pragma unroll 1
        for (int c0 = 0; c0 < HD; c0 += cols) {
#pragma unroll 1
          for (int c = 0; c < cols; c += 32) {
            uint32_t x[32];
            tmem_ld_32x32b_x32(o_col + c0 + c, x);
            tmem_ld_wait_for(x);
            if (__any_sync(0xffffffffu, nan_blocks != 0)) {
              const uint32_t nb = nan_blocks >> ((c0 + c) >> 4);
#pragma unroll
              for (int i = 0; i < 32; ++i) x[i] = (nb >> (i >> 4)) & 1u ? 0x7FC00000u : x[i];
            }
            if (full) {
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                uint32_t h[4];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  h[k] = pack_bf2(__uint_as_float(x[8 * i + 2 * k]) * f, __uint_as_float(x[8 * i + 2 * k + 1]) * f);
                sts128(put + ((((c >> 3) + i) << 4) ^ xl), h[0], h[1], h[2], h[3]);
              }
            } else {
#pragma unroll
              for (int i = 0; i < 8; ++i) sts128(put + ((i << 4) ^ xl), x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
            }
          }
          __syncwarp();
#pragma unroll 4
          for (int i = 0; i < 8; ++i) {
            const int rw = i * 4 + (lane >> 3);
            const uint4 v = lds128(stage + rw * 128 + (((lane & 7) ^ (rw & 7)) << 4));
            const int64_t at = __shfl_sync(0xffffffffu, base, rw);
            if ((warp & 3) * 32 + rw < rows_now)
              *reinterpret_cast<uint4 *>(dst + at + c0 * (full ? 2 : 4) + (lane & 7) * 16) = v;
          }
          __syncwarp();
        }
        tc_fence_before();
        if (!more) break;
        continue;
        }
        first_seg = false;
        if (!w.next(p)) break;
        open();
        ask_q();
      } while (true);
      cp_async_wait<0>();
    } else if (warp < 12) {
      // -------------------------------------------------------- K and V tiles --
      const int key_in = tid - 256;                 // this thread's key of a tile
      const uint32_t sk = smem + 2 * T::kHalf, sv = sk + S * T::kHalf;
      const uint32_t row_off = key_in * 128, sw = key_in & 7;
      struct At {
        int b, h, key, n;
        bool on;
      };
      struct Row {
        uint4 c[HD / 32];
        uint32_t s[HD / 64];
        bool ok;
      };
      Walk a = w;                                   // the walk of the tile two on
      int aj = a.j0, an = 0, ab = -1;
      bool more = true;
      auto take = [&] {                             // the next tile of the span
        At t{0, 0, 0, 0, more};
        if (more) {
          if (a.seq != ab) {
            ab = a.seq;
            an = kv_seq(p, ab).n;
          }
          t.b = ab;
          t.h = a.h;
          t.key = (a.t0 + aj) * 128 + key_in;
          t.n = an;
          if (++aj == a.j1) {
            more = a.next(p);
            aj = a.j0;
          }
        }
        return t;
      };
      auto page_of = [&](const At &t) {             // -1: no such key
        return t.on && t.key < t.n ? __ldg(p.table + (int64_t)t.b * p.table_ld + (t.key >> p.page_shift)) : -1;
      };
      auto read = [&](const At &t, int id, const uint8_t *codes, const uint8_t *sf) {
        Row r;
        r.ok = t.on && t.key < t.n && id >= 0 && id < p.num_pages;
        const int64_t at = ((int64_t)t.h << p.page_shift) + (t.key & ((1 << p.page_shift) - 1));
        const uint4 *c = reinterpret_cast<const uint4 *>(codes + id * p.codes_stride + at * (HD / 2));
        const uint32_t *s = reinterpret_cast<const uint32_t *>(sf + id * p.sf_stride + at * (HD / 16));
#pragma unroll
        for (int i = 0; i < HD / 32; ++i) r.c[i] = r.ok ? __ldg(c + i) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < HD / 64; ++i) r.s[i] = r.ok ? __ldg(s + i) : 0u;
        return r;
      };
      auto write = [&](const Row &r, uint32_t base) {
#pragma unroll
        for (int i = 0; i < HD / 32; ++i) {          // 32 channels, two scales
          const uint32_t pair = e4m3x2_to_h2(i & 1 ? r.s[i >> 1] >> 16 : r.s[i >> 1] & 0xFFFFu);
          const uint32_t cw[4] = {r.c[i].x, r.c[i].y, r.c[i].z, r.c[i].w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t sc2 = __byte_perm(pair, pair, k < 2 ? 0x1010 : 0x3232);
            uint32_t h[4];
            e2m1x8_to_h2(cw[k], h);
            const int c = 4 * i + k;
            sts128(base + (c >> 3) * 16384 + row_off + (((c & 7) ^ sw) << 4), hmul2(h[0], sc2), hmul2(h[1], sc2),
                   hmul2(h[2], sc2), hmul2(h[3], sc2));
          }
        }
        fence_proxy_async_shared();
      };
      At t0 = take(), t1 = take();
      int id0 = page_of(t0), id1 = page_of(t1);
      Row cur = read(t0, id0, p.k_codes, p.k_sf);
      uint32_t tiles = 0, phase = 0;
      int st = 0;
      bool ok = true;
      while (ok && t0.on) {
        At t2;
        int id2;
#pragma unroll 1
        for (int val = 0; val < 2; ++val) {         // the tile's keys, then its values: one copy of the code
          // the row after this one
          Row nxt = read(val ? t1 : t0, val ? id1 : id0, val ? p.k_codes : p.v_codes, val ? p.k_sf : p.v_sf);
          if (val == 0) {
            t2 = take();
            id2 = page_of(t2);
          }
          const uint32_t full = (val ? v_full : k_full) + 8 * st;
          if (!(ok = warp_wait(full + 8 * S, phase ^ 1))) break;
          if (val == 0) {
            const uint32_t have = __ballot_sync(0xffffffffu, cur.ok);
            if (lane == 0) kmask[tiles & 3][warp - 8] = have;
          } else {
#pragma unroll
            for (int i = 0; i < HD / 64; ++i) {
              if ((((cur.s[i] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) != 0) {
#pragma unroll
                for (int y = 0; y < 4; ++y)
                  if (((cur.s[i] >> (8 * y)) & 0x7Fu) == 0x7Fu) cur.s[i] &= ~(0xFFu << (8 * y));
                atomicMax(&nan_end, (int)tiles + 1);
              }
            }
          }
          write(cur, (val ? sv : sk) + st * T::kHalf);
          __syncwarp();
          if (lane == 0) mbar_arrive_u(full);
          cur = nxt;
        }
        t0 = t1;
        t1 = t2;
        id0 = id1;
        id1 = id2;
        ++tiles;
        if (++st == S) {
          st = 0;
          phase ^= 1;
        }
      }
    } else {
      // ------------------------------------------------------------ MMA issue --
      if (warp == 12 && elect_one()) {
        constexpr uint32_t id_s = idesc_f16(128, 128, 0), id_o = idesc_f16(128, HD, 1);
        const uint64_t qd = sdesc_k_sw128_u(smem), kd = sdesc_k_sw128_u(smem + 2 * T::kHalf);
        const uint64_t vd = sdesc_mn_sw128(smem + (2 + S) * T::kHalf, 16384);
        uint32_t q_seen = 0, p_seen = 0;              // phases, a bit for each half
        int st = 0;                                   // stage of the tile at hand, of K and of V
        uint32_t ph = 0;
        bool ok = true;
        // (one lane walks, waits and issues: with the whole warp a step's waits, votes and elections cost 400 cycles)
        auto twait = [&](uint32_t at, uint32_t par) {
          if (mbar_try_wait_u(at, par)) return true;
          if (!abort_flag && mbar_wait_u(at, par, p.timeout_ns)) return true;
          give_up();
          return false;
        };
        if (p.stall_probe) ok = twait(never, 0);   // the expiry path under test
        if (ok) do {
#pragma unroll 1
          for (int j = w.j0 - 1; ok && j < w.j1; ++j) {
            const bool pv = j >= w.j0, more = j + 1 < w.j1;
            const int next = !pv ? st : st + 1 == S ? 0 : st + 1;
            if (pv && !(ok = twait(v_full + 8 * st, ph))) break;
#pragma unroll 1
            for (int half = 0; half < (w.two ? 2 : 1); ++half) {
              if (pv) {
                if (!(ok = twait(p_ready + 8 * half, (p_seen >> half) & 1))) break;
                p_seen ^= 1u << half;
                tc_fence_after();
                const uint64_t b = vd + (uint32_t)(st * (T::kHalf >> 4));
                const uint32_t d = T::kO + half * HD, a = half * 128;
#pragma unroll 4
                for (int k = 0; k < 8; ++k) tc_mma_f16_ts(d, a + k * 8, b + k * 128, id_o, j > w.j0 || k ? 1u : 0u);
              } else {
                if (!(ok = twait(q_ready + 8 * half, (q_seen >> half) & 1))) break;
                q_seen ^= 1u << half;
                tc_fence_after();
              }
              if (more) {
                if (half == 0) {
                  if (!(ok = twait(k_full + 8 * next, pv && next == 0 ? ph ^ 1 : ph))) break;
                  tc_fence_after();
                }
                const uint64_t a = qd + (uint32_t)(half * (T::kHalf >> 4)), b = kd + (uint32_t)(next * (T::kHalf >> 4));
#pragma unroll 4
                for (int k = 0; k < HD / 16; ++k)
                  tc_mma_bf16(half * 128, a + ((k >> 2) * 1024 + (k & 3) * 2), b + ((k >> 2) * 1024 + (k & 3) * 2), id_s, k ? 1u : 0u);
                tc_commit_u(s_ready + 8 * half);
              } else {
                tc_commit_u(o_full + 8 * half);
              }
            }
            if (!ok) break;
            if (pv) tc_commit_u(v_empty + 8 * st);
            if (more) tc_commit_u(k_empty + 8 * next);
            if (pv && ++st == S) {
              st = 0;
              ph ^= 1;
            }
          }
        } while (ok && w.next(p));
        // every MMA issued here completes before tensor memory is freed
        tc_commit_u(drain);
        mbar_wait_u(drain, 0, kKvDrainNs);
      }
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 12) tmem_dealloc(tmem, 512);
}

// Segments that lie in several spans: block = (border between two spans, 8
// rows); the border behind a segment's first span stands for it.
template <int HD>
__global__ void __launch_bounds__(256) k_kv_join(const KvAttnParams p, int ctas) {
  constexpr int kV = HD / 32;
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x + 1, count = *p.item_count;
  const int4 bd = p.borders[c];
  const int64_t total = count > 0 ? p.item_prefix[count] * p.kv_heads : 0;
  if (c >= min((int64_t)ctas, total) || bd.x < 0) return;
  const int4 it = p.items[bd.x];      // (its key tiles are not needed)
  const int h = bd.y, c0 = c - 1, c1 = bd.z, first_slot = bd.w;
  const KvSeq s = kv_seq(p, it.x);
  const int64_t rows = min((int64_t)s.qn * p.group - (int64_t)it.y * kRowsTile, (int64_t)kRowsTile);
  for (int r = blockIdx.y * 8 + warp; r < rows; r += 8 * gridDim.y) {
    float m = -CUDART_INF_F, l = 0.0f, o[kV];
#pragma unroll
    for (int v = 0; v < kV; ++v) o[v] = 0.0f;
#pragma unroll 2
    for (int x = c0; x <= c1; ++x) {
      const int64_t prow = (2ll * x + (x == c0 ? first_slot : 0)) * kRowsTile + r;
      const float2 ml = __ldg(reinterpret_cast<const float2 *>(p.pr_part_ml) + prow);
      const float *src = p.pr_part_o + prow * HD + lane * kV;
      float y[kV];
      if constexpr (kV == 4) {
        const float4 v = __ldg(reinterpret_cast<const float4 *>(src));
        y[0] = v.x; y[1] = v.y; y[2] = v.z; y[3] = v.w;
      } else {
        const float2 v = __ldg(reinterpret_cast<const float2 *>(src));
        y[0] = v.x; y[1] = v.y;
      }
      const float m2 = fmaxf(m, ml.x), ref = m2 == -CUDART_INF_F ? 0.0f : m2;
      const float f0 = ex2(m - ref), f1 = ex2(ml.x - ref);
      m = m2;
      l = l * f0 + ml.y * f1;
#pragma unroll
      for (int v = 0; v < kV; ++v) o[v] = o[v] * f0 + y[v] * f1;
    }
    const int64_t rr = (int64_t)it.y * kRowsTile + r;
    const int tok = (int)(rr / p.group), head = h * p.group + (int)(rr % p.group);
    const float f = l == 0.0f ? 0.0f : p.gv[h] / l;
    __nv_bfloat16 *dst = p.out + (int64_t)(s.q0 + tok) * p.out_ld + (int64_t)head * p.out_head_ld + lane * kV;
    if constexpr (kV == 4)
      *reinterpret_cast<uint2 *>(dst) = make_uint2(pack_bf2(o[0] * f, o[1] * f), pack_bf2(o[2] * f, o[3] * f));
    else
      *reinterpret_cast<uint32_t *>(dst) = pack_bf2(o[0] * f, o[1] * f);
    if (p.lse && lane == 0)
      p.lse[(int64_t)(s.q0 + tok) * p.kv_heads * p.group + head] = kv_lse(m, l);
  }
}

template <int HD>
cudaError_t run_prompt(const KvAttnParams &p, int num_sms, cudaStream_t st) {
  if (cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void *>(k_kv_prompt<HD>), Pr<HD>::kSmem);
      e != cudaSuccess)
    return e;
  if (cudaError_t e = launch_pdl(k_kv_list, dim3(1), dim3(1024), 0, st, p); e != cudaSuccess) return e;
  if (cudaError_t e = launch_pdl(k_kv_prompt<HD>, dim3(num_sms), dim3(kThreads), Pr<HD>::kSmem, st, p);
      e != cudaSuccess)
    return e;
  if (num_sms < 2) return cudaSuccess;
  return launch_pdl(k_kv_join<HD>, dim3(num_sms - 1, kRowsTile / 8), dim3(256), 0, st, p, num_sms);
}

}  // namespace

int64_t kv_prompt_max_items(int64_t total_q, int64_t group, int64_t seqs) {
  return total_q * group / kRowsTile + seqs;
}
int64_t kv_prompt_slots(int num_sms) { return 2ll * num_sms * kRowsTile; }

cudaError_t launch_kv_prompt(const KvAttnParams &p, int head_dim, int num_sms, cudaStream_t st) {
  return head_dim == 128 ? run_prompt<128>(p, num_sms, st) : run_prompt<64>(p, num_sms, st);
}

}  // namespace nvfp4
