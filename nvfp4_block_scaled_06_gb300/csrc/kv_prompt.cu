// kv_prompt.cu -- attention of many query rows over the pages of the NVFP4
// cache: prompts, later chunks of them, large groups of heads.
//
// The product's rows are (new token, query head of the group) of one sequence
// and key-value head, 256 to a tile (two M = 128 halves), its keys come 128 at a
// time:  S = Q K^T (f16 operands, exact K, q scaled by a power of two per row),
// P = exp2(S - m), O += P V, m a running reference of the row as in the kernel
// for few rows: it is raised, and O and l rescaled, only when a numerator would
// exceed 2^8.
//
// Bound: the tensor cores, 4 x 128 x 256 x head_dim operations per step and 4096
// multiply-adds a cycle; next to them 32768 exponentials (32 a cycle) and the
// decode of 2 x 128 x head_dim cached values.  Roles of a CTA's warps:
//   0-3, 4-7  softmax of one half each, a thread per row: S from tensor memory,
//             P back into the same columns as f16, O's rescaling and the result
//   8-11      a thread per key: packed row -> f16 row in the swizzled K or V
//             tile (a cached value is decoded once per 256 rows)
//   12        issues the MMAs: P V of one half and S of its next step while the
//             softmax of the other half runs (13-15 idle: registers move by
//             warpgroup)
// V's tile lies as K's does, a key per row; it enters as the transposed operand.
//
// Work: the steps of all (row tile, head) segments in one line, cut into equal
// spans, one per CTA, so that long contexts with few rows and causal prompts both
// fill the GPU; segments in several spans leave partial (o, m, l), joined in
// order by a second kernel.  A first kernel lists the row tiles.
#include <float.h>
#include <math_constants.h>

#include <type_traits>

#include "internal.h"
#include "kv.cuh"
#include "ptx.cuh"

namespace nvfp4 {

namespace {

constexpr int kRowsTile = 256;
constexpr int kThreads = 16 * 32;
// Registers per thread of the three kinds of warpgroups (softmax twice): as many as the launch's 512 x 128.
constexpr int kRegsSoftmax = 184, kRegsTiles = 88, kRegsMma = 56;
static_assert(128 * (2 * kRegsSoftmax + kRegsTiles + kRegsMma) == kThreads * 128, "");
constexpr float kRaiseBy = 8.0f;
constexpr uint64_t kKvDrainNs = 200000000ull;

template <int HD>
struct Pr {
  static constexpr int kStages = HD == 128 ? 2 : 3;   // of K and of V
  static constexpr int kHalf = 128 * HD * 2;          // 128 f16 rows: Q of one half, a K or V tile
  static constexpr int kO = 256;                      // first column of O in tensor memory (S: 0 and 128)
  static constexpr size_t kSmem = (size_t)(2 + 2 * kStages) * kHalf + 1024;
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
// D(tmem) (+)= A(tmem) * B(smem), f16.
__device__ __forceinline__ void tc_mma_f16_ts(uint32_t d, uint32_t a, uint64_t bdesc, uint32_t idesc,
                                              uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(bdesc), "r"(idesc), "r"(accumulate)
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
template <int N>
__device__ __forceinline__ void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
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
__device__ __forceinline__ uint32_t hmax2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

__device__ __forceinline__ int64_t pr_start(int64_t c, int64_t total, int64_t spans) { return c * total / spans; }
__device__ __forceinline__ int64_t pr_owner(int64_t u, int64_t total, int64_t spans) {
  return ((u + 1) * spans - 1) / total;
}

// ------------------------------------------------------------------- listing --
// Row tiles of the sequences with more than few_rows rows, in order: {sequence,
// tile, first key tile, key tiles}, and the key tiles before each.  One block.
__global__ void __launch_bounds__(1024) k_kv_list(const KvAttnParams p) {
  __shared__ int base[1025];
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
    base[tid] = (int)at;
    if (tid == 0) base[1024] = (int)count;
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
        it = make_int4(b0 + lo, tile, t0, (int)nt);
      }
      const int64_t u = scan(nt, sum);
      // (offsets that make sequences share rows can name more tiles than there are rows for: those are dropped)
      if (i < count && items + i <= p.max_items) p.item_prefix[items + i] = units + u;
      if (i < count && NVFP4_NOTE(items + i < p.max_items, p.status)) p.items[items + i] = it;
      units += sum;
    }
    items += count;
    __syncthreads();
  }
  if (tid == 0) {
    if (items <= p.max_items) p.item_prefix[items] = units;
    *p.item_count = (int)min(items, p.max_items);
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

// A CTA's way through the segments of its span.
struct Walk {
  int item, h, j0, j1;      // key tiles [j0, j1) of the segment's
  int4 it;
  int64_t left;             // units of the span from j0 on
  __device__ __forceinline__ void clip() { j1 = (int)min((int64_t)it.w, j0 + left); }
  __device__ __forceinline__ bool next(const KvAttnParams &p) {
    left -= j1 - j0;
    if (left <= 0) return false;
    if (++h == p.kv_heads) {
      h = 0;
      it = __ldg(p.items + ++item);
    }
    j0 = 0;
    clip();
    return true;
  }
};

// -------------------------------------------------------------------- kernel --
template <int HD>
__global__ void __launch_bounds__(kThreads, 1) k_kv_prompt(const KvAttnParams p) {
  using T = Pr<HD>;
  constexpr int S = T::kStages;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[2 * S + 2 * S + 8 + 2];
  __shared__ uint32_t tmem_holder;
  __shared__ uint32_t kmask[4][4];          // keys that exist, of the last four tiles
  __shared__ volatile int abort_flag, nan_flag;
  uint64_t *k_full = bars, *k_empty = bars + S, *v_full = bars + 2 * S, *v_empty = bars + 3 * S;
  uint64_t *s_ready = bars + 4 * S, *p_ready = s_ready + 2, *o_full = s_ready + 4, *q_ready = s_ready + 6;
  uint64_t *drain = s_ready + 8, *never = s_ready + 9;
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;

  if (tid == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(k_full + i, 4);
      mbar_init(k_empty + i, 1);
      mbar_init(v_full + i, 4);
      mbar_init(v_empty + i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(s_ready + i, 1);
      mbar_init(p_ready + i, 128);
      mbar_init(o_full + i, 1);
      mbar_init(q_ready + i, 128);
    }
    mbar_init(drain, 1);
    mbar_init(never, 1);
    abort_flag = 0;
    nan_flag = 0;
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
  auto warp_wait = [&](uint64_t *bar, uint32_t parity) {
    const bool ok = __all_sync(0xffffffffu, !abort_flag && mbar_wait(bar, parity, p.timeout_ns));
    if (!ok && lane == 0) give_up();
    return ok;
  };

  const int count = *p.item_count;
  const int64_t total = count > 0 ? p.item_prefix[count] * p.kv_heads : 0;
  const int64_t spans = min((int64_t)gridDim.x, total), cta = blockIdx.x;
  if (cta < spans) {
    Walk w;
    {
      const int64_t u0 = pr_start(cta, total, spans);
      w.left = pr_start(cta + 1, total, spans) - u0;
      w.item = find_item(p.item_prefix, count, u0 / p.kv_heads);
      // (prefix counts the units of one head: item i's lie from prefix[i] * kv_heads on)
      w.it = __ldg(p.items + w.item);
      const int64_t r = u0 - p.item_prefix[w.item] * p.kv_heads;
      w.h = (int)(r / w.it.w);
      w.j0 = (int)(r - (int64_t)w.h * w.it.w);
      w.clip();
    }
    if (warp < 8) {
      // -------------------------------------------------------------- softmax --
      regs_up<kRegsSoftmax>();
      const int half = warp >> 2, row = (warp & 3) * 32 + lane;     // of the half
      const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
      const uint32_t s_col = tmem + lane_off + half * 128, o_col = tmem + lane_off + T::kO + half * HD;
      uint8_t *sq = smem + half * T::kHalf;
      uint32_t tiles = 0, segs = 0, steps = 0;      // key tiles passed; segments and steps of this half
      bool first_seg = true, ok = true;
      do {
        const KvSeq s = kv_seq(p, w.it.x);
        const int64_t rows = (int64_t)s.qn * p.group - (int64_t)w.it.y * kRowsTile;
        if (rows <= half * 128) {                    // nothing in this half
          tiles += w.j1 - w.j0;
          first_seg = false;
          continue;
        }
        const bool live = half * 128 + row < rows;
        // row r of the tile: token tok0 + (rem0 + r) / group, head (rem0 + r) % group of the group
        const int tok0 = (int)((int64_t)w.it.y * kRowsTile / p.group);
        const uint32_t rem0 = (uint32_t)((int64_t)w.it.y * kRowsTile % p.group) + half * 128, grp = p.group;
        const int tok = tok0 + (int)((rem0 + row) / grp), head = w.h * p.group + (int)((rem0 + row) % grp);
        // the keys [see_lo, see_hi) of this row; rows past the last see all and hold zeros
        int see_lo = 0, see_hi = 0x7FFFFFFF;
        if (live) {
          const int64_t pos = (int64_t)s.n - s.qt + tok;
          see_hi = p.causal ? (int)max((int64_t)0, pos + 1) : s.n;
          if (p.window > 0) see_lo = (int)max((int64_t)0, pos + 1 - p.window);
        }
        const int all_lo = __reduce_max_sync(0xffffffffu, see_lo), all_hi = __reduce_min_sync(0xffffffffu, see_hi);
        // Q: 16-byte runs of a row on consecutive lanes; a row's lanes agree on its power of two
        float sc = 0.0f;
        {
          constexpr int kL = HD / 8, kR = 32 / kL;   // lanes of a row, rows at a time
          const float gsc = p.scale_log2 * p.gk[w.h];
          const int c = lane % kL;
          const int64_t own = (int64_t)(s.q0 + tok) * p.q_ld + (int64_t)head * p.q_head_ld;
          uint4 v[32 / kR];
#pragma unroll
          for (int i = 0; i < 32 / kR; ++i) {
            const int src = i * kR + lane / kL;
            const int64_t at = __shfl_sync(0xffffffffu, own, src);
            v[i] = make_uint4(0, 0, 0, 0);
            if (half * 128 + (warp & 3) * 32 + src < rows) v[i] = __ldg(reinterpret_cast<const uint4 *>(p.q + at) + c);
          }
#pragma unroll
          for (int i = 0; i < 32 / kR; ++i) {
            const int rw = (warp & 3) * 32 + i * kR + lane / kL;
            const uint32_t x[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
            uint32_t m2 = __vmaxu2(__vmaxu2(x[0] & 0x7FFF7FFFu, x[1] & 0x7FFF7FFFu),
                                   __vmaxu2(x[2] & 0x7FFF7FFFu, x[3] & 0x7FFF7FFFu));
#pragma unroll
            for (int o = 1; o < kL; o <<= 1) m2 = __vmaxu2(m2, __shfl_xor_sync(0xffffffffu, m2, o));
            const int e = (int)(max(m2 & 0xFFFFu, m2 >> 16) >> 7);
            // a power of two that brings the row's maximum to [2^13, 2^14); 1 for rows with an infinity or a NaN
            const int up = e == 255 ? 127 : min(267 - e, 190);
            const float mul = __uint_as_float((uint32_t)up << 23);
            uint32_t h[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) h[k] = pack_h2(bf16lo(x[k]) * mul, bf16hi(x[k]) * mul);
            sts128(smem_u32(sq) + rw * 128 + (c >> 3) * 16384 + (((c & 7) ^ (rw & 7)) << 4), h[0], h[1], h[2], h[3]);
            const int back = __shfl_sync(0xffffffffu, 254 - up, lane % kR * kL);
            if (lane / kR == i) sc = fmaxf(__uint_as_float((uint32_t)back << 23) * gsc, FLT_MIN);
          }
        }
        fence_proxy_async_shared();
        tc_fence_before();
        mbar_arrive(q_ready + half);
        {
          // the next segment's row of Q on its way to L2
          Walk nx = w;
          if (nx.next(p)) {
            const KvSeq s2 = kv_seq(p, nx.it.x);
            const int64_t r2 = (int64_t)nx.it.y * kRowsTile + half * 128 + row;
            if (r2 < (int64_t)s2.qn * p.group) {
              const __nv_bfloat16 *src = p.q + (s2.q0 + r2 / p.group) * p.q_ld +
                                         (nx.h * p.group + r2 % p.group) * p.q_head_ld;
#pragma unroll
              for (int i = 0; i < HD; i += 64) asm volatile("prefetch.global.L2 [%0];" ::"l"(src + i));
            }
          }
        }
        float m = -CUDART_INF_F, l = 0.0f;
        for (int j = w.j0; j < w.j1; ++j, ++tiles, ++steps) {
          if (!(ok = warp_wait(s_ready + half, steps & 1))) break;
          tc_fence_after();
          const int key0 = (w.it.z + j) * 128;
          const uint32_t *km = kmask[tiles & 3];
          const bool whole = key0 >= all_lo && key0 + 128 <= all_hi && (km[0] & km[1] & km[2] & km[3]) == 0xFFFFFFFFu;
          // -inf where the row does not see a key, of the 32 from chunk c on
          auto mask = [&](int c, uint32_t (&x)[32]) {
            if (whole) return;
            // of the row's range: the bits from its first key on and below its last
            const int from = min(max(see_lo - key0 - c * 32, 0), 32), to = min(max(see_hi - key0 - c * 32, 0), 32);
            const uint32_t bits = km[c] & (uint32_t)((1ull << to) - 1) & ~(uint32_t)((1ull << from) - 1);
#pragma unroll
            for (int i = 0; i < 32; ++i) x[i] = bits & (1u << i) ? x[i] : 0xFF800000u;
          };
          uint32_t pk[64];
          float sum;
          bool scan = __any_sync(0xffffffffu, m == -CUDART_INF_F);
          while (true) {
            if (scan) {
              float mx = -CUDART_INF_F;
#pragma unroll 1
              for (int c = 0; c < 4; ++c) {
                uint32_t x[32];
                tmem_ld_32x32b_x32(s_col + c * 32, x);
                tmem_ld_wait_for(x);
                mask(c, x);
#pragma unroll
                for (int i = 0; i < 32; ++i) mx = fmaxf(mx, __uint_as_float(x[i]));
              }
              mx *= sc;
              const bool up = mx > m + kRaiseBy;
              const float f = up ? ex2(m - mx) : 1.0f;
              if (up) m = mx;
              l *= f;
              if (j > w.j0 && __any_sync(0xffffffffu, up)) {
#pragma unroll 1
                for (int c = 0; c < HD / 32; ++c) {
                  uint32_t x[32];
                  tmem_ld_32x32b_x32(o_col + c * 32, x);
                  tmem_ld_wait_for(x);
#pragma unroll
                  for (int i = 0; i < 32; ++i) x[i] = __float_as_uint(__uint_as_float(x[i]) * f);
                  tmem_st_x32(o_col + c * 32, x);
                }
              }
            }
            const float ref = m == -CUDART_INF_F ? 0.0f : m;
            const uint64_t sc2 = pack2(sc, sc), ref2 = pack2(-ref, -ref);
            uint64_t acc[2] = {0, 0};
            uint32_t top = 0;
            uint32_t buf[2][32];
            tmem_ld_32x32b_x32(s_col, buf[0]);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              uint32_t (&x)[32] = buf[c & 1];
              tmem_ld_wait_for(x);
              if (c < 3) tmem_ld_32x32b_x32(s_col + (c + 1) * 32, buf[(c + 1) & 1]);
              mask(c, x);
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                const uint64_t y = fma2(((uint64_t)x[2 * i + 1] << 32) | x[2 * i], sc2, ref2);
                const float e0 = ex2(lo2(y)), e1 = ex2(hi2(y));
                acc[i & 1] = add2(acc[i & 1], pack2(e0, e1));
                pk[c * 16 + i] = pack_h2(e0, e1);
                top = hmax2(top, pk[c * 16 + i]);
              }
            }
            sum = (lo2(acc[0]) + hi2(acc[0])) + (lo2(acc[1]) + hi2(acc[1]));
            // f16 256 = 0x5C00; numerators are not negative, so their bits are in order
            const bool over = max(top & 0xFFFFu, top >> 16) > 0x5C00u;
            if (scan || !__any_sync(0xffffffffu, over)) break;
            scan = true;
          }
          l += sum;
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t x[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) x[i] = pk[c * 32 + i];
            tmem_st_x32(s_col + c * 32, x);
          }
          tmem_st_wait();
          tc_fence_before();
          mbar_arrive(p_ready + half);
        }
        if (!ok) break;
        if (!(ok = warp_wait(o_full + half, segs & 1))) break;
        tc_fence_after();
        ++segs;

        // A value row with a NaN scale entered the sums as zeros; the rows that see it get their NaN here.
        uint32_t nan_blocks = 0;
        if (nan_flag && live) {
          const int k0 = max((w.it.z + w.j0) * 128, see_lo), k1 = min(min((w.it.z + w.j1) * 128, see_hi), s.n);
          for (int k = k0; k < k1; ++k) {
            const int id = __ldg(p.table + (int64_t)w.it.x * p.table_ld + (k >> p.page_shift));
            if (id < 0 || id >= p.num_pages) continue;
            const uint8_t *sf = p.v_sf + id * p.sf_stride +
                                (((int64_t)w.h << p.page_shift) + (k & ((1 << p.page_shift) - 1))) * (HD / 16);
            for (int i = 0; i < HD / 16; ++i)
              if ((__ldg(sf + i) & 0x7Fu) == 0x7Fu) nan_blocks |= 1u << i;
          }
        }
        const bool full = w.j0 == 0 && w.j1 == w.it.w;
        const int64_t prow = (2 * cta + (first_seg ? 0 : 1)) * kRowsTile + half * 128 + row;
        // 256 bytes of each of the warp's rows at a time go through its rows of Q, which no MMA reads any more
        // (o_full), so that 16 lanes write one row; own: this thread's row of the destination in 16-byte runs
        const uint32_t stage = smem_u32(sq) + (warp & 3) * 32 * 128;
        auto put = [&](int q, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
          sts128(stage + lane * 128 + (q >> 3) * 16384 + (((q & 7) ^ (lane & 7)) << 4), a0, a1, a2, a3);
        };
        auto flush = [&](auto width, uint4 *base, int64_t own) {
          constexpr int kL = decltype(width)::value / 16, kR = 32 / kL;   // lanes of a row, rows at a time
          const int q = lane % kL;
          uint4 v[32 / kR];
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 32 / kR; ++i) {
            const int rw = i * kR + lane / kL;
            v[i] = lds128(stage + rw * 128 + (q >> 3) * 16384 + (((q & 7) ^ (rw & 7)) << 4));
          }
#pragma unroll
          for (int i = 0; i < 32 / kR; ++i) {
            const int rw = i * kR + lane / kL;
            const int64_t at = __shfl_sync(0xffffffffu, own, rw);
            if (half * 128 + (warp & 3) * 32 + rw < rows) base[at + q] = v[i];
          }
          __syncwarp();
        };
        auto nans = [&](int c, uint32_t (&x)[32]) {      // columns 32 c ...
          if (!__any_sync(0xffffffffu, nan_blocks != 0)) return;
          const uint32_t nb = nan_blocks >> (2 * c);
#pragma unroll
          for (int i = 0; i < 32; ++i) x[i] = (nb >> (i >> 4)) & 1u ? 0x7FC00000u : x[i];
        };
        if (full) {
          const float f = l == 0.0f ? 0.0f : p.gv[w.h] / l;
#pragma unroll
          for (int c = 0; c < HD / 32; ++c) {
            uint32_t x[32];
            tmem_ld_32x32b_x32(o_col + c * 32, x);
            tmem_ld_wait_for(x);
            nans(c, x);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t h[4];
#pragma unroll
              for (int k = 0; k < 4; ++k)
                h[k] = pack_bf2(__uint_as_float(x[8 * i + 2 * k]) * f, __uint_as_float(x[8 * i + 2 * k + 1]) * f);
              put(4 * c + i, h[0], h[1], h[2], h[3]);
            }
          }
          flush(std::integral_constant<int, HD * 2>(), reinterpret_cast<uint4 *>(p.out),
                ((int64_t)(s.q0 + tok) * p.out_ld + (int64_t)head * p.out_head_ld) / 8);
          if (live && p.lse)
            p.lse[(int64_t)(s.q0 + tok) * p.kv_heads * p.group + head] = (m + __log2f(l)) * CUDART_LN2_F;
        } else {
          constexpr int kCols = HD / 2;                  // of a round: 2 HD bytes of a row
#pragma unroll 1
          for (int rd = 0; rd < 2; ++rd) {
#pragma unroll
            for (int c = 0; c < kCols / 32; ++c) {
              uint32_t x[32];
              tmem_ld_32x32b_x32(o_col + rd * kCols + c * 32, x);
              tmem_ld_wait_for(x);
              nans(rd * (kCols / 32) + c, x);
#pragma unroll
              for (int i = 0; i < 8; ++i) put(8 * c + i, x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
            }
            flush(std::integral_constant<int, HD * 2>(), reinterpret_cast<uint4 *>(p.pr_part_o) + rd * (HD / 8),
                  prow * (HD / 4));
          }
          if (live) *reinterpret_cast<float2 *>(p.pr_part_ml + prow * 2) = make_float2(m, l);
        }
        tc_fence_before();
        first_seg = false;
      } while (w.next(p));
    } else if (warp < 12) {
      // -------------------------------------------------------- K and V tiles --
      regs_down<kRegsTiles>();
      const int key_in = tid - 256;                 // this thread's key of a tile
      const uint32_t sk = smem_u32(smem) + 2 * T::kHalf, sv = sk + S * T::kHalf;
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
          if (a.it.x != ab) {
            ab = a.it.x;
            an = kv_seq(p, ab).n;
          }
          t.b = ab;
          t.h = a.h;
          t.key = (a.it.z + aj) * 128 + key_in;
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
        r.ok = t.on && t.key < t.n && NVFP4_NOTE(id >= 0 && id < p.num_pages, p.status);
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
      Row k = read(t0, id0, p.k_codes, p.k_sf);
      uint32_t tiles = 0, phase = 0;
      int st = 0;
      while (t0.on) {
        Row v = read(t0, id0, p.v_codes, p.v_sf);
        const At t2 = take();
        const int id2 = page_of(t2);
        if (!warp_wait(k_empty + st, phase ^ 1)) break;
        const uint32_t have = __ballot_sync(0xffffffffu, k.ok);
        if (lane == 0) kmask[tiles & 3][warp - 8] = have;
        write(k, sk + st * T::kHalf);
        __syncwarp();
        if (lane == 0) mbar_arrive(k_full + st);
        k = read(t1, id1, p.k_codes, p.k_sf);
        if (!warp_wait(v_empty + st, phase ^ 1)) break;
#pragma unroll
        for (int i = 0; i < HD / 64; ++i) {
          if ((((v.s[i] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) != 0) {
#pragma unroll
            for (int y = 0; y < 4; ++y)
              if (((v.s[i] >> (8 * y)) & 0x7Fu) == 0x7Fu) v.s[i] &= ~(0xFFu << (8 * y));
            nan_flag = 1;
          }
        }
        write(v, sv + st * T::kHalf);
        __syncwarp();
        if (lane == 0) mbar_arrive(v_full + st);
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
      regs_down<kRegsMma>();
      // (the whole warp walks and waits, one lane issues)
      if (warp == 12) {
        constexpr uint32_t id_s = idesc_f16(128, 128, 0), id_o = idesc_f16(128, HD, 1);
        const uint64_t qd = sdesc_k_sw128(smem), kd = sdesc_k_sw128(smem + 2 * T::kHalf);
        const uint64_t vd = sdesc_mn_sw128(smem_u32(smem) + (2 + S) * T::kHalf, 16384);
        uint32_t q_seen[2] = {0, 0}, p_seen[2] = {0, 0};
        int st_k = 0, st_v = 0;
        uint32_t ph_k = 0, ph_v = 0;
        bool ok = true;
        if (p.stall_probe) ok = warp_wait(never, 0);   // the expiry path under test
        auto issue_s = [&](int half) {
          const uint64_t a = qd + (uint64_t)((half * T::kHalf) >> 4), b = kd + (uint64_t)((st_k * T::kHalf) >> 4);
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < HD / 16; ++k)          // (the kind::f16 MMA; the descriptor says f16)
              tc_mma_bf16(tmem + half * 128, a + ((k >> 2) * 1024 + (k & 3) * 2), b + ((k >> 2) * 1024 + (k & 3) * 2),
                          id_s, k ? 1u : 0u);
            tc_commit(s_ready + half);
          }
          __syncwarp();
        };
        auto issue_pv = [&](int half, bool first) {
          const uint64_t b = vd + (uint64_t)((st_v * T::kHalf) >> 4);
          const uint32_t d = tmem + T::kO + half * HD, a = tmem + half * 128, acc = first ? 0u : 1u;
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < 8; ++k) tc_mma_f16_ts(d, a + k * 8, b + k * 128, id_o, k ? 1u : acc);
          }
          __syncwarp();
        };
        auto commit = [&](uint64_t *bar) {
          if (elect_one()) tc_commit(bar);
          __syncwarp();
        };
        if (ok) do {
          const KvSeq s = kv_seq(p, w.it.x);
          const bool two = (int64_t)s.qn * p.group - (int64_t)w.it.y * kRowsTile > 128;
          if (!(ok = warp_wait(k_full + st_k, ph_k))) break;
          if (!(ok = warp_wait(q_ready, q_seen[0]++ & 1))) break;
          tc_fence_after();
          issue_s(0);
          if (two) {
            if (!(ok = warp_wait(q_ready + 1, q_seen[1]++ & 1))) break;
            tc_fence_after();
            issue_s(1);
          }
          commit(k_empty + st_k);
          if (++st_k == S) {
            st_k = 0;
            ph_k ^= 1;
          }
          for (int j = w.j0; j < w.j1; ++j) {
            const bool more = j + 1 < w.j1;
            if (!(ok = warp_wait(v_full + st_v, ph_v))) break;
            if (!(ok = warp_wait(p_ready, p_seen[0]++ & 1))) break;
            tc_fence_after();
            issue_pv(0, j == w.j0);
            if (more) {
              if (!(ok = warp_wait(k_full + st_k, ph_k))) break;
              tc_fence_after();
              issue_s(0);
            } else {
              commit(o_full);
            }
            if (two) {
              if (!(ok = warp_wait(p_ready + 1, p_seen[1]++ & 1))) break;
              tc_fence_after();
              issue_pv(1, j == w.j0);
              if (more)
                issue_s(1);
              else
                commit(o_full + 1);
            }
            commit(v_empty + st_v);
            if (++st_v == S) {
              st_v = 0;
              ph_v ^= 1;
            }
            if (more) {
              commit(k_empty + st_k);
              if (++st_k == S) {
                st_k = 0;
                ph_k ^= 1;
              }
            }
          }
          if (!ok) break;
        } while (w.next(p));
        // every MMA issued here completes before tensor memory is freed
        commit(drain);
        mbar_wait(drain, 0, kKvDrainNs);
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
// rows); the border right behind a segment's first span stands for it.
template <int HD>
__global__ void __launch_bounds__(256) k_kv_join(const KvAttnParams p, int ctas) {
  constexpr int kV = HD / 32;
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int count = *p.item_count;
  const int64_t total = count > 0 ? p.item_prefix[count] * p.kv_heads : 0;
  const int64_t spans = min((int64_t)ctas, total), c = blockIdx.x + 1;
  if (c >= spans) return;
  const int64_t u = pr_start(c, total, spans);
  const int item = find_item(p.item_prefix, count, u / p.kv_heads);
  const int4 it = __ldg(p.items + item);
  const int64_t base = p.item_prefix[item] * p.kv_heads;
  const int h = (int)((u - base) / it.w);
  const int64_t first = base + (int64_t)h * it.w;
  if (first == u || pr_owner(first, total, spans) != c - 1) return;
  const int64_t c0 = c - 1, c1 = pr_owner(first + it.w - 1, total, spans);
  const KvSeq s = kv_seq(p, it.x);
  const int64_t rows = min((int64_t)s.qn * p.group - (int64_t)it.y * kRowsTile, (int64_t)kRowsTile);
  const int first_slot = pr_start(c0, total, spans) < first ? 1 : 0;
  for (int r = blockIdx.y * 8 + warp; r < rows; r += 8 * gridDim.y) {
    float m = -CUDART_INF_F, l = 0.0f, o[kV];
#pragma unroll
    for (int v = 0; v < kV; ++v) o[v] = 0.0f;
    for (int64_t x = c0; x <= c1; ++x) {
      const int64_t prow = (2 * x + (x == c0 ? first_slot : 0)) * kRowsTile + r;
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
      p.lse[(int64_t)(s.q0 + tok) * p.kv_heads * p.group + head] = (m + __log2f(l)) * CUDART_LN2_F;
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
