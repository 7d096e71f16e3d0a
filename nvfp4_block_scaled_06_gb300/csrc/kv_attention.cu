// kv_attention.cu -- attention of few query rows over the pages of the NVFP4
// cache: decoding steps, drafted tokens, short chunks.
//
// Per sequence and key-value head the rows are (new token, query head of the
// group): up to 8 NT of them, over keys j of the sequence
//   s_rj = scale (q_r . K_j),  o_r = sum_j exp(s_rj - m_r) V_j / sum_j exp(s_rj - m_r)
// in one pass with a running maximum m and sum.
//
// Bound: HBM, 2 x 0.5625 B per key and channel, if what a key costs in
// instructions stays below.  So every step feeds the f16 MMA from registers, as
// the packed rows lie in memory: a lane's 16 (or 8) code bytes of a row are
// exactly its share of the A operand K[16 keys][channels] (the contraction's
// order is free, Q is permuted to match), and its 8 (or 4) bytes of four keys,
// two keys' nibbles merged into one byte before the conversion, its share of the
// A operand V^T[channels][16 keys].  E2M1 x E4M3 has six significant bits and is
// exact in f16; q is scaled by a power of two per row, which keeps bf16's 8 bits
// down to 2^-28 of the row's maximum.  The scores' transpose S^T[keys][rows] is
// in registers already; one 8x8 transpose per eight keys makes it P's operand.
// P is rounded to f16 (half a step is 2^-11, an eighth of a bf16 result's), sums and
// accumulators are fp32.
//
// The reference m is 7 (in units of log2) below the row's maximum and is raised
// only when a score exceeds it by more than 15: P stays below 2^15, keys count
// down to 2^-32 of the maximum (f16 ends at 2^-25), and the usual step needs no
// reduction over lanes and no rescaling.
//
// Work: a line of items, cut into equal spans, one per CTA.  An item is a
// (sequence, head) with its 32-key units, which the span's warps take in turn and
// whose (o, m, l) they join in shared memory; items that lie in several spans
// leave one partial result per span, which a second kernel sums in order.  Where
// sequences are short against a span an item is four heads of one, a warp each,
// with nothing to join.  A warp's ring of asynchronous copies runs on over the
// items' borders.
//
// Measured (calls, cold L2): 4 x 131072 keys of 8 heads 123 us, 4.9 TB/s (6 in its
// steady state, 7 us of start); 32 ragged contexts up to 8192 36 us; 256 up to
// 1024 of 16 heads of 64 54 us; 16 x 5 drafted tokens over up to 16384 43 us.  26 instructions per key and head at head_dim 128
// with 8 rows, half of the issue slots: between HBM and the cores, where contexts
// are short the start's latency.
#include <math_constants.h>

#include <type_traits>

#include "internal.h"
#include "kv.cuh"
#include "ptx.cuh"

namespace nvfp4 {

namespace {

constexpr int kWarps = 4;
constexpr int kMaxEntries = 256;    // prefix entries held in shared memory
constexpr int kKeys = 32;           // of a unit: two 16-key tiles of the MMA, each in one page
// What an item costs beside its units, in units (2 or 4: slower for 256 short
// sequences, nothing gained on long ones).
constexpr int kOver = 8;
// Units of a sequence whose heads may go to one warp each.  Beyond, and where four
// heads are more than a span, the warps share a head: 256 sequences up to 1024 keys
// took 57 us with the rule (54 since) and 64 to 72 with the bound at a half or a
// quarter of a span, 256 of 16 keys 19 us and 41 with shared heads.  16, 32, 64 and 128 as
// the most, us: 256 sequences of 2048 keys of 16 heads of 64 172, 172, 186, 186; 512 of them
// 333, 333, 363, 366; 512 up to 4096 267, 271, 295, 311; 1024 up to 2048 270, 280, 266, 267;
// of 8 heads of 128 1024 up to 1024 keys 167, 142, 144, 143, up to 2048 214, 264, 247, 245.
constexpr int kSoloMost = 32;
constexpr int kSumWarps = 8;        // of a block that adds up partial results
constexpr float kLift = 7.0f;       // log2 of the numerator at the maximum
constexpr float kRaise = kLift + 8.0f;   // a score further above the reference raises it

template <int HD, int NT>
struct Few {
  static constexpr int kStages = 3;
  static constexpr int kRows = 8 * NT;
  static constexpr int kCodes = kKeys * HD / 2;           // a unit's codes of K (or V)
  static constexpr int kSf = kKeys * HD / 16;             // and its scales
  static constexpr int kStage = 2 * (kCodes + kSf);
  static constexpr int kCtas = kv_few_ctas(HD, NT);       // per SM
  static constexpr int kPitch = HD + 4;                   // floats of a row of the warps' results
  static constexpr size_t kRing = (size_t)kWarps * kStages * kStage;
  static constexpr size_t kSmem = kRing + (size_t)kWarps * kRows * kPitch * 4;
};

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// Sequence b: first unit, units per head (0: no rows, or more than this kernel
// takes), rows per head.
struct Seg {
  KvSeq s;
  int u0, units, rows;
};
__device__ __forceinline__ Seg seg_of(const KvAttnParams &p, int b) {
  Seg g;
  g.s = kv_seq(p, b);
  const int64_t rows = (int64_t)g.s.qn * p.group;
  g.rows = rows > p.few_rows ? 0 : (int)rows;
  g.u0 = g.s.lo / kKeys;
  g.units = g.rows > 0 ? max(1, (int)(((int64_t)g.s.hi + kKeys - 1) / kKeys) - g.u0) : 0;
  return g;
}

// The line's rule: with `solo` units or fewer a sequence's items are four heads
// each and are not cut (they are the span's that their first place lies in).
struct Line {
  int solo;
  int64_t begin, end;         // this span's places
  __device__ __forceinline__ bool is_solo(const Seg &g) const { return g.units <= solo; }
  __device__ __forceinline__ int items(const KvAttnParams &p, const Seg &g) const {
    return g.units == 0 ? 0 : is_solo(g) ? (p.kv_heads + kWarps - 1) / kWarps : p.kv_heads;
  }
  __device__ __forceinline__ int places(const Seg &g) const {      // of an item
    return (is_solo(g) ? kWarps * g.units : g.units) + kOver;
  }
};

// An item of the span and this warp's units of it.
struct Cursor {
  int b, item;
  Seg g;
  int64_t at;                 // the item's first place
  int h, u, end, step;        // head; units u, u + step ... below end
  int j0, j1;                 // the span's units of the item (all warps')
  bool solo;
  __device__ __forceinline__ void open(const KvAttnParams &p, const Line &l, int warp) {
    solo = l.is_solo(g);
    if (solo) {
      h = item * kWarps + warp;
      const bool mine = at >= l.begin && at < l.end && h < p.kv_heads;
      j0 = u = 0;
      j1 = end = mine ? g.units : 0;
      step = 1;
    } else {
      h = item;
      j0 = (int)max(l.begin - at - kOver, (int64_t)0);
      j1 = (int)max(min(l.end - at - kOver, (int64_t)g.units), (int64_t)0);
      u = j0 + warp;
      end = j1;
      step = kWarps;
    }
  }
  // On to the span's next item; false past the last.
  __device__ __forceinline__ bool next(const KvAttnParams &p, const Line &l, int warp) {
    at += l.places(g);
    if (at >= l.end) return false;
    if (++item == l.items(p, g)) {
      item = 0;
      do {
        if (++b >= p.seqs) return false;
        g = seg_of(p, b);
      } while (g.units == 0);
    }
    open(p, l, warp);
    return true;
  }
};

template <int HD, int NT>
__global__ void __launch_bounds__(kWarps * 32, Few<HD, NT>::kCtas) k_kv_few(const KvAttnParams p) {
  using F = Few<HD, NT>;
  constexpr int S = F::kStages;
  constexpr int kKw = HD / 32;        // code words of a key a lane takes (eight channels each)
  constexpr int kVw = HD / 64;        // code words of a key a lane takes of V
  constexpr int kMt = HD / 16;        // 16-channel tiles of O^T
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int64_t pre[kMaxEntries + 1];
  __shared__ int64_t wsum[2][kWarps];
  __shared__ int limits[kWarps][S];
  __shared__ float2 warp_ml[kWarps][F::kRows];
  float *warp_o = reinterpret_cast<float *>(smem + F::kRing);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  griddep_launch_dependents();
  griddep_wait();

  // All units, then the places before each entry of `per` sequences, by scans over the block.
  const int per = (p.seqs + kMaxEntries - 1) / kMaxEntries;
  const int entries = (p.seqs + per - 1) / per;
  const int each = (entries + kWarps * 32 - 1) / (kWarps * 32);   // entries of a thread
  const int b0 = min(tid * each * per, p.seqs), b1 = min(b0 + each * per, p.seqs);
  Line line;
  int64_t total;
  {
    // (passes over the same loop, for little code: what runs once waits for the instruction cache)
    int64_t units = 0, sum = 0, base = 0;
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
#pragma unroll 1
      for (int b = b0; b < b1; ++b) {
        const Seg g2 = seg_of(p, b);
        if (pass == 0) {
          units += g2.units;
        } else {
          if (pass == 2 && (per == 1 || b % per == 0)) pre[per == 1 ? b : b / per] = base;
          const int64_t places = (int64_t)line.items(p, g2) * line.places(g2);
          sum += places;
          base += places;
        }
      }
      if (pass == 0) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) units += __shfl_xor_sync(0xffffffffu, units, o);
        if (lane == 0) wsum[0][warp] = units;
        __syncthreads();
        units = 0;
        for (int w = 0; w < kWarps; ++w) units += wsum[0][w];
        // four heads of a sequence are at most a span of the units
        line.solo = p.kv_heads < kWarps
                        ? 0
                        : (int)min(kv_div(units * p.kv_heads, (int64_t)gridDim.x * kWarps), (int64_t)kSoloMost);
      } else if (pass == 1) {
        int64_t scan = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int64_t v = __shfl_up_sync(0xffffffffu, scan, o);
          if (lane >= o) scan += v;
        }
        if (lane == 31) wsum[1][warp] = scan;
        __syncthreads();
        base = scan - sum;
        total = 0;
        for (int w = 0; w < kWarps; ++w) {
          if (w < warp) base += wsum[1][w];
          total += wsum[1][w];
        }
      }
    }
    __syncthreads();
  }

  // (a warp has a unit at least: spans of a place each take 1 us more for the sum of one sequence's 1021 keys)
  const KvCut cut(total, min((int64_t)gridDim.x, max(total / kWarps, (int64_t)1)));
  const int64_t span = blockIdx.x;
  if (span >= cut.spans) {
    if (tid == 0) p.few_borders[span] = make_int4(-1, 0, 0, 0);
    return;
  }
  line.begin = cut.start(span);
  line.end = cut.start(span + 1);

  Cursor cur;                                       // the item at hand
  {
    int lo = 0, hi = entries;                       // the last entry that starts at or before the span
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (pre[mid] <= line.begin) lo = mid; else hi = mid;
    }
    cur.at = pre[lo];
    cur.b = lo * per;
    int places;
    for (;; ++cur.b) {                              // (ends before p.seqs: the span starts before the line's end)
      cur.g = seg_of(p, cur.b);
      places = line.places(cur.g);
      const int64_t n = (int64_t)line.items(p, cur.g) * places;
      if (line.begin < cur.at + n) break;
      cur.at += n;
    }
    cur.item = (int)kv_div(line.begin - cur.at, places);
    cur.at += (int64_t)cur.item * places;
    cur.open(p, line, warp);
    // the first border inside a cut item stands for it in the summing kernel
    if (tid == 0) {
      const int64_t c0 = cut.owner(cur.at + kOver);
      p.few_borders[span] = make_int4(!cur.solo && cur.j0 > 0 && c0 == span - 1 ? cur.b : -1, cur.h,
                                      (int)cut.owner(cur.at + places - 1), cut.start(c0) < cur.at ? 1 : 0);
    }
  }

  // An item's rows of q as they are, this lane's: row 8 nt + g, HD / 4 channels from t * HD / 4 on.
  uint32_t xq[NT][HD / 8];
  float gsc;
  auto ask_q = [&](const Cursor &c) {
    gsc = p.scale_log2 * p.gk[min(c.h, p.kv_heads - 1)];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = nt * 8 + g, tok = r / p.group, head = c.h * p.group + r % p.group;
      const uint4 *src = reinterpret_cast<const uint4 *>(p.q + (int64_t)(c.g.s.q0 + tok) * p.q_ld +
                                                         (int64_t)head * p.q_head_ld + t * (HD / 4));
#pragma unroll
      for (int v = 0; v < HD / 32; ++v) {
        const uint4 y = r < c.g.rows && c.j0 < c.j1 ? __ldg(src + v) : make_uint4(0, 0, 0, 0);
        xq[nt][4 * v] = y.x; xq[nt][4 * v + 1] = y.y; xq[nt][4 * v + 2] = y.z; xq[nt][4 * v + 3] = y.w;
      }
    }
  };
  ask_q(cur);

  uint8_t *ring = smem + (size_t)warp * S * F::kStage;
  const uint32_t ring_u = smem_u32(ring);
  int ids = 0, ids_b = -1, ids_at = 0;              // this lane's entry of 32 of the page table
  const int page_mask = (1 << p.page_shift) - 1;

  Cursor ahead = cur;                               // the copies' place
  bool more = true;
  auto settle = [&] {                               // on to this warp's next unit, where it has none left here
    while (more && ahead.u >= ahead.end) more = ahead.next(p, line, warp);
  };
  // Copies of the unit at `ahead` into a stage; keys outside [0, n) and pages
  // outside the cache are zero-filled and left out by their limits.  (Kept to
  // few instructions: address arithmetic once took half of a unit's time.)
  const uint8_t *kc0 = p.k_codes + lane * 16, *vc0 = p.v_codes + lane * 16;
  constexpr int kR = F::kSf / 16;                   // 16-byte runs of a unit's K scales: lanes 0 .. kR - 1, V's follow
  const uint8_t *sf0 = (lane < kR ? p.k_sf : p.v_sf) + lane % kR * 16;
  // The keys from `key` on, kN of them, all in one page: stage bytes at `dst`, runs `part` of kParts of the unit.
  auto copy_keys = [&](int key, uint32_t dst, auto parts, int part) {
    constexpr int kParts = decltype(parts)::value, kN = kKeys / kParts, kC = F::kCodes / 512 / kParts;
    const int page = key >> p.page_shift;
    if (ids_b != ahead.b || (uint32_t)(page - ids_at) >= 32u) {
      ids_b = ahead.b;
      ids_at = page & ~31;
      ids = ids_at + lane < p.max_pages ? __ldg(p.table + (int64_t)ids_b * p.table_ld + ids_at + lane) : -1;
    }
    const int id = __shfl_sync(0xffffffffu, ids, page & 31);
    const bool in = key < ahead.g.s.n && (uint32_t)id < (uint32_t)p.num_pages;
    const int row = (ahead.h << p.page_shift) + (key & page_mask);
    const int64_t oc = in ? id * p.codes_stride + row * (HD / 2) : 0;
    const int64_t os = in ? id * p.sf_stride + row * (HD / 16) : 0;
    const uint32_t bytes = in ? 16u : 0u, at = dst + part * (F::kCodes / kParts);
#pragma unroll
    for (int i = 0; i < kC; ++i) {
      cp_async_16(at + i * 512, kc0 + oc + i * 512, bytes);
      cp_async_16(at + F::kCodes + i * 512, vc0 + oc + i * 512, bytes);
    }
    // (a part's scales are the lanes' whose runs lie in it)
    if (lane < 2 * kR && lane % kR / (kR / kParts) == part)
      cp_async_16(dst + 2 * F::kCodes, sf0 + os - part * (kR / kParts) * 16, bytes);
    return in ? min(kN, ahead.g.s.n - key) : 0;
  };
  auto copy_unit = [&](int stage) {
    const int key = (ahead.g.u0 + ahead.u) * kKeys;
    const uint32_t dst = ring_u + stage * F::kStage + lane * 16;
    int l0, l1;
    if (p.page_shift >= 5) {
      const int l = copy_keys(key, dst, std::integral_constant<int, 1>(), 0);
      l0 = min(l, 16);
      l1 = l - l0;
    } else {
      l0 = copy_keys(key, dst, std::integral_constant<int, 2>(), 0);
      l1 = copy_keys(key + 16, dst, std::integral_constant<int, 2>(), 1);
    }
    if (lane == 0) limits[warp][stage] = l0 | l1 << 8;
  };
  auto fetch = [&](int stage) {
    settle();
    if (more) {
      copy_unit(stage);
      ahead.u += ahead.step;
    }
    cp_async_commit();
  };

#pragma unroll 1
  for (int i = 0; i < S - 1; ++i) fetch(i);

  uint32_t qf[NT][kMt][2];
  float sc[NT][2], m[NT][2], l[NT][2], o[kMt][NT][4];
  int see_lo[NT][2], see_hi[NT][2];                 // keys [see_lo, see_hi) of this lane's rows (8 nt + 2 t, + 1)
  int stage = 0, fill = S - 1;

#pragma unroll 1
  while (true) {
    // --------------------------------------------------------- an item's rows --
    const int rows = cur.g.rows;
    int all_lo = 0, all_hi = 0x7FFFFFFF;            // keys that every row sees
    {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        uint32_t (&x)[HD / 8] = xq[nt];
        uint32_t m2 = 0;
        // the order of |x| is that of its bits, infinities and NaNs last
#pragma unroll
        for (int v = 0; v < HD / 8; ++v) m2 = __vmaxu2(m2, x[v] & 0x7FFF7FFFu);
        m2 = __vmaxu2(m2, __shfl_xor_sync(0xffffffffu, m2, 1));
        m2 = __vmaxu2(m2, __shfl_xor_sync(0xffffffffu, m2, 2));
        const int e = (int)(max(m2 & 0xFFFFu, m2 >> 16) >> 7);
        // a power of two that brings the row's maximum to [2^13, 2^14); 1 for rows with an infinity or a NaN; at most
        // 2^126, which makes f16 numbers of all that bf16 holds below 2^-113
        const int up = e == 255 ? 127 : min(267 - e, 253);
        const float mul = __uint_as_float((uint32_t)up << 23);
        const float back = __uint_as_float((uint32_t)(254 - up) << 23) * gsc;
#pragma unroll
        for (int j = 0; j < kMt; ++j)
#pragma unroll
          for (int k = 0; k < 2; ++k)
            qf[nt][j][k] = pack_h2(bf16lo(x[2 * j + k]) * mul, bf16hi(x[2 * j + k]) * mul);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          // row 8 nt + 2 t + k is held by the lanes of g = 2 t + k
          sc[nt][k] = __shfl_sync(0xffffffffu, back, (2 * t + k) * 4);
          const int r2 = nt * 8 + 2 * t + k;
          const int64_t pos = (int64_t)cur.g.s.n - cur.g.s.qt + r2 / p.group;
          see_hi[nt][k] = p.causal ? (int)max((int64_t)0, pos + 1) : cur.g.s.n;
          see_lo[nt][k] = p.window > 0 ? (int)max((int64_t)0, pos + 1 - p.window) : 0;
          if (r2 < rows) {
            all_lo = max(all_lo, see_lo[nt][k]);
            all_hi = min(all_hi, see_hi[nt][k]);
          }
          m[nt][k] = -CUDART_INF_F;
          l[nt][k] = 0.0f;
        }
#pragma unroll
        for (int mt = 0; mt < kMt; ++mt)
#pragma unroll
          for (int k = 0; k < 4; ++k) o[mt][nt][k] = 0.0f;
      }
#pragma unroll
      for (int x = 1; x < 4; x <<= 1) {
        all_lo = max(all_lo, __shfl_xor_sync(0xffffffffu, all_lo, x));
        all_hi = min(all_hi, __shfl_xor_sync(0xffffffffu, all_hi, x));
      }
    }

    // -------------------------------------------------------- its units, in turn --
#pragma unroll 1
    for (int u = cur.u; u < cur.end; u += cur.step) {
      fetch(fill);
      cp_async_wait<S - 1>();
      __syncwarp();

      const uint8_t *st = ring + stage * F::kStage;
      const int limit0 = limits[warp][stage] & 255, limit1 = limits[warp][stage] >> 8;
      const int key = (cur.g.u0 + u) * kKeys;
      const bool whole = limit0 + limit1 == kKeys && key >= all_lo && key + kKeys <= all_hi;

      // S^T = K Q^T: keys g and g + 8 of both tiles
      float s[2][NT][4];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float s2[NT][4];                            // every other step's sum: half the chain
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < 4; ++k) s[i][nt][k] = s2[nt][k] = 0.0f;
        uint32_t w[2][kKw], sf[2][2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int j = 16 * i + 8 * r + g;
          const uint8_t *row = st + j * (HD / 2) + t * (HD / 8);
          const uint8_t *srow = st + 2 * F::kCodes + j * (HD / 16);
          if constexpr (HD == 128) {
            const uint4 x = *reinterpret_cast<const uint4 *>(row);
            w[r][0] = x.x; w[r][1] = x.y; w[r][2] = x.z; w[r][3] = x.w;
            const uint32_t h2 = e4m3x2_to_h2(*reinterpret_cast<const uint16_t *>(srow + 2 * t));
            sf[r][0] = __byte_perm(h2, h2, 0x1010);
            sf[r][1] = __byte_perm(h2, h2, 0x3232);
          } else {
            const uint2 x = *reinterpret_cast<const uint2 *>(row);
            w[r][0] = x.x; w[r][1] = x.y;
            const uint32_t h2 = e4m3x2_to_h2(srow[t]);
            sf[r][0] = sf[r][1] = __byte_perm(h2, h2, 0x1010);
          }
        }
#pragma unroll
        for (int j = 0; j < kKw; ++j) {
          uint32_t a[2][4];
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            e2m1x8_to_h2(w[r][j], a[r]);
#pragma unroll
            for (int k = 0; k < 4; ++k) a[r][k] = hmul2(a[r][k], sf[r][HD == 128 ? j >> 1 : 0]);
          }
#pragma unroll
          for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma_f16(k ? s2[nt] : s[i][nt], a[0][2 * k], a[1][2 * k], a[0][2 * k + 1], a[1][2 * k + 1],
                      qf[nt][2 * j + k][0], qf[nt][2 * j + k][1]);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < 4; ++k) s[i][nt][k] += s2[nt][k];
      }

#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < 4; ++k) s[i][nt][k] *= sc[nt][k & 1];
      if (!whole) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int j = g + (k >> 1) * 8, at = key + 16 * i + j;
              const bool out = (j >= (i ? limit1 : limit0)) | (at < see_lo[nt][k & 1]) | (at >= see_hi[nt][k & 1]);
              s[i][nt][k] = out ? -CUDART_INF_F : s[i][nt][k];
            }
      }
      bool raise = false;
      float top[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          top[nt][k] = fmaxf(fmaxf(s[0][nt][k], s[0][nt][k + 2]), fmaxf(s[1][nt][k], s[1][nt][k + 2]));
          raise |= top[nt][k] - m[nt][k] > kRaise;     // (near m exact, as m + kRaise is not from 2^24 on)
        }
      if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            float x = top[nt][k];
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
            const float m2 = fmaxf(m[nt][k], x - kLift);
            const float f = m2 == m[nt][k] ? 1.0f : ex2(m[nt][k] - m2);
            m[nt][k] = m2;
            l[nt][k] *= f;
#pragma unroll
            for (int mt = 0; mt < kMt; ++mt) {
              o[mt][nt][k] *= f;
              o[mt][nt][k + 2] *= f;
            }
          }
      }
      uint32_t pf[2][NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float ref[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) ref[k] = m[nt][k] == -CUDART_INF_F ? 0.0f : m[nt][k];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            s[i][nt][k] = ex2(s[i][nt][k] - ref[k & 1]);
            l[nt][k & 1] += s[i][nt][k];
          }
          pf[i][nt][0] = transpose8(pack_h2(s[i][nt][0], s[i][nt][1]));
          pf[i][nt][1] = transpose8(pack_h2(s[i][nt][2], s[i][nt][3]));
        }
      }

      // O^T += V^T P^T: keys 2 t, 2 t + 1 and those + 8 of both tiles, channels g * HD / 8 ...
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint32_t w[4][kVw], sf[4];
        const uint8_t *scales = st + 2 * F::kCodes + F::kSf + (HD == 128 ? g : g >> 1);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int j = 16 * i + 2 * t + (r & 1) + (r >> 1) * 8;
          const uint8_t *row = st + F::kCodes + j * (HD / 2) + g * (HD / 16);
          if constexpr (HD == 128) {
            const uint2 x = *reinterpret_cast<const uint2 *>(row);
            w[r][0] = x.x; w[r][1] = x.y;
          } else {
            w[r][0] = *reinterpret_cast<const uint32_t *>(row);
          }
          sf[r] = scales[j * (HD / 16)];
        }
        if (!whole) {
          // A key with a NaN scale reaches the rows that see it, and no other: 0 * NaN stays out of the sums.
          bool nan = false;
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const bool bad = (sf[r] & 0x7Fu) == 0x7Fu;
            if (bad) sf[r] = 0;
            nan |= bad;
          }
          if (__any_sync(0xffffffffu, nan)) {
            for (int j = 0; j < (i ? limit1 : limit0); ++j) {
              const uint32_t b = scales[(16 * i + j) * (HD / 16)];
              if ((b & 0x7Fu) != 0x7Fu) continue;
              const int at = key + 16 * i + j;
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int k = 0; k < 2; ++k)
                  if (at >= see_lo[nt][k] && at < see_hi[nt][k]) {
#pragma unroll
                    for (int mt = 0; mt < kMt; ++mt) o[mt][nt][k] = o[mt][nt][k + 2] = CUDART_NAN_F;
                  }
            }
          }
        }
        const uint32_t s0 = e4m3x2_to_h2(sf[0] | sf[1] << 8), s1 = e4m3x2_to_h2(sf[2] | sf[3] << 8);
#pragma unroll
        for (int j = 0; j < kVw; ++j) {
          uint32_t a[4][4];   // even and odd channels of keys (2 t, 2 t + 1), then of those + 8
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const uint32_t x = w[2 * r][j], y = w[2 * r + 1][j];
            e2m1x8_to_h2((x & 0x0F0F0F0Fu) | ((y << 4) & 0xF0F0F0F0u), a[2 * r]);
            e2m1x8_to_h2(((x >> 4) & 0x0F0F0F0Fu) | (y & 0xF0F0F0F0u), a[2 * r + 1]);
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t a0 = hmul2(a[0][k], s0), a1 = hmul2(a[1][k], s0), a2 = hmul2(a[2][k], s1),
                           a3 = hmul2(a[3][k], s1);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma_f16(o[j * 4 + k][nt], a0, a1, a2, a3, pf[i][nt][0], pf[i][nt][1]);
          }
        }
      }
      __syncwarp();                                 // the stage is free
      stage = stage + 1 == S ? 0 : stage + 1;
      fill = fill + 1 == S ? 0 : fill + 1;
    }

    // the next item's rows on their way, meanwhile
    Cursor nxt = cur;
    const bool another = nxt.next(p, line, warp);
    if (NT == 1 && another) ask_q(nxt);              // (more rows have no registers for it)
    if (cur.j0 >= cur.j1) {
      // (nothing of this item for this span, or for this warp)
    } else if (cur.solo) {
      // ------------------------------------------------------- a warp's own head --
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float sum_l = l[nt][k];
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) sum_l += __shfl_xor_sync(0xffffffffu, sum_l, d);
          const int r = nt * 8 + 2 * t + k;
          if (r >= rows) continue;
          const int64_t q = cur.g.s.q0 + r / p.group;
          const int head = cur.h * p.group + r % p.group;
          const float f = sum_l == 0.0f ? 0.0f : p.gv[cur.h] / sum_l;
          uint4 *dst = reinterpret_cast<uint4 *>(p.out + q * p.out_ld + (int64_t)head * p.out_head_ld + g * (HD / 8));
#pragma unroll
          for (int j = 0; j < kVw; ++j)
            dst[j] = make_uint4(pack_bf2(o[4 * j][nt][k] * f, o[4 * j][nt][k + 2] * f),
                                pack_bf2(o[4 * j + 1][nt][k] * f, o[4 * j + 1][nt][k + 2] * f),
                                pack_bf2(o[4 * j + 2][nt][k] * f, o[4 * j + 2][nt][k + 2] * f),
                                pack_bf2(o[4 * j + 3][nt][k] * f, o[4 * j + 3][nt][k + 2] * f));
          if (p.lse && g == 0) p.lse[q * p.kv_heads * p.group + head] = kv_lse(m[nt][k], sum_l);
        }
    } else {
    // --------------------------------------------------- the warps' results, joined --
    __syncthreads();                                // (the last item's have been read)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float sum_l = l[nt][k];
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) sum_l += __shfl_xor_sync(0xffffffffu, sum_l, d);
        const int r = nt * 8 + 2 * t + k;
        if (r >= rows) continue;
        float4 *dst = reinterpret_cast<float4 *>(warp_o + (warp * F::kRows + r) * F::kPitch + g * (HD / 8));
#pragma unroll
        for (int j = 0; j < HD / 32; ++j)
          dst[j] = make_float4(o[2 * j][nt][k], o[2 * j][nt][k + 2], o[2 * j + 1][nt][k], o[2 * j + 1][nt][k + 2]);
        if (g == 0) warp_ml[warp][r] = make_float2(m[nt][k], sum_l);
      }
    __syncthreads();
    const bool full = cur.j0 == 0 && cur.j1 == cur.g.units;
    const int64_t slot = 2 * span + (cur.at > line.begin ? 1 : 0);   // (an item cut at the span's start, at its end)
    for (int i = tid; i < rows * (HD / 8); i += kWarps * 32) {
      const int r = i / (HD / 8), c = i % (HD / 8) * 8;
      float mm = -CUDART_INF_F, ll = 0.0f, y[8];
#pragma unroll
      for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, warp_ml[w][r].x);
      const float ref = mm == -CUDART_INF_F ? 0.0f : mm;
#pragma unroll
      for (int k = 0; k < 8; ++k) y[k] = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float2 ml = warp_ml[w][r];
        const float f = ex2(ml.x - ref);
        ll += ml.y * f;
        const float4 *src = reinterpret_cast<const float4 *>(warp_o + (w * F::kRows + r) * F::kPitch + c);
        const float4 v0 = src[0], v1 = src[1];
        y[0] += v0.x * f; y[1] += v0.y * f; y[2] += v0.z * f; y[3] += v0.w * f;
        y[4] += v1.x * f; y[5] += v1.y * f; y[6] += v1.z * f; y[7] += v1.w * f;
      }
      if (full) {
        const int64_t q = cur.g.s.q0 + r / p.group;
        const int head = cur.h * p.group + r % p.group;
        const float f = ll == 0.0f ? 0.0f : p.gv[cur.h] / ll;
        *reinterpret_cast<uint4 *>(p.out + q * p.out_ld + (int64_t)head * p.out_head_ld + c) =
            make_uint4(pack_bf2(y[0] * f, y[1] * f), pack_bf2(y[2] * f, y[3] * f), pack_bf2(y[4] * f, y[5] * f),
                       pack_bf2(y[6] * f, y[7] * f));
        if (p.lse && c == 0) p.lse[q * p.kv_heads * p.group + head] = kv_lse(mm, ll);
      } else {
        float4 *dst = reinterpret_cast<float4 *>(p.part_o + (slot * F::kRows + r) * HD + c);
        dst[0] = make_float4(y[0], y[1], y[2], y[3]);
        dst[1] = make_float4(y[4], y[5], y[6], y[7]);
        if (c == 0) *reinterpret_cast<float2 *>(p.part_ml + (slot * F::kRows + r) * 2) = make_float2(mm, ll);
      }
    }
    }
    if (!another) break;
    cur = nxt;
    if (NT > 1) ask_q(cur);
  }
  cp_async_wait<0>();
}

// Segments that lie in several spans: block = (border between two spans, rows);
// the border behind a segment's first span stands for it.  A row's partial results
// are added in order by W warps: one, eight results at a time, where items have
// few (256 short sequences 57.5 -> 53 us, 16 x 5 drafted tokens 44 -> 41.5, both with a
// warm L2: most blocks find no border, fewer of them end sooner), or the block's eight (one
// sequence of 131072 keys 44 us, 58 with one warp; 4 of them 123 and 125).
template <int HD, int NT, int W>
__global__ void __launch_bounds__(kSumWarps * 32) k_kv_sum(const KvAttnParams p) {
  static_assert(W == 1 || W == kSumWarps);
  constexpr int kRows = 8 * NT, kV = HD / 32, kBatch = 8;
  __shared__ float sh_o[W > 1 ? kSumWarps : 1][HD];
  __shared__ float2 sh_ml[kSumWarps];
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int r = W > 1 ? blockIdx.y : blockIdx.y * kSumWarps + warp;
  const int4 bd = p.few_borders[blockIdx.x + 1];
  if (bd.x < 0) return;
  const int c0 = blockIdx.x, c1 = bd.z, h = bd.y;
  const KvSeq s = kv_seq(p, bd.x);
  if (r >= s.qn * p.group) return;                  // (the whole block, or a warp that waits for no other)
  auto row_of = [&](int c) { return (2ll * c + (c == c0 ? bd.w : 0)) * kRows + r; };
  float m = -CUDART_INF_F, l = 0.0f, o[kV];
#pragma unroll
  for (int v = 0; v < kV; ++v) o[v] = 0.0f;
  // partial result c of the row
  auto load = [&](int c, float2 &ml, float (&y)[kV]) {
    const int64_t row = row_of(c);
    ml = reinterpret_cast<const float2 *>(p.part_ml)[row];
    const float *src = p.part_o + row * HD + lane * kV;
    if constexpr (kV == 4) {
      const float4 v = *reinterpret_cast<const float4 *>(src);
      y[0] = v.x; y[1] = v.y; y[2] = v.z; y[3] = v.w;
    } else {
      const float2 v = *reinterpret_cast<const float2 *>(src);
      y[0] = v.x; y[1] = v.y;
    }
  };
  if constexpr (W == 1) {
#pragma unroll 1
    for (int c = c0; c <= c1; c += kBatch) {
      float2 ml[kBatch];
      float y[kBatch][kV], top = m;
#pragma unroll
      for (int i = 0; i < kBatch; ++i) load(min(c + i, c1), ml[i], y[i]);
#pragma unroll
      for (int i = 0; i < kBatch; ++i) top = fmaxf(top, ml[i].x);   // (the last one's again at most)
      const float ref = top == -CUDART_INF_F ? 0.0f : top, f0 = ex2(m - ref);
      m = top;
      l *= f0;
#pragma unroll
      for (int v = 0; v < kV; ++v) o[v] *= f0;
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        if (c + i > c1) break;
        const float f = ex2(ml[i].x - ref);
        l += ml[i].y * f;
#pragma unroll
        for (int v = 0; v < kV; ++v) o[v] += y[i][v] * f;
      }
    }
  } else {
    // this warp's: c0 + warp, W apart; their maximum first, so that the rows' loads are independent
    for (int c = c0 + warp + lane * W; c <= c1; c += 32 * W)
      m = fmaxf(m, reinterpret_cast<const float2 *>(p.part_ml)[row_of(c)].x);
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    const float top = m == -CUDART_INF_F ? 0.0f : m;
#pragma unroll 8
    for (int c = c0 + warp; c <= c1; c += W) {
      float2 ml;
      float y[kV];
      load(c, ml, y);
      const float f = ex2(ml.x - top);
      l += ml.y * f;
#pragma unroll
      for (int v = 0; v < kV; ++v) o[v] += y[v] * f;
    }
#pragma unroll
    for (int v = 0; v < kV; ++v) sh_o[warp][lane * kV + v] = o[v];
    if (lane == 0) sh_ml[warp] = make_float2(m, l);
    __syncthreads();
    if (warp != 0) return;
    m = -CUDART_INF_F;
    l = 0.0f;
#pragma unroll
    for (int w = 0; w < W; ++w) m = fmaxf(m, sh_ml[w].x);
    const float ref = m == -CUDART_INF_F ? 0.0f : m;
#pragma unroll
    for (int v = 0; v < kV; ++v) o[v] = 0.0f;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float f = ex2(sh_ml[w].x - ref);
      l += sh_ml[w].y * f;
#pragma unroll
      for (int v = 0; v < kV; ++v) o[v] += sh_o[w][lane * kV + v] * f;
    }
  }
  const int64_t q = s.q0 + r / p.group;
  const int head = h * p.group + r % p.group;
  const float f = l == 0.0f ? 0.0f : p.gv[h] / l;
  __nv_bfloat16 *dst = p.out + q * p.out_ld + (int64_t)head * p.out_head_ld + lane * kV;
  if constexpr (kV == 4)
    *reinterpret_cast<uint2 *>(dst) = make_uint2(pack_bf2(o[0] * f, o[1] * f), pack_bf2(o[2] * f, o[3] * f));
  else
    *reinterpret_cast<uint32_t *>(dst) = pack_bf2(o[0] * f, o[1] * f);
  if (p.lse && lane == 0) p.lse[q * p.kv_heads * p.group + head] = kv_lse(m, l);
}

template <int HD, int NT>
cudaError_t run_few(const KvAttnParams &p, int num_sms, cudaStream_t st) {
  using F = Few<HD, NT>;
  if (cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void *>(k_kv_few<HD, NT>), F::kSmem); e != cudaSuccess)
    return e;
  const int ctas = num_sms * F::kCtas;
  if (cudaError_t e = launch_pdl(k_kv_few<HD, NT>, dim3(ctas), dim3(kWarps * 32), F::kSmem, st, p); e != cudaSuccess)
    return e;
  const int rows = std::min(F::kRows, p.few_rows_most);
  return (int64_t)p.seqs * p.kv_heads * kSumWarps <= ctas
             ? launch_pdl(k_kv_sum<HD, NT, kSumWarps>, dim3(ctas - 1, rows), dim3(kSumWarps * 32), 0, st, p)
             : launch_pdl(k_kv_sum<HD, NT, 1>, dim3(ctas - 1, (rows + kSumWarps - 1) / kSumWarps),
                          dim3(kSumWarps * 32), 0, st, p);
}

}  // namespace

int kv_few_spans(int head_dim, int nt, int num_sms) { return num_sms * kv_few_ctas(head_dim, nt); }

cudaError_t launch_kv_few(const KvAttnParams &p, int head_dim, int nt, int num_sms, cudaStream_t st) {
  if (head_dim == 128)
    return nt == 1   ? run_few<128, 1>(p, num_sms, st)
           : nt == 2 ? run_few<128, 2>(p, num_sms, st)
                     : run_few<128, 3>(p, num_sms, st);
  return nt == 1   ? run_few<64, 1>(p, num_sms, st)
         : nt == 2 ? run_few<64, 2>(p, num_sms, st)
                   : run_few<64, 3>(p, num_sms, st);
}

}  // namespace nvfp4
