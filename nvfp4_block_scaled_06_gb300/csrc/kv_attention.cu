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
// P is rounded to f16 (2^-11 relative, half of what bf16 results keep), sums and
// accumulators are fp32.
//
// The reference m is raised only when a score exceeds it by more than 8 (in
// units of log2): P stays below 2^8, and the usual step needs no reduction
// over lanes and no rescaling.
//
// Work: 16-key units of all (sequence, head) segments in one line, cut into equal
// spans, one per warp; a warp's ring of asynchronous copies runs on
// over segment borders.  Segments that lie in more than one span leave partial
// (o, m, l) per span, which a second kernel sums in order.
#include <math_constants.h>

#include "internal.h"
#include "kv.cuh"
#include "ptx.cuh"

namespace nvfp4 {

namespace {

constexpr int kWarps = 4;
constexpr int kMaxEntries = 1024;   // prefix entries held in shared memory
constexpr float kRaise = 8.0f;

template <int HD, int NT>
struct Few {
  static constexpr int kStages = 5;
  static constexpr int kRows = 8 * NT;
  static constexpr int kCodes = 16 * HD / 2;              // a unit's codes of K (or V)
  static constexpr int kSf = HD;                          // and its scales
  static constexpr int kStage = 2 * (kCodes + kSf);
  static constexpr int kCtas = NT == 1 ? 4 : 2;           // per SM
  static constexpr size_t kSmem = (size_t)kWarps * kStages * kStage;
};

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// The segments of sequence b: first unit, units (0: no rows, or more than this
// kernel takes), rows.
struct Seg {
  KvSeq s;
  int u0, units, rows;
};
__device__ __forceinline__ Seg seg_of(const KvAttnParams &p, int b) {
  Seg g;
  g.s = kv_seq(p, b);
  const int64_t rows = (int64_t)g.s.qn * p.group;
  g.rows = rows > p.few_rows ? 0 : (int)rows;
  g.u0 = g.s.lo >> 4;
  g.units = g.rows > 0 ? max(1, (int)(((int64_t)g.s.hi + 15) >> 4) - g.u0) : 0;
  return g;
}
__device__ __forceinline__ int64_t units_of(const KvAttnParams &p, const Seg &g) {
  return (int64_t)g.units * p.kv_heads;
}

// A position in the line of units.
struct Cursor {
  int b, h, u;         // u: unit within the segment
  Seg g;
};

__device__ __forceinline__ int64_t span_start(int64_t w, int64_t total, int64_t spans) { return w * total / spans; }
__device__ __forceinline__ int64_t span_of(int64_t u, int64_t total, int64_t spans) {
  return ((u + 1) * spans - 1) / total;
}

__device__ __forceinline__ void next_unit(const KvAttnParams &p, Cursor &c) {
  if (++c.u < c.g.units) return;
  c.u = 0;
  if (++c.h < p.kv_heads) return;
  c.h = 0;
  do {
    if (++c.b >= p.seqs) return;
    c.g = seg_of(p, c.b);
  } while (c.g.units == 0);
}

template <int HD, int NT>
__global__ void __launch_bounds__(kWarps * 32, Few<HD, NT>::kCtas) k_kv_few(const KvAttnParams p) {
  using F = Few<HD, NT>;
  constexpr int S = F::kStages;
  constexpr int kKw = HD / 32;        // code words of a key a lane takes (eight channels each)
  constexpr int kVw = HD / 64;        // code words of a key a lane takes of V
  constexpr int kMt = HD / 16;        // 16-channel tiles of O^T
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int64_t pre[kMaxEntries + 1];
  __shared__ int64_t wsum[kWarps];
  __shared__ int limits[kWarps][S];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  griddep_launch_dependents();
  griddep_wait();

  // Units before each entry of `per` sequences, by a scan over the block.
  const int per = (p.seqs + kMaxEntries - 1) / kMaxEntries;
  const int entries = (p.seqs + per - 1) / per;
  const int each = (entries + kWarps * 32 - 1) / (kWarps * 32);   // entries of a thread
  const int e0 = min(tid * each, entries), e1 = min(e0 + each, entries);
  int64_t sum = 0;
  for (int b = e0 * per; b < min(e1 * per, p.seqs); ++b) sum += units_of(p, seg_of(p, b));
  int64_t scan = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, scan, o);
    if (lane >= o) scan += v;
  }
  if (lane == 31) wsum[warp] = scan;
  __syncthreads();
  int64_t base = scan - sum;
  for (int w = 0; w < warp; ++w) base += wsum[w];
  for (int e = e0; e < e1; ++e) {
    pre[e] = base;
    for (int b = e * per; b < min((e + 1) * per, p.seqs); ++b) {
      if (blockIdx.x == 0) p.prefix[b] = base;
      base += units_of(p, seg_of(p, b));
    }
  }
  int64_t total = 0;
  for (int w = 0; w < kWarps; ++w) total += wsum[w];
  if (blockIdx.x == 0 && tid == 0) p.prefix[p.seqs] = total;
  __syncthreads();
  if (total == 0) return;

  const int64_t spans = min((int64_t)gridDim.x * kWarps, total), span = (int64_t)blockIdx.x * kWarps + warp;
  if (span >= spans) return;
  const int64_t u_begin = span_start(span, total, spans), u_end = span_start(span + 1, total, spans);

  Cursor cur;
  {
    int lo = 0, hi = entries;                       // the last entry that starts at or before u_begin
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (pre[mid] <= u_begin) lo = mid; else hi = mid;
    }
    int64_t at = pre[lo];
    cur.b = lo * per;
    for (;; ++cur.b) {                              // (ends before p.seqs: u_begin < total)
      cur.g = seg_of(p, cur.b);
      const int64_t n = units_of(p, cur.g);
      if (u_begin < at + n) break;
      at += n;
    }
    const int64_t r = u_begin - at;
    const int64_t seg = r / cur.g.units;
    cur.u = (int)(r - seg * cur.g.units);
    cur.h = (int)seg;
  }
  Cursor ahead = cur;                               // of the copies

  uint8_t *ring = smem + (size_t)warp * S * F::kStage;
  const uint32_t ring_u = smem_u32(ring);
  int ids = 0, ids_b = -1, ids_at = 0;              // this lane's entry of 32 of the page table

  // Copies of the unit at `ahead` into a stage; keys outside [0, n) and pages
  // outside the cache are zero-filled and left out by their limit.
  auto copy_unit = [&](int stage) {
    const int key = (ahead.g.u0 + ahead.u) << 4, page = key >> p.page_shift;
    if (ids_b != ahead.b || page < ids_at || page >= ids_at + 32) {
      ids_b = ahead.b;
      ids_at = page & ~31;
      ids = ids_at + lane < p.max_pages ? __ldg(p.table + (int64_t)ids_b * p.table_ld + ids_at + lane) : -1;
    }
    const int id = __shfl_sync(0xffffffffu, ids, page - ids_at);
    int limit = min(16, ahead.g.s.n - key);
    if (limit <= 0 || !NVFP4_NOTE(id >= 0 && id < p.num_pages, p.status)) limit = 0;
    const int64_t row = ((int64_t)ahead.h << p.page_shift) + (key & ((1 << p.page_shift) - 1));
    const int64_t oc = limit ? id * p.codes_stride + row * (HD / 2) : 0;
    const int64_t os = limit ? id * p.sf_stride + row * (HD / 16) : 0;
    const uint32_t bytes = limit ? 16u : 0u;
    const uint32_t dst = ring_u + stage * F::kStage;
#pragma unroll
    for (int i = 0; i < F::kCodes / 512; ++i) {
      cp_async_16(dst + (i * 32 + lane) * 16, p.k_codes + oc + (i * 32 + lane) * 16, bytes);
      cp_async_16(dst + F::kCodes + (i * 32 + lane) * 16, p.v_codes + oc + (i * 32 + lane) * 16, bytes);
    }
    if (lane < 2 * (F::kSf / 16)) {
      const bool val = lane >= F::kSf / 16;
      const int i = val ? lane - F::kSf / 16 : lane;
      cp_async_16(dst + 2 * F::kCodes + lane * 16, (val ? p.v_sf : p.k_sf) + os + i * 16, bytes);
    }
    if (lane == 0) limits[warp][stage] = limit;
  };

  const int64_t count = u_end - u_begin;
  int64_t issued = 0;
#pragma unroll 1
  for (; issued < S - 1; ++issued) {
    if (issued < count) {
      copy_unit((int)issued);
      next_unit(p, ahead);
    }
    cp_async_commit();
  }

  uint32_t qf[NT][kMt][2];
  float sc[NT][2], m[NT][2], l[NT][2], o[kMt][NT][4];
  int see_lo[NT][2], see_hi[NT][2];                 // keys [see_lo, see_hi) of this lane's rows (8 nt + 2 t, + 1)
  int all_lo = 0, all_hi = 0;                       // keys that every row of the tile sees
  bool fresh = true;
  int64_t part_slot = 2 * span;
  const int64_t seg_first = u_begin - cur.u;        // the first unit of the segment that the span starts in
  int64_t u = u_begin;
  int stage = 0, fill = S - 1;

#pragma unroll 1
  for (int64_t i = 0; i < count; ++i, ++u) {
    if (fresh) {
      fresh = false;
      const int rows = cur.g.rows;
      const float gk = p.gk[cur.h];
      all_lo = 0;
      all_hi = 0x7FFFFFFF;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float f[2][HD / 8];
        float mx = 0.0f;
        const int r = nt * 8 + g;
        if (r < rows) {
          const int tok = r / p.group, head = cur.h * p.group + r % p.group;
          const uint4 *src = reinterpret_cast<const uint4 *>(p.q + (int64_t)(cur.g.s.q0 + tok) * p.q_ld +
                                                             (int64_t)head * p.q_head_ld + t * (HD / 4));
#pragma unroll
          for (int v = 0; v < HD / 32; ++v) {
            const uint4 x = __ldg(src + v);
            const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              f[0][v * 4 + e] = bf16lo(w[e]);
              f[1][v * 4 + e] = bf16hi(w[e]);
            }
          }
        } else {
#pragma unroll
          for (int e = 0; e < HD / 8; ++e) f[0][e] = f[1][e] = 0.0f;
        }
        // the order of |x| is that of its bits, infinities and NaNs last
        uint32_t top = 0;
#pragma unroll
        for (int e = 0; e < HD / 8; ++e)
          top = max(top, max(__float_as_uint(f[0][e]) & 0x7FFFFFFFu, __float_as_uint(f[1][e]) & 0x7FFFFFFFu));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int e = (int)(top >> 23);
        // a power of two that brings the row's maximum to [2^13, 2^14); 1 for rows with an infinity or a NaN
        const int up = e == 255 ? 127 : min(267 - e, 190);
        const float mul = __uint_as_float((uint32_t)up << 23);
        mx = __uint_as_float((uint32_t)(254 - up) << 23) * (p.scale_log2 * gk);
#pragma unroll
        for (int j = 0; j < kMt; ++j) {
          qf[nt][j][0] = pack_h2(f[0][2 * j] * mul, f[1][2 * j] * mul);
          qf[nt][j][1] = pack_h2(f[0][2 * j + 1] * mul, f[1][2 * j + 1] * mul);
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          // row 8 nt + 2 t + k is held by the lanes of g = 2 t + k
          sc[nt][k] = __shfl_sync(0xffffffffu, mx, (2 * t + k) * 4);
          const int r2 = nt * 8 + 2 * t + k;
          const int tok = r2 / p.group;
          const int64_t pos = (int64_t)cur.g.s.n - cur.g.s.qt + tok;
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

    if (issued < count) {
      copy_unit(fill);
      next_unit(p, ahead);
    }
    ++issued;
    cp_async_commit();
    cp_async_wait<S - 1>();
    __syncwarp();

    const uint8_t *st = ring + stage * F::kStage;
    const int limit = limits[warp][stage];
    const int key = (cur.g.u0 + cur.u) << 4;
    const bool whole = limit == 16 && key >= all_lo && key + 16 <= all_hi;

    // S^T = K Q^T: keys g and g + 8
    float s[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int k = 0; k < 4; ++k) s[nt][k] = 0.0f;
    {
      uint32_t w[2][kKw], sf[2][2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const uint8_t *row = st + (g + 8 * r) * (HD / 2) + t * (HD / 8);
        const uint8_t *srow = st + 2 * F::kCodes + (g + 8 * r) * (HD / 16);
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
            mma_f16(s[nt], a[0][2 * k], a[1][2 * k], a[0][2 * k + 1], a[1][2 * k + 1], qf[nt][2 * j + k][0],
                    qf[nt][2 * j + k][1]);
      }
    }

    bool raise = false;
    float top[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        s[nt][k] *= sc[nt][k & 1];
        if (!whole) {
          const int j = g + (k >> 1) * 8;
          if (j >= limit || key + j < see_lo[nt][k & 1] || key + j >= see_hi[nt][k & 1]) s[nt][k] = -CUDART_INF_F;
        }
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        top[nt][k] = fmaxf(s[nt][k], s[nt][k + 2]);
        raise |= top[nt][k] > m[nt][k] + kRaise;
      }
    }
    if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float x = top[nt][k];
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
          const float m2 = fmaxf(m[nt][k], x);
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
    uint32_t pf[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float ref = m[nt][k & 1] == -CUDART_INF_F ? 0.0f : m[nt][k & 1];
        s[nt][k] = ex2(s[nt][k] - ref);
        l[nt][k & 1] += s[nt][k];
      }
      pf[nt][0] = transpose8(pack_h2(s[nt][0], s[nt][1]));
      pf[nt][1] = transpose8(pack_h2(s[nt][2], s[nt][3]));
    }

    // O^T += V^T P^T: keys 2 t, 2 t + 1 and those + 8, channels g * HD / 8 ...
    {
      uint32_t w[4][kVw], sf[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int j = 2 * t + (r & 1) + (r >> 1) * 8;
        const uint8_t *row = st + F::kCodes + j * (HD / 2) + g * (HD / 16);
        if constexpr (HD == 128) {
          const uint2 x = *reinterpret_cast<const uint2 *>(row);
          w[r][0] = x.x; w[r][1] = x.y;
        } else {
          w[r][0] = *reinterpret_cast<const uint32_t *>(row);
        }
        sf[r] = st[2 * F::kCodes + F::kSf + j * (HD / 16) + (HD == 128 ? g : g >> 1)];
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
          for (int j = 0; j < limit; ++j) {
            const uint32_t b = st[2 * F::kCodes + F::kSf + j * (HD / 16) + (HD == 128 ? g : g >> 1)];
            if ((b & 0x7Fu) != 0x7Fu) continue;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int k = 0; k < 2; ++k)
                if (key + j >= see_lo[nt][k] && key + j < see_hi[nt][k]) {
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
          for (int nt = 0; nt < NT; ++nt) mma_f16(o[j * 4 + k][nt], a0, a1, a2, a3, pf[nt][0], pf[nt][1]);
        }
      }
    }
    __syncwarp();                                   // the stage is free
    stage = stage + 1 == S ? 0 : stage + 1;
    fill = fill + 1 == S ? 0 : fill + 1;

    const bool last = cur.u + 1 == cur.g.units;     // of the segment
    if (last || i + 1 == count) {
      const bool whole_seg = last && (u - cur.u) >= u_begin;
      const int64_t slot = (u - cur.u) == seg_first ? part_slot : part_slot + 1;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float sum_l = l[nt][k];
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) sum_l += __shfl_xor_sync(0xffffffffu, sum_l, d);
          const int r = nt * 8 + 2 * t + k;
          if (r >= cur.g.rows) continue;
          if (whole_seg) {
            const int tok = r / p.group, head = cur.h * p.group + r % p.group;
            const float f = sum_l == 0.0f ? 0.0f : p.gv[cur.h] / sum_l;
            uint4 *dst = reinterpret_cast<uint4 *>(p.out + (int64_t)(cur.g.s.q0 + tok) * p.out_ld +
                                                   (int64_t)head * p.out_head_ld + g * (HD / 8));
#pragma unroll
            for (int j = 0; j < kVw; ++j)
              dst[j] = make_uint4(pack_bf2(o[4 * j][nt][k] * f, o[4 * j][nt][k + 2] * f),
                                  pack_bf2(o[4 * j + 1][nt][k] * f, o[4 * j + 1][nt][k + 2] * f),
                                  pack_bf2(o[4 * j + 2][nt][k] * f, o[4 * j + 2][nt][k + 2] * f),
                                  pack_bf2(o[4 * j + 3][nt][k] * f, o[4 * j + 3][nt][k + 2] * f));
            if (p.lse && g == 0)
              p.lse[(int64_t)(cur.g.s.q0 + tok) * p.kv_heads * p.group + head] =
                  (m[nt][k] + __log2f(sum_l)) * CUDART_LN2_F;
          } else {
            float4 *dst = reinterpret_cast<float4 *>(p.part_o + (slot * F::kRows + r) * HD + g * (HD / 8));
#pragma unroll
            for (int j = 0; j < HD / 32; ++j)
              dst[j] = make_float4(o[2 * j][nt][k], o[2 * j][nt][k + 2], o[2 * j + 1][nt][k], o[2 * j + 1][nt][k + 2]);
            if (g == 0)
              *reinterpret_cast<float2 *>(p.part_ml + (slot * F::kRows + r) * 2) = make_float2(m[nt][k], sum_l);
          }
        }
      if (i + 1 == count) break;
      next_unit(p, cur);
      fresh = true;
    } else {
      ++cur.u;
    }
  }
  cp_async_wait<0>();
}

// Rows of the segments that lie in several spans: block = (segment, row), the
// spans' partial results dealt to its warps in order, one 16-byte (8-byte) run
// of channels per lane.
template <int HD, int NT>
__global__ void __launch_bounds__(256) k_kv_combine(const KvAttnParams p, int max_spans) {
  constexpr int kRows = 8 * NT, kV = HD / 32, kW = 8;
  __shared__ float sh_o[kW][HD];
  __shared__ float sh_m[kW], sh_l[kW];
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int b = blockIdx.x;
  const Seg g = seg_of(p, b);
  if (g.units == 0) return;
  const int64_t total = p.prefix[p.seqs], spans = min((int64_t)max_spans, total);
  for (int x = blockIdx.y; x < p.kv_heads * g.rows; x += gridDim.y) {
    const int r = x % g.rows, h = x / g.rows;
    const int64_t first = p.prefix[b] + (int64_t)h * g.units;
    const int64_t c0 = span_of(first, total, spans), c1 = span_of(first + g.units - 1, total, spans);
    if (c0 == c1) continue;
    float m = -CUDART_INF_F, l = 0.0f, o[kV];
#pragma unroll
    for (int v = 0; v < kV; ++v) o[v] = 0.0f;
    for (int64_t c = c0 + warp; c <= c1; c += kW) {
      const int64_t slot = 2 * c + (c == c0 && span_start(c, total, spans) < first ? 1 : 0);
      const float2 ml = __ldg(reinterpret_cast<const float2 *>(p.part_ml) + slot * kRows + r);
      const float *src = p.part_o + (slot * kRows + r) * HD + lane * kV;
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
    __syncthreads();
#pragma unroll
    for (int v = 0; v < kV; ++v) sh_o[warp][lane * kV + v] = o[v];
    if (lane == 0) {
      sh_m[warp] = m;
      sh_l[warp] = l;
    }
    __syncthreads();
    if (warp != 0) continue;
    float mm = -CUDART_INF_F;
    for (int w = 0; w < kW; ++w) mm = fmaxf(mm, sh_m[w]);
    const float ref = mm == -CUDART_INF_F ? 0.0f : mm;
    float ll = 0.0f;
#pragma unroll
    for (int v = 0; v < kV; ++v) o[v] = 0.0f;
    for (int w = 0; w < kW; ++w) {
      const float f = ex2(sh_m[w] - ref);
      ll += sh_l[w] * f;
#pragma unroll
      for (int v = 0; v < kV; ++v) o[v] += sh_o[w][lane * kV + v] * f;
    }
    const int tok = r / p.group, head = h * p.group + r % p.group;
    const float f = ll == 0.0f ? 0.0f : p.gv[h] / ll;
    __nv_bfloat16 *dst = p.out + (int64_t)(g.s.q0 + tok) * p.out_ld + (int64_t)head * p.out_head_ld + lane * kV;
    if constexpr (kV == 4)
      *reinterpret_cast<uint2 *>(dst) = make_uint2(pack_bf2(o[0] * f, o[1] * f), pack_bf2(o[2] * f, o[3] * f));
    else
      *reinterpret_cast<uint32_t *>(dst) = pack_bf2(o[0] * f, o[1] * f);
    if (p.lse && lane == 0)
      p.lse[(int64_t)(g.s.q0 + tok) * p.kv_heads * p.group + head] = (mm + __log2f(ll)) * CUDART_LN2_F;
  }
}

template <int HD, int NT>
cudaError_t run_few(const KvAttnParams &p, int num_sms, cudaStream_t st) {
  using F = Few<HD, NT>;
  if (cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void *>(k_kv_few<HD, NT>), F::kSmem); e != cudaSuccess)
    return e;
  const int ctas = num_sms * F::kCtas;
  if (cudaError_t e = launch_pdl(k_kv_few<HD, NT>, dim3(ctas), dim3(kWarps * 32), F::kSmem, st, p); e != cudaSuccess)
    return e;
  const int64_t rows = (int64_t)p.kv_heads * F::kRows;
  const int y = (int)std::min<int64_t>(rows, std::max(1, num_sms * 16 / p.seqs));
  return launch_pdl(k_kv_combine<HD, NT>, dim3(p.seqs, y), dim3(256), 0, st, p, ctas * kWarps);
}

}  // namespace

int kv_few_spans(int nt, int num_sms) {
  return num_sms * (nt == 1 ? 4 : 2) * kWarps;
}

cudaError_t launch_kv_few(const KvAttnParams &p, int head_dim, int nt, int num_sms, cudaStream_t st) {
  if (head_dim == 128) return nt == 1 ? run_few<128, 1>(p, num_sms, st) : run_few<128, 2>(p, num_sms, st);
  return nt == 1 ? run_few<64, 1>(p, num_sms, st) : run_few<64, 2>(p, num_sms, st);
}

}  // namespace nvfp4
