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
// Work: 32-key units of all (sequence, head) segments in one line, cut into equal
// spans, one per CTA, whose warps take its units in turn; a warp's ring of
// asynchronous copies runs on over segment borders.  At a segment's end the
// warps' (o, m, l) are joined in shared memory; segments that lie in several spans
// leave one partial result per span, which a second kernel sums in order.
#include <math_constants.h>

#include "internal.h"
#include "kv.cuh"
#include "ptx.cuh"

namespace nvfp4 {

namespace {

constexpr int kWarps = 4;
constexpr int kMaxEntries = 256;    // prefix entries held in shared memory
constexpr int kKeys = 32;           // of a unit: two 16-key tiles of the MMA, each in one page
constexpr float kRaise = 8.0f;

template <int HD, int NT>
struct Few {
  static constexpr int kStages = 3;
  static constexpr int kRows = 8 * NT;
  static constexpr int kCodes = kKeys * HD / 2;           // a unit's codes of K (or V)
  static constexpr int kSf = kKeys * HD / 16;             // and its scales
  static constexpr int kStage = 2 * (kCodes + kSf);
  static constexpr int kCtas = kv_few_ctas(NT);           // per SM
  static constexpr int kPitch = HD + 4;                   // floats of a row of the warps' results
  static constexpr size_t kRing = (size_t)kWarps * kStages * kStage;
  static constexpr size_t kSmem = kRing + (size_t)kWarps * kRows * kPitch * 4;
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
  g.u0 = g.s.lo / kKeys;
  g.units = g.rows > 0 ? max(1, (int)(((int64_t)g.s.hi + kKeys - 1) / kKeys) - g.u0) : 0;
  return g;
}
__device__ __forceinline__ int64_t units_of(const KvAttnParams &p, const Seg &g) {
  return (int64_t)g.units * p.kv_heads;
}

__device__ __forceinline__ int64_t span_start(int64_t w, int64_t total, int64_t spans) { return w * total / spans; }
__device__ __forceinline__ int64_t span_of(int64_t u, int64_t total, int64_t spans) {
  return ((u + 1) * spans - 1) / total;
}

// A position in the line of units: sequence, head, unit of the segment.
struct Cursor {
  int b, h, u;
  Seg g;
  // On to the next segment; false past the last.
  __device__ __forceinline__ bool next(const KvAttnParams &p) {
    if (++h < p.kv_heads) return true;
    h = 0;
    do {
      if (++b >= p.seqs) return false;
      g = seg_of(p, b);
    } while (g.units == 0);
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
  __shared__ int64_t wsum[kWarps];
  __shared__ int limits[kWarps][S][2];
  __shared__ float2 warp_ml[kWarps][F::kRows];
  float *warp_o = reinterpret_cast<float *>(smem + F::kRing);
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
    for (int b = e * per; b < min((e + 1) * per, p.seqs); ++b) base += units_of(p, seg_of(p, b));
  }
  int64_t total = 0;
  for (int w = 0; w < kWarps; ++w) total += wsum[w];
  __syncthreads();

  const int64_t spans = min((int64_t)gridDim.x, total), span = blockIdx.x;
  if (span >= spans) {
    if (tid == 0) p.few_borders[span] = make_int4(-1, 0, 0, 0);
    return;
  }
  const int64_t u_begin = span_start(span, total, spans), u_end = span_start(span + 1, total, spans);

  Cursor cur;                                       // of the segment at hand
  int64_t seg0;                                     // its first unit in the line
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
    cur.h = (int)((u_begin - at) / cur.g.units);
    seg0 = at + (int64_t)cur.h * cur.g.units;
    cur.u = (int)(u_begin - seg0);
  }
  // the first border inside a segment stands for it in the summing kernel
  if (tid == 0) {
    const int64_t c0 = span_of(seg0, total, spans);
    p.few_borders[span] = make_int4(cur.u > 0 && c0 == span - 1 ? cur.b : -1, cur.h,
                                    (int)span_of(seg0 + cur.g.units - 1, total, spans),
                                    span_start(c0, total, spans) < seg0 ? 1 : 0);
  }

  uint8_t *ring = smem + (size_t)warp * S * F::kStage;
  const uint32_t ring_u = smem_u32(ring);
  int ids = 0, ids_b = -1, ids_at = 0;              // this lane's entry of 32 of the page table
  const int page_mask = (1 << p.page_shift) - 1;

  // The copies' place: this warp's units, every kWarps-th of the span.
  Cursor ahead = cur;
  int left = (int)min(u_end - u_begin, (int64_t)0x7FFFFFFF) - warp;   // units of the span from there on
  auto forward = [&](int n) {
    ahead.u += n;
    while (ahead.u >= ahead.g.units) {
      ahead.u -= ahead.g.units;
      if (!ahead.next(p)) {
        left = 0;
        return;
      }
    }
  };
  forward(warp);
  // Copies of the unit at `ahead` into a stage; keys outside [0, n) and pages
  // outside the cache are zero-filled and left out by their limit.
  auto copy_unit = [&](int stage) {
    int64_t oc[2], os[2];
    uint32_t bytes[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int key = (ahead.g.u0 + ahead.u) * kKeys + 16 * i, page = key >> p.page_shift;
      if (ids_b != ahead.b || page < ids_at || page >= ids_at + 32) {
        ids_b = ahead.b;
        ids_at = page & ~31;
        ids = ids_at + lane < p.max_pages ? __ldg(p.table + (int64_t)ids_b * p.table_ld + ids_at + lane) : -1;
      }
      const int id = __shfl_sync(0xffffffffu, ids, page - ids_at);
      int limit = min(16, ahead.g.s.n - key);
      if (limit <= 0 || !NVFP4_NOTE(id >= 0 && id < p.num_pages, p.status)) limit = 0;
      const int row = (ahead.h << p.page_shift) + (key & page_mask);
      oc[i] = limit ? id * p.codes_stride + row * (HD / 2) : 0;
      os[i] = limit ? id * p.sf_stride + row * (HD / 16) : 0;
      bytes[i] = limit ? 16u : 0u;
      if (lane == 0) limits[warp][stage][i] = limit;
    }
    const uint32_t dst = ring_u + stage * F::kStage;
    constexpr int kC = F::kCodes / 512;             // 16-byte runs of K's codes per lane
#pragma unroll
    for (int i = 0; i < kC; ++i) {
      const int hf = i / (kC / 2), at = ((i % (kC / 2)) * 32 + lane) * 16;
      cp_async_16(dst + (i * 32 + lane) * 16, p.k_codes + oc[hf] + at, bytes[hf]);
      cp_async_16(dst + F::kCodes + (i * 32 + lane) * 16, p.v_codes + oc[hf] + at, bytes[hf]);
    }
    constexpr int kR = F::kSf / 16;                 // 16-byte runs of K's scales
    if (lane < 2 * kR) {
      const int c = lane % kR, hf = c / (kR / 2);
      cp_async_16(dst + 2 * F::kCodes + lane * 16,
                  (lane < kR ? p.k_sf : p.v_sf) + (hf ? os[1] : os[0]) + (c % (kR / 2)) * 16, hf ? bytes[1] : bytes[0]);
    }
  };
  auto fetch = [&](int stage) {
    if (left > 0) {
      copy_unit(stage);
      left -= kWarps;
      if (left > 0) forward(kWarps);
    }
    cp_async_commit();
  };

#pragma unroll 1
  for (int i = 0; i < S - 1; ++i) fetch(i);

  uint32_t qf[NT][kMt][2];
  float sc[NT][2], m[NT][2], l[NT][2], o[kMt][NT][4];
  int see_lo[NT][2], see_hi[NT][2];                 // keys [see_lo, see_hi) of this lane's rows (8 nt + 2 t, + 1)
  int64_t u = u_begin + warp, first = u_begin;      // this warp's next unit; the span's first of the segment
  int stage = 0, fill = S - 1;

#pragma unroll 1
  while (true) {
    // ------------------------------------------------------- a segment's rows --
    const int rows = cur.g.rows;
    int all_lo = 0, all_hi = 0x7FFFFFFF;            // keys that every row sees
    {
      const float gsc = p.scale_log2 * p.gk[cur.h];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        uint32_t x[HD / 8];
        const int r = nt * 8 + g;
        const int tok = r / p.group, head = cur.h * p.group + r % p.group;
        const uint4 *src = reinterpret_cast<const uint4 *>(p.q + (int64_t)(cur.g.s.q0 + tok) * p.q_ld +
                                                           (int64_t)head * p.q_head_ld + t * (HD / 4));
        uint32_t m2 = 0;
#pragma unroll
        for (int v = 0; v < HD / 32; ++v) {
          const uint4 y = r < rows ? __ldg(src + v) : make_uint4(0, 0, 0, 0);
          x[4 * v] = y.x; x[4 * v + 1] = y.y; x[4 * v + 2] = y.z; x[4 * v + 3] = y.w;
        }
        // the order of |x| is that of its bits, infinities and NaNs last
#pragma unroll
        for (int v = 0; v < HD / 8; ++v) m2 = __vmaxu2(m2, x[v] & 0x7FFF7FFFu);
        m2 = __vmaxu2(m2, __shfl_xor_sync(0xffffffffu, m2, 1));
        m2 = __vmaxu2(m2, __shfl_xor_sync(0xffffffffu, m2, 2));
        const int e = (int)(max(m2 & 0xFFFFu, m2 >> 16) >> 7);
        // a power of two that brings the row's maximum to [2^13, 2^14); 1 for rows with an infinity or a NaN
        const int up = e == 255 ? 127 : min(267 - e, 190);
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
    const int64_t seg_end = seg0 + cur.g.units, end = min(seg_end, u_end);

    // -------------------------------------------------------- its units, in turn --
#pragma unroll 1
    for (; u < end; u += kWarps) {
      fetch(fill);
      cp_async_wait<S - 1>();
      __syncwarp();

      const uint8_t *st = ring + stage * F::kStage;
      const int limit0 = limits[warp][stage][0], limit1 = limits[warp][stage][1];
      const int key = (cur.g.u0 + (int)(u - seg0)) * kKeys;
      const bool whole = limit0 + limit1 == kKeys && key >= all_lo && key + kKeys <= all_hi;

      // S^T = K Q^T: keys g and g + 8 of both tiles
      float s[2][NT][4];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < 4; ++k) s[i][nt][k] = 0.0f;
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
              mma_f16(s[i][nt], a[0][2 * k], a[1][2 * k], a[0][2 * k + 1], a[1][2 * k + 1], qf[nt][2 * j + k][0],
                      qf[nt][2 * j + k][1]);
        }
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
          raise |= top[nt][k] > m[nt][k] + kRaise;
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

    // --------------------------------------------------- the warps' results, joined --
    __syncthreads();                                // (the last segment's have been read)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float sum_l = l[nt][k];
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) sum_l += __shfl_xor_sync(0xffffffffu, sum_l, d);
        const int r = nt * 8 + 2 * t + k;
        float4 *dst = reinterpret_cast<float4 *>(warp_o + (warp * F::kRows + r) * F::kPitch + g * (HD / 8));
#pragma unroll
        for (int j = 0; j < HD / 32; ++j)
          dst[j] = make_float4(o[2 * j][nt][k], o[2 * j][nt][k + 2], o[2 * j + 1][nt][k], o[2 * j + 1][nt][k + 2]);
        if (g == 0) warp_ml[warp][r] = make_float2(m[nt][k], sum_l);
      }
    __syncthreads();
    const bool full = first == seg0 && end == seg_end;
    const int64_t slot = 2 * span + (first == u_begin ? 0 : 1);
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
        if (p.lse && c == 0) p.lse[q * p.kv_heads * p.group + head] = (mm + __log2f(ll)) * CUDART_LN2_F;
      } else {
        float4 *dst = reinterpret_cast<float4 *>(p.part_o + (slot * F::kRows + r) * HD + c);
        dst[0] = make_float4(y[0], y[1], y[2], y[3]);
        dst[1] = make_float4(y[4], y[5], y[6], y[7]);
        if (c == 0) *reinterpret_cast<float2 *>(p.part_ml + (slot * F::kRows + r) * 2) = make_float2(mm, ll);
      }
    }
    if (end == u_end) break;
    seg0 = first = end;
    cur.next(p);
  }
  cp_async_wait<0>();
}

// Segments that lie in several spans: block = (border between two spans, row);
// the border behind a segment's first span stands for it.  The spans' partial
// results are dealt to the block's warps in order.
template <int HD, int NT>
__global__ void __launch_bounds__(128) k_kv_sum(const KvAttnParams p) {
  constexpr int kRows = 8 * NT, kV = HD / 32, kW = 4;
  __shared__ float sh_o[kW][HD];
  __shared__ float2 sh_ml[kW];
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, r = blockIdx.y;
  const int4 bd = __ldg(p.few_borders + blockIdx.x + 1);
  if (bd.x < 0) return;
  const int c0 = blockIdx.x, c1 = bd.z, h = bd.y;
  const KvSeq s = kv_seq(p, bd.x);
  if (r >= s.qn * p.group) return;
  float m = -CUDART_INF_F, l = 0.0f, o[kV];
#pragma unroll
  for (int v = 0; v < kV; ++v) o[v] = 0.0f;
#pragma unroll 4
  for (int c = c0 + warp; c <= c1; c += kW) {
    const int64_t row = (2ll * c + (c == c0 ? bd.w : 0)) * kRows + r;
    const float2 ml = __ldg(reinterpret_cast<const float2 *>(p.part_ml) + row);
    const float *src = p.part_o + row * HD + lane * kV;
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
#pragma unroll
  for (int v = 0; v < kV; ++v) sh_o[warp][lane * kV + v] = o[v];
  if (lane == 0) sh_ml[warp] = make_float2(m, l);
  __syncthreads();
  if (warp != 0) return;
  float mm = -CUDART_INF_F, ll = 0.0f;
#pragma unroll
  for (int w = 0; w < kW; ++w) mm = fmaxf(mm, sh_ml[w].x);
  const float ref = mm == -CUDART_INF_F ? 0.0f : mm;
#pragma unroll
  for (int v = 0; v < kV; ++v) o[v] = 0.0f;
#pragma unroll
  for (int w = 0; w < kW; ++w) {
    const float f = ex2(sh_ml[w].x - ref);
    ll += sh_ml[w].y * f;
#pragma unroll
    for (int v = 0; v < kV; ++v) o[v] += sh_o[w][lane * kV + v] * f;
  }
  const int64_t q = s.q0 + r / p.group;
  const int head = h * p.group + r % p.group;
  const float f = ll == 0.0f ? 0.0f : p.gv[h] / ll;
  __nv_bfloat16 *dst = p.out + q * p.out_ld + (int64_t)head * p.out_head_ld + lane * kV;
  if constexpr (kV == 4)
    *reinterpret_cast<uint2 *>(dst) = make_uint2(pack_bf2(o[0] * f, o[1] * f), pack_bf2(o[2] * f, o[3] * f));
  else
    *reinterpret_cast<uint32_t *>(dst) = pack_bf2(o[0] * f, o[1] * f);
  if (p.lse && lane == 0) p.lse[q * p.kv_heads * p.group + head] = (mm + __log2f(ll)) * CUDART_LN2_F;
}

template <int HD, int NT>
cudaError_t run_few(const KvAttnParams &p, int num_sms, cudaStream_t st) {
  using F = Few<HD, NT>;
  if (cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void *>(k_kv_few<HD, NT>), F::kSmem); e != cudaSuccess)
    return e;
  const int ctas = num_sms * F::kCtas;
  if (cudaError_t e = launch_pdl(k_kv_few<HD, NT>, dim3(ctas), dim3(kWarps * 32), F::kSmem, st, p); e != cudaSuccess)
    return e;
  return launch_pdl(k_kv_sum<HD, NT>, dim3(ctas - 1, std::min(F::kRows, p.few_rows_most)), dim3(128), 0, st, p);
}

}  // namespace

int kv_few_spans(int nt, int num_sms) { return num_sms * kv_few_ctas(nt); }

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
