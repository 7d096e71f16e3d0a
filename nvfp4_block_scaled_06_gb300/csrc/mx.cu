// mx.cu -- MXFP4 (OCP Microscaling Formats v1.0): bf16 <-> E2M1 codes with one
// E8M0 scale, a power of two, per 32 consecutive elements of a row.
//
//   amax = max |x| over the block;  X = 2^(floor(log2 amax) - 2)   (2 = E2M1's largest exponent)
//   scale byte = log2 X + 127, at least 0; an all-zero block has byte 0
//   code = sign(x) | E2M1_rn_satfinite(|x| / X)
//   a block that holds an infinity or a NaN: byte 255 (E8M0 NaN), codes 0
// x / X is exact in fp32 (a power-of-two scale of a bf16 value; what would
// fall below 2^-126 encodes to 0 either way), so the only rounding is the
// code's.  Back: E2M1(code) * 2^(byte - 127) is exact in bf16 for every byte
// the quantizer writes.
//
// HBM-bound, one pass: 2 B read + 0.53125 B written per element, and back.
// 32 x [2048, 6144] (1.02 GB either way): packing 157 us = 6.5 TB/s, unpacking
// 152 us = 6.7 TB/s (copy: 6.74 TB/s).
#include "internal.h"
#include "mxfp4.cuh"
#include "ptx.cuh"

namespace nvfp4 {

namespace {

constexpr int kMxUnit = 2;   // blocks per lane and step: 128 bytes of loads in flight per lane

// A warp's work item is (row, 64 consecutive blocks), a lane's block one
// 32-element block.  With the swizzled layout every scale byte of the padded
// rows and columns is written (0 outside the matrix).
// kScatter (swizzled): each source row goes to its `copies` rows of the grouped
// layout (a routed token's experts): X is read once and every copy is written
// from registers, 28.7 us for 4096 tokens of 6144 to 8 rows each (157 MB) instead
// of 35 us for packing the tokens and copying the packed rows.
template <bool kV8, bool kScatter>
__global__ void __launch_bounds__(256) k_mx_quant(const MxQuantParams p) {
  griddep_launch_dependents();
  griddep_wait();   // inputs may come from the previous kernel in the stream
  const int lane = threadIdx.x & 31;
  const uint32_t warp = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  const uint32_t nwarps = gridDim.x * (blockDim.x >> 5);
  const int64_t nblk = p.cols / 32, sfc_pad = (nblk + 3) & ~int64_t(3);
  const __nv_bfloat16 *src = p.src + (int64_t)blockIdx.y * p.bstride;
  uint8_t *codes = p.codes + (int64_t)blockIdx.y * p.codes_bstride;
  uint8_t *sf = p.sf + (int64_t)blockIdx.y * p.sf_bstride;
  int64_t rows_out = kScatter ? p.rows : p.sf_swizzled ? ((p.dst_rows + 127) & ~int64_t(127)) : p.dst_rows;
  if (p.num_mtiles) rows_out = min(rows_out, (int64_t)128 * *p.num_mtiles);
  const uint32_t nch = (uint32_t)((sfc_pad + 32 * kMxUnit - 1) / (32 * kMxUnit));
  const uint64_t items = (uint64_t)rows_out * nch;
  uint64_t r = warp / nch;
  uint32_t ch = warp % nch;
  const uint32_t dr = nwarps / nch, dch = nwarps % nch;
  for (uint64_t it = warp; it < items; it += nwarps) {
    int64_t sr = -1;
    if ((int64_t)r < (kScatter ? p.rows : p.dst_rows)) sr = p.row_map ? (int64_t)p.row_map[r] : (int64_t)r;
    if (!NVFP4_GUARD(sr < p.rows, p.status)) sr = -1;
    if (!(p.row_map && sr < 0)) {      // unmapped (padding) rows are left untouched
      const __nv_bfloat16 *srow = src + sr * p.ld;
      const int64_t blk0 = (int64_t)ch * (32 * kMxUnit) + lane;
      uint32_t w[kMxUnit][16];
#pragma unroll
      for (int u = 0; u < kMxUnit; ++u)
        if (sr >= 0 && blk0 + 32 * u < nblk) load32<kV8>(srow + (blk0 + 32 * u) * 32, w[u]);
#pragma unroll
      for (int u = 0; u < kMxUnit; ++u) {
        const int64_t blk = blk0 + 32 * u;
        uint32_t sb = 0;
        if constexpr (kScatter) {
          uint4 c = make_uint4(0, 0, 0, 0);
          if (blk < nblk) c = mx_encode32(w[u], sb);
          uint32_t v = sb;
          v |= __shfl_down_sync(0xffffffffu, sb, 1) << 8;
          v |= __shfl_down_sync(0xffffffffu, sb, 2) << 16;
          v |= __shfl_down_sync(0xffffffffu, sb, 3) << 24;
          for (int j = 0; j < p.copies; ++j) {
            const int64_t d = p.pair_row[(int64_t)r * p.copies + j];
            if (d < 0 || !NVFP4_GUARD(d < p.dst_rows, p.status)) continue;
            if (blk < nblk) *reinterpret_cast<uint4 *>(codes + d * (p.cols / 2) + blk * 16) = c;
            if ((lane & 3) == 0 && blk < sfc_pad)
              *reinterpret_cast<uint32_t *>(sf + 512 * ((d >> 7) * (sfc_pad >> 2) + (blk >> 2)) + 16 * (d & 31) +
                                            4 * ((d & 127) >> 5)) = v;
          }
          continue;
        }
        if (sr >= 0 && blk < nblk)
          *reinterpret_cast<uint4 *>(codes + (int64_t)r * (p.cols / 2) + blk * 16) = mx_encode32(w[u], sb);
        if (p.sf_swizzled) {
          uint32_t v = sb;
          v |= __shfl_down_sync(0xffffffffu, sb, 1) << 8;
          v |= __shfl_down_sync(0xffffffffu, sb, 2) << 16;
          v |= __shfl_down_sync(0xffffffffu, sb, 3) << 24;
          if ((lane & 3) == 0 && blk < sfc_pad)
            *reinterpret_cast<uint32_t *>(sf + 512 * ((int64_t)(r >> 7) * (sfc_pad >> 2) + (blk >> 2)) +
                                          16 * (r & 31) + 4 * ((r & 127) >> 5)) = v;
        } else if (blk < nblk) {
          sf[(int64_t)r * nblk + blk] = (uint8_t)sb;
        }
      }
    }
    r += dr;
    ch += dch;
    if (ch >= nch) {
      ch -= nch;
      ++r;
    }
  }
}

// 2^(byte - 127) as a bf16 pair; 255 is NaN.
__device__ __forceinline__ uint32_t mx_scale2(uint32_t byte) {
  const uint32_t h = byte == 0u ? 0x0040u : byte == 255u ? 0x7FC0u : byte << 7;
  return h * 0x00010001u;
}

__device__ __forceinline__ const uint8_t *mx_scale_at(const uint8_t *sf, int swz, int64_t r, int64_t blk,
                                                      int64_t nblk) {
  if (!swz) return sf + r * nblk + blk;
  const int64_t katoms = (nblk + 3) >> 2;
  return sf + 512 * ((r >> 7) * katoms + (blk >> 2)) + 16 * (r & 31) + 4 * ((r & 127) >> 5) + (blk & 3);
}
__device__ __forceinline__ uint32_t mx_scale_byte(const uint8_t *sf, int swz, int64_t r, int64_t blk, int64_t nblk) {
  return __ldg(mx_scale_at(sf, swz, r, blk, nblk));
}

// Eight codes (element i in nibble i) times the scale, as four bf16 pairs.  A
// magnitude's two bf16 bytes come from eight-entry byte tables (the byte
// permute's two source words), the sign from the permute's sign replication;
// the product with a power of two is exact.
__device__ __forceinline__ void mx_decode8(uint32_t c, uint32_t scale2, uint32_t (&o)[4]) {
  const uint32_t even = c << 4;                  // the even codes' signs on top of their bytes
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t sel = (h ? c >> 16 : c) & 0x7777u;
    const uint32_t lo = __byte_perm(0xC0800000u, 0xC0804000u, sel);
    uint32_t hi = __byte_perm(0x3F3F3F00u, 0x40404040u, sel), sign;
    if (h)
      asm("prmt.b32 %0, %1, %2, 0xBFAE;" : "=r"(sign) : "r"(c), "r"(even));
    else
      asm("prmt.b32 %0, %1, %2, 0x9D8C;" : "=r"(sign) : "r"(c), "r"(even));
    hi |= sign & 0x80808080u;
    const uint32_t w0 = __byte_perm(lo, hi, 0x5140), w1 = __byte_perm(lo, hi, 0x7362);
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(o[2 * h]) : "r"(w0), "r"(scale2));
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(o[2 * h + 1]) : "r"(w1), "r"(scale2));
  }
}

// Row-major: a thread takes one block, 16 bytes of codes in, 64 bytes of bf16
// out (whole 32-byte sectors where the row allows it).  Grid (ctas, batch).
__global__ void __launch_bounds__(256) k_mx_dequant(const uint8_t *__restrict__ codes, const uint8_t *__restrict__ sf,
                                                    int swz, int64_t rows, int64_t cols, int64_t sf_bstride,
                                                    __nv_bfloat16 *__restrict__ out, int64_t ldo,
                                                    int64_t out_bstride) {
  griddep_launch_dependents();
  griddep_wait();   // inputs may come from the previous kernel in the stream
  const int64_t nblk = cols / 32, total = rows * nblk;
  codes += (int64_t)blockIdx.y * rows * (cols / 2);
  sf += (int64_t)blockIdx.y * sf_bstride;
  out += (int64_t)blockIdx.y * out_bstride;
  for (int64_t t = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; t < total; t += (int64_t)gridDim.x * blockDim.x) {
    const int64_t r = t / nblk, blk = t - r * nblk;
    const uint4 c = __ldg(reinterpret_cast<const uint4 *>(codes) + t);
    const uint32_t s = mx_scale2(mx_scale_byte(sf, swz, r, blk, nblk));
    const uint32_t cw[4] = {c.x, c.y, c.z, c.w};
    uint32_t o[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) mx_decode8(cw[i], s, o[i]);
    uint4 *dst = reinterpret_cast<uint4 *>(out + r * ldo + blk * 32);
    if ((reinterpret_cast<uintptr_t>(dst) & 31) == 0) {
#pragma unroll
      for (int i = 0; i < 4; i += 2)
        st_global_v8(dst + i, o[i][0], o[i][1], o[i][2], o[i][3], o[i + 1][0], o[i + 1][1], o[i + 1][2], o[i + 1][3]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) dst[i] = make_uint4(o[i][0], o[i][1], o[i][2], o[i][3]);
    }
  }
}

// Transposed: thread = (row pair, block).  Consecutive threads take
// consecutive row pairs, so a store instruction writes 32 consecutive bf16
// pairs of one output row; a last single row takes two-byte stores.
__global__ void __launch_bounds__(256) k_mx_dequant_t(const uint8_t *__restrict__ codes,
                                                      const uint8_t *__restrict__ sf, int swz, int64_t rows,
                                                      int64_t cols, int64_t sf_bstride,
                                                      __nv_bfloat16 *__restrict__ out, int64_t ldo,
                                                      int64_t out_bstride) {
  griddep_launch_dependents();
  griddep_wait();   // inputs may come from the previous kernel in the stream
  const int64_t nblk = cols / 32, pairs = (rows + 1) / 2, total = pairs * nblk;
  codes += (int64_t)blockIdx.y * rows * (cols / 2);
  sf += (int64_t)blockIdx.y * sf_bstride;
  out += (int64_t)blockIdx.y * out_bstride;
  for (int64_t t = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; t < total; t += (int64_t)gridDim.x * blockDim.x) {
    const int64_t blk = t / pairs, r0 = 2 * (t - blk * pairs);
    const bool two = r0 + 1 < rows;
    uint4 c[2];
    uint32_t s[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      c[h] = make_uint4(0, 0, 0, 0);
      s[h] = 0u;
      if (h == 0 || two) {
        c[h] = __ldg(reinterpret_cast<const uint4 *>(codes + (r0 + h) * (cols / 2)) + blk);
        s[h] = mx_scale2(mx_scale_byte(sf, swz, r0 + h, blk, nblk));
      }
    }
    const uint32_t c0[4] = {c[0].x, c[0].y, c[0].z, c[0].w}, c1[4] = {c[1].x, c[1].y, c[1].z, c[1].w};
    __nv_bfloat16 *dst = out + blk * 32 * ldo + r0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      uint32_t pa[4], pb[4];
      mx_decode8(c0[i >> 2], s[0], pa);   // (unrolled: once per four i)
      mx_decode8(c1[i >> 2], s[1], pb);
      const uint32_t a = pa[i & 3], b = pb[i & 3];
      if (two) {
        *reinterpret_cast<uint32_t *>(dst + (2 * i) * ldo) = __byte_perm(a, b, 0x5410);
        *reinterpret_cast<uint32_t *>(dst + (2 * i + 1) * ldo) = __byte_perm(a, b, 0x7632);
      } else {
        *reinterpret_cast<uint16_t *>(dst + (2 * i) * ldo) = (uint16_t)a;
        *reinterpret_cast<uint16_t *>(dst + (2 * i + 1) * ldo) = (uint16_t)(a >> 16);
      }
    }
  }
}

// Transposed with whole vectors (rows and ldo multiples of 8): thread = (eight
// rows, half a block), 8 bytes of codes of each row in, per column one 16-byte
// store of its eight rows.  Of a warp's lanes eight take consecutive row groups
// (a store fills 128 bytes of four output rows) and four consecutive half
// blocks (a load reads 32 bytes of a row).  [2048, 6144]: 9 us alone with cold
// caches, one wave's latency; in front of the gradient GEMM 4 to 5 us.
__global__ void __launch_bounds__(128) k_mx_dequant_t8(const uint8_t *__restrict__ codes,
                                                       const uint8_t *__restrict__ sf, int swz, int64_t rows,
                                                       int64_t cols, int64_t sf_bstride,
                                                       __nv_bfloat16 *__restrict__ out, int64_t ldo,
                                                       int64_t out_bstride) {
  griddep_launch_dependents();
  griddep_wait();   // inputs may come from the previous kernel in the stream
  const int64_t nblk = cols / 32, groups = rows / 8;
  const int64_t gt = (groups + 7) / 8, bt = (nblk + 1) / 2;     // warps' tiles of 8 groups x 2 blocks
  codes += (int64_t)blockIdx.y * rows * (cols / 2);
  sf += (int64_t)blockIdx.y * sf_bstride;
  out += (int64_t)blockIdx.y * out_bstride;
  const int lane = threadIdx.x & 31;
  const int64_t nwarps = (int64_t)gridDim.x * 4;
  for (int64_t w = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5); w < gt * bt; w += nwarps) {
    const int64_t b4 = w / gt, g8 = w - b4 * gt;
    const int64_t g = g8 * 8 + (lane & 7), half = b4 * 4 + (lane >> 3), blk = half >> 1;
    if (g >= groups || blk >= nblk) continue;
    uint2 c[8];
    uint32_t s[8];
    const uint8_t *cr = codes + g * 8 * (cols / 2) + half * 8;
    const uint8_t *sr = mx_scale_at(sf, swz, g * 8, blk, nblk);
    const int64_t sstep = swz ? 16 : nblk;                 // (eight rows from a multiple of 8: one run of an atom)
#pragma unroll
    for (int r = 0; r < 8; ++r, cr += cols / 2) c[r] = __ldg(reinterpret_cast<const uint2 *>(cr));
#pragma unroll
    for (int r = 0; r < 8; ++r, sr += sstep) s[r] = mx_scale2(__ldg(sr));
    __nv_bfloat16 *d0 = out + half * 16 * ldo + g * 8;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      uint32_t v[8][4];
#pragma unroll
      for (int r = 0; r < 8; ++r) mx_decode8(q ? c[r].y : c[r].x, s[r], v[r]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        *reinterpret_cast<uint4 *>(d0) =
            make_uint4(__byte_perm(v[0][i], v[1][i], 0x5410), __byte_perm(v[2][i], v[3][i], 0x5410),
                       __byte_perm(v[4][i], v[5][i], 0x5410), __byte_perm(v[6][i], v[7][i], 0x5410));
        d0 += ldo;
        *reinterpret_cast<uint4 *>(d0) =
            make_uint4(__byte_perm(v[0][i], v[1][i], 0x7632), __byte_perm(v[2][i], v[3][i], 0x7632),
                       __byte_perm(v[4][i], v[5][i], 0x7632), __byte_perm(v[6][i], v[7][i], 0x7632));
        d0 += ldo;
      }
    }
  }
}

}  // namespace

cudaError_t launch_mx_quant(const MxQuantParams &p, int num_sms, cudaStream_t st) {
  const int64_t nblk = p.cols / 32, sfc_pad = (nblk + 3) & ~int64_t(3);
  const int64_t rows_out = p.pair_row      ? p.rows
                           : p.sf_swizzled ? ((p.dst_rows + 127) & ~int64_t(127))
                                           : p.dst_rows;
  const int64_t items = rows_out * ((sfc_pad + 32 * kMxUnit - 1) / (32 * kMxUnit));
  const int64_t cap = std::max<int64_t>(1, (int64_t)num_sms * 8 / p.batch);
  const dim3 grid((unsigned)std::max<int64_t>(1, std::min<int64_t>((items + 7) / 8, cap)), (unsigned)p.batch);
  const bool v8 = (reinterpret_cast<uintptr_t>(p.src) & 31) == 0 && p.ld % 16 == 0 && p.bstride % 16 == 0;
  if (p.pair_row)
    return v8 ? launch_pdl(k_mx_quant<true, true>, grid, dim3(256), 0, st, p)
              : launch_pdl(k_mx_quant<false, true>, grid, dim3(256), 0, st, p);
  return v8 ? launch_pdl(k_mx_quant<true, false>, grid, dim3(256), 0, st, p)
            : launch_pdl(k_mx_quant<false, false>, grid, dim3(256), 0, st, p);
}

cudaError_t launch_mx_dequant(const uint8_t *codes, const uint8_t *sf, int sf_swz, int64_t batch, int64_t rows,
                              int64_t cols, int64_t sf_bstride, int transpose, __nv_bfloat16 *out, int64_t ldo,
                              int64_t out_bstride, int num_sms, cudaStream_t st) {
  if (transpose && rows % 8 == 0 && ldo % 8 == 0 && out_bstride % 8 == 0 && reinterpret_cast<uintptr_t>(out) % 16 == 0) {
    const int64_t warps = (rows / 8 + 7) / 8 * ((cols / 32 + 1) / 2);
    const int64_t cap = std::max<int64_t>(1, (int64_t)num_sms * 32 / batch);
    const dim3 grid((unsigned)std::max<int64_t>(1, std::min<int64_t>((warps + 3) / 4, cap)), (unsigned)batch);
    return launch_pdl(k_mx_dequant_t8, grid, dim3(128), 0, st, codes, sf, sf_swz, rows, cols, sf_bstride, out, ldo,
                      out_bstride);
  }
  const int64_t work = (transpose ? (rows + 1) / 2 : rows) * (cols / 32);
  const int64_t cap = std::max<int64_t>(1, (int64_t)num_sms * 16 / batch);
  const dim3 grid((unsigned)std::max<int64_t>(1, std::min<int64_t>((work + 255) / 256, cap)), (unsigned)batch);
  return transpose ? launch_pdl(k_mx_dequant_t, grid, dim3(256), 0, st, codes, sf, sf_swz, rows, cols, sf_bstride, out,
                                ldo, out_bstride)
                   : launch_pdl(k_mx_dequant, grid, dim3(256), 0, st, codes, sf, sf_swz, rows, cols, sf_bstride, out,
                                ldo, out_bstride);
}

}  // namespace nvfp4
