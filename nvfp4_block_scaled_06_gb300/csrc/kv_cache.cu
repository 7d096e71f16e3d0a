// kv_cache.cu -- keys and values into the pages of the NVFP4 cache, and back.
//
// A row of a head (head_dim channels) is packed as nvfp4_quantize packs a
// matrix row under a static scale, g per key-value head:
//   byte = E4M3(amax / (6 g)),  code = E2M1(x * (1 / (byte * g)))
// every operation one IEEE fp32 rounding; back: bf16(E2M1(code) * (byte * g)).
// Infinities saturate; a block that holds a NaN gets byte 0x7F (NaN), codes 0.
// Blocks run along the channels, so a token is written without its neighbours.
//
// HBM-bound: 2 B read + 0.5625 B written per element, and back.  A warp takes
// consecutive tokens of one head: its codes are one run of a page where the
// slots are consecutive, while consecutive warps take the heads of the same
// tokens, whose bf16 rows are neighbours.
#include <float.h>

#include "encode.cuh"
#include "internal.h"
#include "kv.cuh"
#include "ptx.cuh"

namespace nvfp4 {

namespace {

// Slot -> byte offsets of its codes and scales; false where it is outside the cache.
__device__ __forceinline__ bool kv_at(const KvPages &c, int64_t slot, int h, int64_t &codes, int64_t &sf) {
  const int64_t page = slot >> c.page_shift;
  if (slot < 0 || page >= c.num_pages) return false;
  const int64_t row = ((int64_t)h << c.page_shift) + (slot & ((1 << c.page_shift) - 1));
  codes = page * c.codes_stride + row * (c.head_dim / 2);
  sf = page * c.sf_stride + row * (c.head_dim / 16);
  return true;
}

// Grid (ctas, 2): y = 0 the keys, 1 the values.  A lane takes one 16-channel
// block; kLanes = head_dim / 16 lanes a row.
template <int kLanes>
__global__ void __launch_bounds__(256) k_kv_write(const KvCopyParams p) {
  griddep_launch_dependents();
  griddep_wait();   // inputs may come from the previous kernel in the stream
  constexpr int kRows = 32 / kLanes;
  const int lane = threadIdx.x & 31, blk = lane % kLanes;
  const bool val = blockIdx.y != 0;
  const __nv_bfloat16 *src = static_cast<const __nv_bfloat16 *>(val ? p.v : p.k);
  const int64_t ld = val ? p.v_ld : p.k_ld, hld = val ? p.v_head_ld : p.k_head_ld;
  uint8_t *codes = val ? p.c.v_codes : p.c.k_codes, *sf = val ? p.c.v_sf : p.c.k_sf;
  const int64_t items = (p.tokens + kRows - 1) / kRows * p.c.kv_heads;
  const int64_t nwarps = (int64_t)gridDim.x * (blockDim.x >> 5);
  for (int64_t it = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); it < items; it += nwarps) {
    const int64_t t = it / p.c.kv_heads * kRows + lane / kLanes;
    const int h = (int)(it % p.c.kv_heads);
    int64_t oc = 0, os = 0;
    const bool on = t < p.tokens && kv_at(p.c, p.slots[t], h, oc, os);
    uint32_t sb = 0;
    if (on) {
      const float g = (val ? p.gv : p.gk)[h];
      const uint4 *s4 = reinterpret_cast<const uint4 *>(src + t * ld + h * hld + blk * 16);
      const uint4 a = __ldg(s4), b = __ldg(s4 + 1);
      const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
      uint32_t m2 = w[0] & 0x7FFF7FFFu;
#pragma unroll
      for (int i = 1; i < 8; ++i) m2 = __vmaxu2(m2, w[i] & 0x7FFF7FFFu);
      const float amax = __uint_as_float(max(m2 & 0xFFFFu, m2 >> 16) << 16);
      if (g > 0.0f) sb = cvt_e4m3(__fdiv_rn(amax, __fmul_rn(6.0f, g)));
      uint64_t c = 0;
      if (sb != 0 && sb != 0x7Fu) c = encode16(w, fminf(__frcp_rn(__fmul_rn(e4m3_to_f32(sb), g)), FLT_MAX));
      *reinterpret_cast<uint2 *>(codes + oc + blk * 8) = make_uint2((uint32_t)c, (uint32_t)(c >> 32));
    }
    uint32_t v = sb;
    v |= __shfl_down_sync(0xffffffffu, sb, 1) << 8;
    v |= __shfl_down_sync(0xffffffffu, sb, 2) << 16;
    v |= __shfl_down_sync(0xffffffffu, sb, 3) << 24;
    if (on && (blk & 3) == 0) *reinterpret_cast<uint32_t *>(sf + os + blk) = v;
  }
}

template <int kLanes, bool kF32>
__global__ void __launch_bounds__(256) k_kv_read(const KvCopyParams p) {
  griddep_launch_dependents();
  griddep_wait();   // inputs may come from the previous kernel in the stream
  constexpr int kRows = 32 / kLanes;
  const int lane = threadIdx.x & 31, blk = lane % kLanes;
  const bool val = blockIdx.y != 0;
  const int64_t ld = val ? p.v_ld : p.k_ld, hld = val ? p.v_head_ld : p.k_head_ld;
  const uint8_t *codes = val ? p.c.v_codes : p.c.k_codes, *sf = val ? p.c.v_sf : p.c.k_sf;
  const int64_t items = (p.tokens + kRows - 1) / kRows * p.c.kv_heads;
  const int64_t nwarps = (int64_t)gridDim.x * (blockDim.x >> 5);
  for (int64_t it = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); it < items; it += nwarps) {
    const int64_t t = it / p.c.kv_heads * kRows + lane / kLanes;
    const int h = (int)(it % p.c.kv_heads);
    int64_t oc = 0, os = 0;
    if (!(t < p.tokens && kv_at(p.c, p.slots[t], h, oc, os))) continue;
    const float s = __fmul_rn(e4m3_to_f32(__ldg(sf + os + blk)), (val ? p.gv : p.gk)[h]);
    const uint2 c = __ldg(reinterpret_cast<const uint2 *>(codes + oc) + blk);
    uint32_t h2[2][4];
    e2m1x8_to_h2(c.x, h2[0]);
    e2m1x8_to_h2(c.y, h2[1]);
    float f[16];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 x = __half22float2(*reinterpret_cast<const __half2 *>(&h2[i >> 2][i & 3]));
      f[2 * i] = __fmul_rn(x.x, s);
      f[2 * i + 1] = __fmul_rn(x.y, s);
    }
    const int64_t at = t * ld + h * hld + blk * 16;
    if (kF32) {
      float4 *dst = reinterpret_cast<float4 *>(static_cast<float *>(val ? p.v : p.k) + at);
#pragma unroll
      for (int i = 0; i < 4; ++i) dst[i] = make_float4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
    } else {
      uint4 *dst = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(val ? p.v : p.k) + at);
#pragma unroll
      for (int i = 0; i < 2; ++i)
        dst[i] = make_uint4(pack_bf2(f[8 * i], f[8 * i + 1]), pack_bf2(f[8 * i + 2], f[8 * i + 3]),
                            pack_bf2(f[8 * i + 4], f[8 * i + 5]), pack_bf2(f[8 * i + 6], f[8 * i + 7]));
    }
  }
}

dim3 kv_grid(const KvCopyParams &p, int num_sms) {
  const int64_t rows = 512 / p.c.head_dim;   // tokens per warp
  const int64_t warps = (p.tokens + rows - 1) / rows * p.c.kv_heads;
  return dim3((unsigned)std::min<int64_t>((warps + 7) / 8, (int64_t)num_sms * 4), 2);
}

}  // namespace

cudaError_t launch_kv_write(const KvCopyParams &p, int num_sms, cudaStream_t st) {
  return p.c.head_dim == 128 ? launch_pdl(k_kv_write<8>, kv_grid(p, num_sms), dim3(256), 0, st, p)
                             : launch_pdl(k_kv_write<4>, kv_grid(p, num_sms), dim3(256), 0, st, p);
}

cudaError_t launch_kv_read(const KvCopyParams &p, bool fp32, int num_sms, cudaStream_t st) {
  const dim3 g = kv_grid(p, num_sms), b(256);
  if (p.c.head_dim == 128)
    return fp32 ? launch_pdl(k_kv_read<8, true>, g, b, 0, st, p) : launch_pdl(k_kv_read<8, false>, g, b, 0, st, p);
  return fp32 ? launch_pdl(k_kv_read<4, true>, g, b, 0, st, p) : launch_pdl(k_kv_read<4, false>, g, b, 0, st, p);
}

}  // namespace nvfp4
