// kv_cache.cu -- keys and values into the pages of the NVFP4 cache, and back.
//
// A row of a head (head_dim channels) is packed as nvfp4_quantize packs a
// matrix row under a static scale, g per key-value head:
//   byte = E4M3(amax / (6 g)),  code = E2M1(x * (1 / (byte * g)))
// every operation one IEEE fp32 rounding; back: bf16(E2M1(code) * (byte * g)).
// Infinities saturate; a block that holds a NaN gets byte 0x7F (NaN), codes 0.
// Blocks run along the channels, so a token is written without its neighbours.
//
// HBM-bound: 2 B read + 0.5625 B written per element, and back.  A lane takes 32
// channels (64 bytes of bf16, 16 of codes, two scales) of two tokens at a time,
// all loads first; a warp consecutive tokens of one head, whose codes are one run
// of a page where the slots are consecutive, while consecutive warps take the
// heads of the same tokens, whose bf16 rows are neighbours.  65521 tokens of 16
// heads of 64: the write 65 us for 344 MB (5.3 TB/s, cold), the read 55 us
// (6.2 TB/s); a call of both 125 us in grids of one wave, 133 with a warp's items
// spread over more CTAs.
#include <float.h>

#include "encode.cuh"
#include "internal.h"
#include "kv.cuh"
#include "mxfp4.cuh"
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

constexpr int kTokens = 2;            // of a lane at a time

// What this warp works on: grid (ctas, 2), y = 0 the keys, 1 the values; items of
// kRows x kTokens tokens and one head, heads fastest.
struct KvWalk {
  int64_t group, groups;              // of tokens
  int head, heads, step_head;
  int64_t step_group;
  __device__ __forceinline__ KvWalk(const KvCopyParams &p, int tokens) {
    const int64_t warp = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    const int64_t warps = (int64_t)gridDim.x * (blockDim.x >> 5);
    heads = p.c.kv_heads;
    groups = kv_div(p.tokens + tokens - 1, tokens);
    group = kv_div(warp, heads);
    head = (int)(warp - group * heads);
    step_group = kv_div(warps, heads);
    step_head = (int)(warps - step_group * heads);
  }
  __device__ __forceinline__ bool on() const { return group < groups; }
  __device__ __forceinline__ void next() {
    group += step_group;
    head += step_head;
    if (head >= heads) {
      head -= heads;
      ++group;
    }
  }
};

template <int HD>
__global__ void __launch_bounds__(256, 3) k_kv_write(const KvCopyParams p) {
  griddep_launch_dependents();
  griddep_wait();   // inputs may come from the previous kernel in the stream
  constexpr int kLanes = HD / 32, kRows = 32 / kLanes;
  const int lane = threadIdx.x & 31, q = lane % kLanes;
  const bool val = blockIdx.y != 0;
  const __nv_bfloat16 *src = static_cast<const __nv_bfloat16 *>(val ? p.v : p.k) + q * 32;
  const int64_t ld = val ? p.v_ld : p.k_ld, hld = val ? p.v_head_ld : p.k_head_ld;
  uint8_t *codes = (val ? p.c.v_codes : p.c.k_codes) + q * 16, *sf = (val ? p.c.v_sf : p.c.k_sf) + q * 2;
  const bool wide = ((reinterpret_cast<uintptr_t>(src) >> 1 | ld | hld) & 15) == 0;   // whole 32-byte sectors
  for (KvWalk w(p, kRows * kTokens); w.on(); w.next()) {
    int64_t oc[kTokens], os[kTokens];
    bool on[kTokens];
    uint32_t x[kTokens][16];
#pragma unroll
    for (int i = 0; i < kTokens; ++i) {
      const int64_t t = (w.group * kTokens + i) * kRows + lane / kLanes;
      on[i] = t < p.tokens && kv_at(p.c, __ldg(p.slots + t), w.head, oc[i], os[i]);
      if (on[i]) {
        if (wide)
          load32<true>(src + t * ld + w.head * hld, x[i]);
        else
          load32<false>(src + t * ld + w.head * hld, x[i]);
      }
    }
    const float g = (val ? p.gv : p.gk)[w.head], g6 = __fmul_rn(6.0f, g);
#pragma unroll
    for (int i = 0; i < kTokens; ++i) {
      uint32_t sb2 = 0;
      if (on[i]) {
        uint64_t c[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          uint32_t b[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) b[e] = x[i][8 * k + e];
          uint32_t m2 = b[0] & 0x7FFF7FFFu;
#pragma unroll
          for (int e = 1; e < 8; ++e) m2 = __vmaxu2(m2, b[e] & 0x7FFF7FFFu);
          const float amax = __uint_as_float(max(m2 & 0xFFFFu, m2 >> 16) << 16);
          const uint32_t sb = g > 0.0f ? cvt_e4m3(__fdiv_rn(amax, g6)) : 0u;
          c[k] = 0;
          if (sb != 0 && sb != 0x7Fu) c[k] = encode16(b, fminf(__frcp_rn(__fmul_rn(e4m3_to_f32(sb), g)), FLT_MAX));
          sb2 |= sb << (8 * k);
        }
        *reinterpret_cast<uint4 *>(codes + oc[i]) = make_uint4((uint32_t)c[0], (uint32_t)(c[0] >> 32), (uint32_t)c[1],
                                                               (uint32_t)(c[1] >> 32));
      }
      sb2 |= __shfl_down_sync(0xffffffffu, sb2, 1) << 16;
      if (on[i] && (q & 1) == 0) *reinterpret_cast<uint32_t *>(sf + os[i]) = sb2;
    }
  }
}

template <int HD, bool kF32>
__global__ void __launch_bounds__(256, 6) k_kv_read(const KvCopyParams p) {
  griddep_launch_dependents();
  griddep_wait();   // inputs may come from the previous kernel in the stream
  constexpr int kLanes = HD / 32, kRows = 32 / kLanes;
  const int lane = threadIdx.x & 31, q = lane % kLanes;
  const bool val = blockIdx.y != 0;
  const int64_t ld = val ? p.v_ld : p.k_ld, hld = val ? p.v_head_ld : p.k_head_ld;
  const uint8_t *codes = (val ? p.c.v_codes : p.c.k_codes) + q * 16, *sf = (val ? p.c.v_sf : p.c.k_sf) + q * 2;
  for (KvWalk w(p, kRows * kTokens); w.on(); w.next()) {
    uint4 c[kTokens];
    uint32_t s2[kTokens];
    bool on[kTokens];
#pragma unroll
    for (int i = 0; i < kTokens; ++i) {
      const int64_t t = (w.group * kTokens + i) * kRows + lane / kLanes;
      int64_t oc = 0, os = 0;
      on[i] = t < p.tokens && kv_at(p.c, __ldg(p.slots + t), w.head, oc, os);
      if (on[i]) {
        c[i] = __ldg(reinterpret_cast<const uint4 *>(codes + oc));
        s2[i] = __ldg(reinterpret_cast<const uint16_t *>(sf + os));
      }
    }
    const float g = (val ? p.gv : p.gk)[w.head];
#pragma unroll
    for (int i = 0; i < kTokens; ++i) {
      if (!on[i]) continue;
      const int64_t t = (w.group * kTokens + i) * kRows + lane / kLanes, at = t * ld + w.head * hld + q * 32;
      const uint32_t cw[4] = {c[i].x, c[i].y, c[i].z, c[i].w};
      uint32_t o[16];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float s = __fmul_rn(e4m3_to_f32(s2[i] >> (8 * (k >> 1))), g);
        uint32_t h2[4];
        e2m1x8_to_h2(cw[k], h2);
        float f[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&h2[e]));
          f[2 * e] = __fmul_rn(v.x, s);
          f[2 * e + 1] = __fmul_rn(v.y, s);
        }
        if constexpr (kF32) {
          float4 *dst = reinterpret_cast<float4 *>(static_cast<float *>(val ? p.v : p.k) + at) + 2 * k;
          dst[0] = make_float4(f[0], f[1], f[2], f[3]);
          dst[1] = make_float4(f[4], f[5], f[6], f[7]);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) o[4 * k + e] = pack_bf2(f[2 * e], f[2 * e + 1]);
        }
      }
      if constexpr (!kF32) {
        uint4 *dst = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(val ? p.v : p.k) + at);
        if ((reinterpret_cast<uintptr_t>(dst) & 31) == 0) {
#pragma unroll
          for (int k = 0; k < 2; ++k)
            st_global_v8(dst + 2 * k, o[8 * k], o[8 * k + 1], o[8 * k + 2], o[8 * k + 3], o[8 * k + 4], o[8 * k + 5],
                         o[8 * k + 6], o[8 * k + 7]);
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k) dst[k] = make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
        }
      }
    }
  }
}

// CTAs for half of `per_sm` on each SM in each of the two rows of the grid: one wave.
dim3 kv_grid(const KvCopyParams &p, int num_sms, int per_sm) {
  const int64_t tokens = 32 / (p.c.head_dim / 32) * kTokens;   // of a warp at a time
  const int64_t warps = (p.tokens + tokens - 1) / tokens * p.c.kv_heads;
  return dim3((unsigned)std::min<int64_t>((warps + 7) / 8, std::max<int64_t>(1, (int64_t)num_sms * per_sm / 2)), 2);
}

}  // namespace

cudaError_t launch_kv_write(const KvCopyParams &p, int num_sms, cudaStream_t st) {
  return p.c.head_dim == 128 ? launch_pdl(k_kv_write<128>, kv_grid(p, num_sms, 3), dim3(256), 0, st, p)
                             : launch_pdl(k_kv_write<64>, kv_grid(p, num_sms, 3), dim3(256), 0, st, p);
}

cudaError_t launch_kv_read(const KvCopyParams &p, bool fp32, int num_sms, cudaStream_t st) {
  const dim3 g = kv_grid(p, num_sms, 6), b(256);
  if (p.c.head_dim == 128)
    return fp32 ? launch_pdl(k_kv_read<128, true>, g, b, 0, st, p) : launch_pdl(k_kv_read<128, false>, g, b, 0, st, p);
  return fp32 ? launch_pdl(k_kv_read<64, true>, g, b, 0, st, p) : launch_pdl(k_kv_read<64, false>, g, b, 0, st, p);
}

}  // namespace nvfp4
