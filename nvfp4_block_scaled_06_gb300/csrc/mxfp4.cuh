// mxfp4.cuh -- one MXFP4 block: 32 bf16 values to E2M1 codes and an E8M0 scale
// (the arithmetic is described in mx.cu).
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

namespace nvfp4 {

// Sixteen 32-bit words (element 2i in the low half of w[i]) -> 32 codes as four
// words (element 2j in the low nibble of byte j) and the scale byte.
__device__ __forceinline__ uint4 mx_encode32(const uint32_t (&w)[16], uint32_t &sf) {
  uint32_t m2 = w[0] & 0x7FFF7FFFu;
#pragma unroll
  for (int i = 1; i < 16; ++i) m2 = __vmaxu2(m2, w[i] & 0x7FFF7FFFu);
  // the order of |x| is the order of its magnitude bits, infinities and NaNs last
  const uint32_t be = max(m2 & 0xFFFFu, m2 >> 16) >> 7;     // biased exponent of amax
  if (be == 255u) {
    sf = 255u;
    return make_uint4(0, 0, 0, 0);
  }
  const uint32_t byte = be > 2u ? be - 2u : 0u;
  sf = byte;
  const uint32_t inv = (254u - byte) << 23;                 // 2^(127 - byte), byte <= 252
  const uint64_t ss = ((uint64_t)inv << 32) | inv;
  uint32_t out[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t u = w[4 * q + i];
      const uint64_t x = ((uint64_t)(u & 0xFFFF0000u) << 32) | (uint64_t)(u << 16);
      uint64_t y;
      asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(y) : "l"(x), "l"(ss));
      v[2 * i] = __uint_as_float((uint32_t)y);
      v[2 * i + 1] = __uint_as_float((uint32_t)(y >> 32));
    }
    asm("{\n\t.reg .b8 t0, t1, t2, t3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 t0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 t1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 t2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 t3, %8, %7;\n\t"
        "mov.b32 %0, {t0, t1, t2, t3};\n\t}"
        : "=r"(out[q])
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  }
  return make_uint4(out[0], out[1], out[2], out[3]);
}

// One 32-element block (64 bytes).
template <bool kV8>
__device__ __forceinline__ void load32(const __nv_bfloat16 *src, uint32_t (&w)[16]) {
  if (kV8) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      asm volatile("ld.global.nc.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                   : "=r"(w[8 * h]), "=r"(w[8 * h + 1]), "=r"(w[8 * h + 2]), "=r"(w[8 * h + 3]),
                     "=r"(w[8 * h + 4]), "=r"(w[8 * h + 5]), "=r"(w[8 * h + 6]), "=r"(w[8 * h + 7])
                   : "l"(src + 16 * h));
  } else {
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      const uint4 a = __ldg(reinterpret_cast<const uint4 *>(src) + h);
      w[4 * h] = a.x; w[4 * h + 1] = a.y; w[4 * h + 2] = a.z; w[4 * h + 3] = a.w;
    }
  }
}

}  // namespace nvfp4
