// encode.cuh -- one NVFP4 block: 16 bf16 values to E2M1 codes under a given
// encode scale (the packing kernels of quantize.cu and of the key-value cache).
#pragma once

#include <stdint.h>

namespace nvfp4 {

// max of |x| over the two bf16 halves of each word (sign bits cleared; the bf16
// maximum of non-negative values is exact).
__device__ __forceinline__ uint32_t bmax2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Eight bf16 pairs times one fp32 scale (one IEEE rounding each), encoded as
// 16 E2M1 codes: element 2i in the low nibble of byte i.
__device__ __forceinline__ uint64_t encode16(const uint32_t (&w)[8], float senc) {
  const uint64_t ss = ((uint64_t)__float_as_uint(senc) << 32) | __float_as_uint(senc);
  float v[16];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint64_t x = ((uint64_t)(w[i] & 0xFFFF0000u) << 32) | (uint64_t)(w[i] << 16);
    uint64_t y;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(y) : "l"(x), "l"(ss));
    v[2 * i] = __uint_as_float((uint32_t)y);
    v[2 * i + 1] = __uint_as_float((uint32_t)(y >> 32));
  }
  uint32_t out[2];
#pragma unroll
  for (int h = 0; h < 2; ++h)
    asm("{\n\t.reg .b8 t0, t1, t2, t3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 t0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 t1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 t2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 t3, %8, %7;\n\t"
        "mov.b32 %0, {t0, t1, t2, t3};\n\t}"
        : "=r"(out[h])
        : "f"(v[8 * h]), "f"(v[8 * h + 1]), "f"(v[8 * h + 2]), "f"(v[8 * h + 3]),
          "f"(v[8 * h + 4]), "f"(v[8 * h + 5]), "f"(v[8 * h + 6]), "f"(v[8 * h + 7]));
  return (uint64_t)out[0] | ((uint64_t)out[1] << 32);
}

}  // namespace nvfp4
