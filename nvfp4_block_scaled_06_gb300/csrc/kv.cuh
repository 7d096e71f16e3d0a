// kv.cuh -- what the kernels of the NVFP4 key-value cache share: the page
// addressing, a sequence's clamped sizes, and the decode of packed rows.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "internal.h"
#include "ptx.cuh"

namespace nvfp4 {

// Four E2M1 bytes of a word (low nibble first) -> four f16 pairs, exact.
__device__ __forceinline__ void e2m1x8_to_h2(uint32_t w, uint32_t (&o)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\tcvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\tcvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3])
      : "r"(w));
}
// Two E4M3 bytes (low half word) -> an f16 pair, exact.
__device__ __forceinline__ uint32_t e4m3x2_to_h2(uint32_t b) {
  uint32_t r;
  const uint16_t in = (uint16_t)b;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(in));
  return r;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t pack_bf2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// ln(l 2^m): log2 is taken of l's mantissa, where its error is least (2^-22).
__device__ __forceinline__ float kv_lse(float m, float l) {
  const int e = min((int)(__float_as_uint(l) >> 23), 253) - 127;   // (NaN and infinity stay what they are)
  return (m + (float)e + __log2f(l * __uint_as_float((uint32_t)(127 - e) << 23))) * 0.693147181f;
}

// A sequence's sizes as the kernels use them.  q_offsets and kv_lens are device
// data that the host cannot check: offsets are clamped to [0, total_q] and to
// ascending order, lengths to the page table's width, so inconsistent ones give
// wrong rows, never an access outside the buffers.
struct KvSeq {
  int q0;        // first query row
  int qt, qn;    // new tokens, those of them that are computed (up to max_q)
  int n;         // keys
  int lo, hi;    // keys [lo, hi) that at least one computed row sees
};
__device__ __forceinline__ KvSeq kv_seq(const KvAttnParams &p, int b) {
  KvSeq s;
  int q1;
  if (p.q_offsets) {
    s.q0 = min(max(p.q_offsets[b], 0), p.total_q);
    q1 = min(max(p.q_offsets[b + 1], s.q0), p.total_q);
  } else {
    s.q0 = b;
    q1 = b + 1;
  }
  s.qt = q1 - s.q0;
  s.qn = min(s.qt, p.max_q);
  const int64_t cap = min((int64_t)p.max_pages << p.page_shift, (int64_t)0x7FFFFF00);
  s.n = (int)min((int64_t)max(p.kv_lens[b], 0), cap);
  const int64_t first = p.window > 0 ? (int64_t)s.n - s.qt + 1 - p.window : 0;
  s.lo = (int)min(max(first, (int64_t)0), (int64_t)s.n);
  s.hi = p.causal ? max(s.n - s.qt + s.qn, 0) : s.n;
  s.lo = min(s.lo, s.hi);
  return s;
}

// a / b for non-negative a, with the 32-bit division where both fit (a 64-bit one
// takes some 500 cycles, several of which once stood before a kernel's first load).
__device__ __forceinline__ int64_t kv_div(int64_t a, int64_t b) {
  return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}
// `total` places in `spans` runs that differ by one place at most.
struct KvCut {
  int64_t total, spans, per, longer;   // the first `longer` runs have per + 1 places
  __device__ __forceinline__ KvCut(int64_t t, int64_t most) : total(t), spans(min(t, most)) {
    per = spans > 0 ? kv_div(total, spans) : 0;
    longer = total - per * spans;
  }
  __device__ __forceinline__ int64_t start(int64_t w) const { return w * per + min(w, longer); }
  __device__ __forceinline__ int64_t owner(int64_t u) const {
    const int64_t head = longer * (per + 1);
    return u < head ? kv_div(u, per + 1) : longer + kv_div(u - head, per);
  }
};

}  // namespace nvfp4
