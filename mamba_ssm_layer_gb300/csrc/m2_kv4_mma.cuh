// m2_kv4_mma.cuh -- the 4-bit cache's codes and scales as operands of warp MMA, and
// what the attention kernels over it share.
#pragma once
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "m2_common.cuh"
#include "m2_kv4.cuh"

namespace m2 {

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
      "%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The same from zero.
__device__ __forceinline__ void mma_f16_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, "
      "%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
// a times one half of s: the instruction broadcasts it.
__device__ __forceinline__ uint32_t hmul2_lo(uint32_t a, uint32_t s) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), __low2half2(*reinterpret_cast<const __half2*>(&s)));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t hmul2_hi(uint32_t a, uint32_t s) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), __high2half2(*reinterpret_cast<const __half2*>(&s)));
  return *reinterpret_cast<const uint32_t*>(&r);
}
// The four bytes of a code word as f16x2.
__device__ __forceinline__ void codes4(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\tcvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}
__device__ __forceinline__ uint32_t trans8x8(uint32_t a) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(a));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float ad_ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// 4-byte words of a lane's codes or scales.
template <int N>
__device__ __forceinline__ void lds_words(const uint8_t* p, uint32_t (&w)[N]) {
  if constexpr (N == 8) {
    const uint4 v = reinterpret_cast<const uint4*>(p)[0], x = reinterpret_cast<const uint4*>(p)[1];
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w, w[4] = x.x, w[5] = x.y, w[6] = x.z, w[7] = x.w;
  } else if constexpr (N == 4) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
  } else if constexpr (N == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x, w[1] = v.y;
  } else {
    static_assert(N == 1, "words");
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  }
}
// Two scale bytes of a word (0 and 2, or 1 and 3) as f16x2.
constexpr uint32_t kScaleBits = 0x7F807F80u;
__device__ __forceinline__ uint32_t scales02(uint32_t w, uint32_t mask) { return (w << 7) & mask; }
__device__ __forceinline__ uint32_t scales13(uint32_t w, uint32_t mask) { return (w >> 1) & mask; }

// Scores of a query row with largest magnitude `top`: f16 queries are the row times f
// (+-2^-e for a largest magnitude of 2^e .., exact in f16 except far below the largest;
// the scale's sign goes into them, and a scale of 0 makes them 0), scores their
// products times qs > 0, in log2 units.
__device__ __forceinline__ void kv4_query_scale(float top, float scale, float& f, float& qs) {
  int e = (int)(__float_as_uint(top) >> 23);
  e = e == 255 ? 127 : max(1, min(e, 253));
  const float sc = scale * 1.4426950408889634f, u = __uint_as_float((uint32_t)e << 23);
  f = sc == 0.0f ? 0.0f : copysignf(__uint_as_float((uint32_t)(254 - e) << 23), sc);
  qs = sc == 0.0f ? 1.0f : fmaxf(u * fabsf(sc), 1.17549435e-38f);
}
// Two f16 scales, 0 in the place of those that are not finite.
__device__ __forceinline__ uint32_t kv4_finite(uint32_t s) {
  if ((s & 0x7C00u) == 0x7C00u) s &= 0xFFFF0000u;
  if ((s & 0x7C000000u) == 0x7C000000u) s &= 0xFFFFu;
  return s;
}

// A part's weight against the joined maximum; a part that saw nothing has none
// (its sum is 0), and one of NaN scores passes its NaN on.
__device__ __forceinline__ float ad_weight(float m, float l, float top) {
  return m == -INFINITY ? (l == 0.0f ? 0.0f : 1.0f) : ad_ex2(m - top);
}

}  // namespace m2
