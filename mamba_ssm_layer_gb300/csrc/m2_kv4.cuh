// m2_kv4.cuh -- the paged 4-bit cache's format (include/mamba2.h): scale bytes,
// codes, and where they lie in a block (one page of one kv head).
#pragma once
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "m2_common.cuh"

namespace m2 {

constexpr int kPage = 64;

// Byte offsets in a block of 72 * D bytes.
template <int D>
struct Kv4Block {
  static constexpr int kBytes = 72 * D;
  static constexpr int kK = 0, kV = 32 * D, kKs = 64 * D, kVs = 68 * D;
  // K codes of token t, channels 16g + 4c .. 16g + 4c + 3: two bytes
  __host__ __device__ static constexpr int k(int t, int g, int c) { return kK + t * (D / 2) + c * (D / 8) + g * 2; }
  // V codes of channel 8i + r for the tokens t & ~1 (low nibble) and t | 1
  __host__ __device__ static constexpr int v(int t, int i, int r) {
    return kV + (t >> 3) * (4 * D) + r * (D / 2) + ((t & 7) >> 1) * (D / 8) + i;
  }
  __host__ __device__ static constexpr int ks(int t, int g) { return kKs + t * (D / 16) + g; }
  __host__ __device__ static constexpr int vs(int t, int g) {
    return kVs + (t >> 1) * (D / 8) + (g >> 1) * 4 + (t & 1) * 2 + (g & 1);
  }
};

// The cache kernels leave out what the table does not cover and say so.
#define M2_RECORD_ARG(status) atomicCAS(&(status), 0, -1)

// A product that stands for a quotient: off it by about 2^-23, and rounded to 15
// significant bits the quotient itself wherever that is a boundary of what it is
// rounded to next, and nowhere else.  That holds for quotients of a bf16 value (8
// bits) and 6 or a scale (4 bits): they come no closer than 2^-9 to a boundary of
// at most 5 bits without meeting it.
__device__ __forceinline__ float kv4_quotient(float product) {
  return __uint_as_float((__float_as_uint(product) + 0x100u) & 0xFFFFFE00u);
}
// Scale byte of a group with largest magnitude amax (NaN already found apart):
// amax / 6 rounded to nearest even on 4 significant bits, at most 10240, so
// that 6 * scale stays an f16 value.  Below 2^-14 the step stays 2^-17.
__device__ __forceinline__ uint32_t kv4_scale_byte(float amax) {
  const float t = fminf(kv4_quotient(amax * (1.0f / 6.0f)), 10240.0f);
  if (t < 6.103515625e-5f) return (uint32_t)__float2int_rn(t * 131072.0f);  // 2^-14; a carry to 8 is 2^-14 itself
  const uint32_t b = __float_as_uint(t);
  return ((b + 0x7FFFFu + ((b >> 20) & 1u)) >> 20) - (112u << 3);  // fp32 bias 127 -> 15
}
// Its value: the bits are an f16's without sign and low mantissa bits.
__device__ __forceinline__ float kv4_scale(uint32_t byte) {
  return __half2float(__ushort_as_half((unsigned short)(byte << 7)));
}

// Two channels times the scale's reciprocal -> one byte of codes (x in the low
// nibble): the hardware conversion rounds to nearest even and saturates.  The
// quotients are rounded to multiples of 2^-13 on the way (by a large addend),
// for the same reason: boundaries are multiples of 2^-2, and a quotient that is
// not one of them is at least 2^-11 off.
__device__ __forceinline__ uint32_t kv4_codes(float2 x, float inv) {
  uint32_t r;
  asm("{\n\t.reg .b64 q, i, m, n;\n\t.reg .b32 u, v;\n\t.reg .f32 a, b;\n\t.reg .b8 c;\n\t"
      "mov.b64 q, {%1, %2};\n\tmov.b64 i, {%3, %3};\n\tmov.b64 m, {%4, %4};\n\tmov.b64 n, {%5, %5};\n\t"
      "fma.rn.f32x2 q, q, i, m;\n\tadd.rn.f32x2 q, q, n;\n\tmov.b64 {a, b}, q;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, b, a;\n\tmov.b32 %0, {c, 0, 0, 0};\n\t}"
      : "=r"(r)
      : "f"(x.x), "f"(x.y), "f"(inv), "f"(1536.0f), "f"(-1536.0f));
  return r;
}
// The low byte of codes -> f16x2 (low nibble in the low half), exactly.
__device__ __forceinline__ uint32_t kv4_f16x2(uint32_t codes) {
  uint32_t r;
  asm("{\n\t.reg .b8 c, d, e, f;\n\tmov.b32 {c, d, e, f}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, c;\n\t}" : "=r"(r) : "r"(codes));
  return r;
}
}  // namespace m2
