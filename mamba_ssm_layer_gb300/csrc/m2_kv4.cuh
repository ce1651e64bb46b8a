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

// Scale byte of a group with largest magnitude amax (NaN already found apart):
// amax / 6 rounded to nearest even on 4 significant bits, at most 10240, so
// that 6 * scale stays an f16 value.  Below 2^-14 the step stays 2^-17.
__device__ __forceinline__ uint32_t kv4_scale_byte(float amax) {
  const float t = fminf(__fdiv_rn(amax, 6.0f), 10240.0f);
  if (t < 6.103515625e-5f) return (uint32_t)__float2int_rn(t * 131072.0f);  // 2^-14; a carry to 8 is 2^-14 itself
  const uint32_t b = __float_as_uint(t);
  return ((b + 0x7FFFFu + ((b >> 20) & 1u)) >> 20) - (112u << 3);  // fp32 bias 127 -> 15
}
// Its value: the bits are an f16's without sign and low mantissa bits.
__device__ __forceinline__ float kv4_scale(uint32_t byte) {
  return __half2float(__ushort_as_half((unsigned short)(byte << 7)));
}

// Two channels over their scale -> one byte of codes (lo in the low nibble):
// the hardware conversion rounds to nearest even and saturates; the quotient's
// own rounding moves no value across a code boundary (boundary * scale has at
// most 7 significant bits, exact in fp32).
__device__ __forceinline__ uint32_t kv4_codes(float lo, float hi, float scale) {
  const float a = scale > 0.0f ? __fdiv_rn(lo, scale) : 0.0f;
  const float b = scale > 0.0f ? __fdiv_rn(hi, scale) : 0.0f;
  uint32_t r;
  asm("{\n\t.reg .b8 c;\n\tcvt.rn.satfinite.e2m1x2.f32 c, %2, %1;\n\tmov.b32 %0, {c, 0, 0, 0};\n\t}"
      : "=r"(r)
      : "f"(a), "f"(b));
  return r;
}
// The low byte of codes -> f16x2 (low nibble in the low half), exactly.
__device__ __forceinline__ uint32_t kv4_f16x2(uint32_t codes) {
  uint32_t r;
  asm("{\n\t.reg .b8 c, d, e, f;\n\tmov.b32 {c, d, e, f}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, c;\n\t}" : "=r"(r) : "r"(codes));
  return r;
}
__device__ __forceinline__ float2 kv4_f32x2(uint32_t codes) {
  const uint32_t h = kv4_f16x2(codes);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

}  // namespace m2
