// Device helpers of the 8-bit K/V cache: scales, codes and their fp16 values (see kv8.h).
#pragma once

#include "common.cuh"
#include "kv8.h"

namespace blk {

constexpr uint32_t kKv8ScaleNan = 0x7f;    // upper byte of an fp16 NaN

// The greater of two pairs of fp16 magnitudes as bits: an infinity or NaN wins.
__device__ __forceinline__ uint32_t kv8_max_bits(uint32_t a, uint32_t b) { return __vmaxu2(a, b); }

// The scale of a block whose greatest magnitude has the fp16 bits `amax`.
__device__ __forceinline__ uint32_t kv8_scale(uint32_t amax) {
  if (amax >= 0x7c00u) return kKv8ScaleNan;
  // 64 a / 127 from above, up to the next E5M2 number: the scale, or where the product
  // rounded past an exact one, the number behind it
  const float a = __half2float(__ushort_as_half((unsigned short)amax));
  const unsigned short up = __half_as_ushort(__float2half_ru(__fmul_ru(a, 64.0f / 127.0f)));
  const uint32_t b = (up + 0xffu) >> 8;
  if (b == 0) return 0;
  const float less = __half2float(__ushort_as_half((unsigned short)((b - 1) << 8)));
  return 127.0f * less >= 64.0f * a ? b - 1 : b;      // (both products exact)
}

// 64 / s; 0 for a block of zeros, whose codes are all 128.
__device__ __forceinline__ float kv8_inverse(uint32_t scale) {
  return scale == 0 ? 0.f : __frcp_rn(__half2float(__ushort_as_half((unsigned short)(scale << 8)))) * 64.f;
}

// x's code in the low byte.  q = 64 x / s is x's 11 bits over 3 bits: half way between two
// codes, or 2^-12 or more away from that.  x r is at most 127 * 2^-24 off q, so rounded to
// 2^-14 (at 768) it is half way exactly where q is, and the second sum rounds as the
// definition does, ties to even.
__device__ __forceinline__ uint32_t kv8_code(float x, float r) {
  return __float_as_uint(__fadd_rn(__fmaf_rn(x, r, 768.f), 12582912.f - 768.f + 128.f));
}

// The low bytes of four words.
__device__ __forceinline__ uint32_t kv8_pack4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

// s / 64 in both halves, from a scale byte (exact).
__device__ __forceinline__ __half2 kv8_unit(uint32_t scale) {
  const uint32_t h = (scale << 8) | (scale << 24);
  return __hmul2(*reinterpret_cast<const __half2*>(&h), __float2half2_rn(1.f / 64.f));
}

// Two codes, in the bytes of w that `sel` places (0x4140 or 0x4342), times u: 1024 + code
// less 1152 is exact, and so is the product.
__device__ __forceinline__ uint32_t kv8_pair(uint32_t w, uint32_t sel, __half2 u) {
  const uint32_t x = __byte_perm(w, 0x64646464u, sel);
  const __half2 c = __hsub2(*reinterpret_cast<const __half2*>(&x), __float2half2_rn(1152.f));
  const __half2 y = __hmul2(c, u);
  return *reinterpret_cast<const uint32_t*>(&y);
}

}  // namespace blk
