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

// Two codes' factors, from the fp16 bits of their two scales.  A code u in the low bits of
// 0x4c00 is 16 + u / 64; times s less 18 s that is (u - 128) s / 64, exact as one fused
// operation while 18 s is an fp16 number: up to s = 3584.  Larger scales (kBig) subtract first.
template <bool kBig>
struct Kv8Unit {
  __half2 mul, add;
  __device__ __forceinline__ explicit Kv8Unit(uint32_t bits) {
    mul = *reinterpret_cast<const __half2*>(&bits);
    add = kBig ? __float2half2_rn(-18.f) : __hmul2(mul, __float2half2_rn(-18.f));
  }
  // the codes that `sel` places, from w
  __device__ __forceinline__ uint32_t operator()(uint32_t w, uint32_t sel) const {
    const uint32_t b = __byte_perm(w, 0x4c4c4c4cu, sel);
    const __half2 x = *reinterpret_cast<const __half2*>(&b);
    const __half2 y = kBig ? __hmul2(__hadd2(x, add), mul) : __hfma2(x, mul, add);
    return *reinterpret_cast<const uint32_t*>(&y);
  }
};
// Whether one of four scale bytes is above 3584's, 0x6b (NaN's is).
__device__ __forceinline__ uint32_t kv8_big_scales(uint32_t w) {      // (bit 7 of a byte says so)
  return (w & 0x7f7f7f7fu) + 0x14141414u;
}

// Codes of a page: (0, y, z), all columns of some slots.
__device__ __forceinline__ void kv8_tma_codes(uint32_t dst, const CUtensorMap* map, int y, int z,
                                          uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}
// 16 bytes by this lane, or zeros; and its arrival on `bar` when all such copies are there.
__device__ __forceinline__ void kv8_copy16(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void kv8_copies_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// The scales of a slot in shared memory: D / 32 bytes.
template <int NB>
__device__ __forceinline__ uint32_t kv8_lds_scales(uint32_t addr) {
  uint32_t v;
  if constexpr (NB == 4) {
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  } else {
    uint16_t h;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(h) : "r"(addr) : "memory");
    v = h;
  }
  return v;
}

}  // namespace blk
