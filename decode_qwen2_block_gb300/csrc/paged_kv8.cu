// A paged K/V cache in 8 bits: rows quantised into their slots, and slots read back as rows
// (the form of the cache: kv8.h).
#include "common.cuh"
#include "kv8.cuh"
#include "kv8.h"

namespace blk {
namespace {

constexpr int kThreads = 256;

// The codes of 16 values in two vectors of 8, with r = 64 / s.
__device__ __forceinline__ uint4 codes16(const uint4& a, const uint4& b, float r) {
  float f[16];
  h8_to_f32(a, f);
  h8_to_f32(b, f + 8);
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = kv8_pack4(kv8_code(f[4 * i], r), kv8_code(f[4 * i + 1], r), kv8_code(f[4 * i + 2], r),
                     kv8_code(f[4 * i + 3], r));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ uint32_t max_bits16(const uint4& a, const uint4& b) {
  constexpr uint32_t m = 0x7fff7fffu;
  const uint32_t x = kv8_max_bits(kv8_max_bits(a.x & m, a.y & m), kv8_max_bits(a.z & m, a.w & m));
  const uint32_t y = kv8_max_bits(kv8_max_bits(b.x & m, b.y & m), kv8_max_bits(b.z & m, b.w & m));
  return kv8_max_bits(x, y);
}

// Quantises row r's K and V (Hkv heads of D) into slot slot_map[r].  A thread takes 16
// columns of K and of V, two neighbours a block of 32.
__global__ void __launch_bounds__(kThreads) kv8_append_kernel(const Kv8AppendParams p) {
  // (in this order: see page_append_kernel)
  griddep_wait();
  griddep_launch();
  const uint32_t cpr = p.D >> 4;                  // 16-column pieces of a head's row
  const uint32_t per_row = p.Hkv * cpr;
  const int64_t total = (int64_t)p.N * per_row;   // < 2^32: checked by the launcher; even
  const int64_t step = (int64_t)gridDim.x * kThreads;
  const int64_t mask = ((int64_t)1 << p.page_lg) - 1;
  // (a warp stays together: neighbours exchange their maxima)
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i - (threadIdx.x & 31) < total; i += step) {
    const bool here = i < total;
    uint4 k0 = {}, k1 = {}, v0 = {}, v1 = {};
    int64_t slot = -1;
    uint32_t h = 0, c = 0;
    if (here) {
      const uint32_t r = (uint32_t)i / per_row, e = (uint32_t)i - r * per_row;
      h = e / cpr;
      c = e - h * cpr;
      slot = p.slot_map[r];
      const int64_t src = (int64_t)r * p.row_stride + h * p.head_stride + c * 16;
      const uint4* kp = reinterpret_cast<const uint4*>(p.k + src);
      const uint4* vp = reinterpret_cast<const uint4*>(p.v + src);
      k0 = __ldcs(kp); k1 = __ldcs(kp + 1);
      v0 = __ldcs(vp); v1 = __ldcs(vp + 1);
      if (slot != -1 && (slot < 0 || slot >= p.n_slots)) {
        if (e == 0) set_error(p.err, kDevPage);
        slot = -1;
      }
    }
    uint32_t mk = max_bits16(k0, k1), mv = max_bits16(v0, v1);
    mk = kv8_max_bits(mk, __shfl_xor_sync(0xffffffffu, mk, 1));
    mv = kv8_max_bits(mv, __shfl_xor_sync(0xffffffffu, mv, 1));
    const uint32_t sk = kv8_scale(max(mk & 0xffffu, mk >> 16));
    const uint32_t sv = kv8_scale(max(mv & 0xffffu, mv >> 16));
    if (slot >= 0) {
      const int64_t at = (((slot >> p.page_lg) * p.Hkv + h) << p.page_lg) + (slot & mask);
      *reinterpret_cast<uint4*>(p.to.k + at * p.D + c * 16) = codes16(k0, k1, kv8_inverse(sk));
      *reinterpret_cast<uint4*>(p.to.v + at * p.D + c * 16) = codes16(v0, v1, kv8_inverse(sv));
      if (!(c & 1)) {
        const int64_t sat = at * (p.D / kKv8Block) + (c >> 1);
        p.to.ks[sat] = (uint8_t)sk;
        p.to.vs[sat] = (uint8_t)sv;
      }
    }
  }
}

// Slot slot_map[r] to row r of K and V in fp16.  A thread takes 16 columns of K and of V.
__global__ void __launch_bounds__(kThreads) kv8_read_kernel(const Kv8ReadParams p) {
  griddep_wait();
  griddep_launch();
  const uint32_t cpr = p.D >> 4, per_row = p.Hkv * cpr;
  const int64_t total = (int64_t)p.N * per_row;
  const int64_t step = (int64_t)gridDim.x * kThreads;
  const int64_t mask = ((int64_t)1 << p.page_lg) - 1;
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < total; i += step) {
    const uint32_t r = (uint32_t)i / per_row, e = (uint32_t)i - r * per_row;
    const uint32_t h = e / cpr, c = e - h * cpr;
    const int64_t slot = p.slot_map[r];
    if (slot < 0 || slot >= p.n_slots) {
      if (slot != -1 && e == 0) set_error(p.err, kDevPage);
      continue;
    }
    const int64_t at = (((slot >> p.page_lg) * p.Hkv + h) << p.page_lg) + (slot & mask);
    const int64_t sat = at * (p.D / kKv8Block) + (c >> 1);
    const int64_t dst = (int64_t)r * p.row_stride + h * p.head_stride + c * 16;
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      const uint4 w = *reinterpret_cast<const uint4*>((kv ? p.from.v : p.from.k) + at * p.D + c * 16);
      const __half2 u = kv8_unit((kv ? p.from.vs : p.from.ks)[sat]);
      uint4* o = reinterpret_cast<uint4*>((kv ? p.v : p.k) + dst);
      o[0] = make_uint4(kv8_pair(w.x, 0x4140, u), kv8_pair(w.x, 0x4342, u),
                        kv8_pair(w.y, 0x4140, u), kv8_pair(w.y, 0x4342, u));
      o[1] = make_uint4(kv8_pair(w.z, 0x4140, u), kv8_pair(w.z, 0x4342, u),
                        kv8_pair(w.w, 0x4140, u), kv8_pair(w.w, 0x4342, u));
    }
  }
}

template <typename K, typename P>
cudaError_t launch(K kernel, int grid, cudaStream_t s, bool pdl, const P& p) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

int row_grid(int64_t total, int64_t most) {
  const int64_t want = (total + kThreads - 1) / kThreads;
  return (int)(want < 1 ? 1 : (want > most ? most : want));
}

}  // namespace

cudaError_t launch_kv8_append(const Kv8AppendParams& p, int num_sms, cudaStream_t s, bool pdl) {
  const int64_t total = (int64_t)p.N * p.Hkv * (p.D / 16);
  if (total >= (int64_t)1 << 32 || p.D % kKv8Block) return cudaErrorInvalidValue;
  return launch(kv8_append_kernel, row_grid(total, (int64_t)num_sms * 16), s, pdl, p);
}

cudaError_t launch_kv8_read(const Kv8ReadParams& p, int num_sms, cudaStream_t s, bool pdl) {
  const int64_t total = (int64_t)p.N * p.Hkv * (p.D / 16);
  if (total >= (int64_t)1 << 32 || p.D % kKv8Block) return cudaErrorInvalidValue;
  return launch(kv8_read_kernel, row_grid(total, (int64_t)num_sms * 16), s, pdl, p);
}

}  // namespace blk
