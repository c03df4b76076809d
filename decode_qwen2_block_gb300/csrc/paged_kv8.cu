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
// columns of K and of V, two neighbours a block of 32, so a block's maximum is one exchange
// and a row's codes leave in 16-byte pieces.  Bound by memory, two bytes read and one
// written a value: 32761 rows of 2 heads of 128 9.8 us, 51 MB (5.2 TB/s).
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

// 32 bytes; `wide`: dst is 32-byte aligned (else 16).
__device__ __forceinline__ void store32(__half* dst, const uint32_t* v, bool wide) {
  if (!wide) {
    reinterpret_cast<uint4*>(dst)[0] = make_uint4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<uint4*>(dst)[1] = make_uint4(v[4], v[5], v[6], v[7]);
    return;
  }
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// Slot slot_map[r] to row r of K and V in fp16.  A thread takes 16 columns of K and of V and
// writes whole 32-byte sectors of them; bound by memory, kUnroll items in flight per thread
// (one: 120007 rows 33.3 us; two: 31.8, 5.9 TB/s).
constexpr int kUnroll = 2;
__global__ void __launch_bounds__(kThreads) kv8_read_kernel(const Kv8ReadParams p) {
  griddep_wait();
  griddep_launch();
  const uint32_t cpr = p.D >> 4, per_row = p.Hkv * cpr;
  const int64_t total = (int64_t)p.N * per_row;
  const int64_t step = (int64_t)gridDim.x * kThreads;
  const int64_t mask = ((int64_t)1 << p.page_lg) - 1;
  const bool wide = (reinterpret_cast<uintptr_t>(p.k) | reinterpret_cast<uintptr_t>(p.v)) % 32 == 0 &&
                    (p.row_stride | p.head_stride) % 16 == 0;
  for (int64_t i0 = (int64_t)blockIdx.x * kThreads + threadIdx.x; i0 < total; i0 += step * kUnroll) {
    int64_t at[kUnroll], dst[kUnroll];
    uint32_t c[kUnroll];
    uint4 w[kUnroll][2];
    uint32_t sc[kUnroll][2];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int64_t i = i0 + u * step;
      at[u] = -1;
      if (i < total) {
        const uint32_t r = (uint32_t)i / per_row, e = (uint32_t)i - r * per_row;
        const uint32_t h = e / cpr;
        c[u] = e - h * cpr;
        const int64_t slot = p.slot_map[r];
        dst[u] = (int64_t)r * p.row_stride + h * p.head_stride + c[u] * 16;
        if (slot >= 0 && slot < p.n_slots)
          at[u] = (((slot >> p.page_lg) * p.Hkv + h) << p.page_lg) + (slot & mask);
        else if (slot != -1 && e == 0)
          set_error(p.err, kDevPage);
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      if (at[u] >= 0) {
        const int64_t s = at[u] * (p.D / kKv8Block) + (c[u] >> 1), k = at[u] * p.D + c[u] * 16;
        w[u][0] = __ldcs(reinterpret_cast<const uint4*>(p.from.k + k));
        w[u][1] = __ldcs(reinterpret_cast<const uint4*>(p.from.v + k));
        sc[u][0] = p.from.ks[s];
        sc[u][1] = p.from.vs[s];
      }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      if (at[u] >= 0) {
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          const __half2 unit = kv8_unit(sc[u][kv]);
          const uint32_t x[4] = {w[u][kv].x, w[u][kv].y, w[u][kv].z, w[u][kv].w};
          uint32_t y[8];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            y[2 * k] = kv8_pair(x[k], 0x4140, unit);
            y[2 * k + 1] = kv8_pair(x[k], 0x4342, unit);
          }
          store32((kv ? p.v : p.k) + dst[u], y, wide);
        }
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
