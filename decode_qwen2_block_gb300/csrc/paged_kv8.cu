// A paged K/V cache in 8 bits: rows quantised into their slots, slots read back as rows,
// and attention over them (the form of the cache: kv8.h).
#include <math.h>

#include "common.cuh"
#include "kv8.cuh"
#include "kv8.h"
#include "paged_dev.cuh"

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

// out[r, h] = softmax(q[r, h] . K / sqrt(D)) V over the slots that row r sees: a warp a
// (row, head), a lane D / 32 columns, a slot at a time with the running maximum and sum.
template <int D>
__global__ void __launch_bounds__(kThreads) kv8_attn_kernel(const __grid_constant__ Kv8AttnParams p) {
  griddep_wait();
  griddep_launch();
  constexpr int C = D / 32;
  const PagedAttnParams& a = p.a;
  const int lane = threadIdx.x & 31;
  const int64_t warps = (int64_t)gridDim.x * (kThreads / 32);
  if (blockIdx.x == 0)
    for (int b = threadIdx.x; b < a.B; b += kThreads)
      if (load_seq(a, b).bad) set_error(a.err, kDevPage);
  for (int64_t i = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
       i < (int64_t)a.N * a.Hq; i += warps) {
    const int r = (int)(i / a.Hq), h = (int)(i - (int64_t)r * a.Hq), g = h / a.G;
    int b = 0, t = -1, L = 0;
    for (; b < a.B; ++b) {
      const PagedSeq s = load_seq(a, b);
      if (s.n > 0 && r >= s.r0 && r < s.r0 + s.n) {
        t = r - s.r0;
        L = s.L;
        break;
      }
    }
    if (t < 0) continue;
    const int last = L + t, low = paged_window(a, last);
    float q[C], o[C], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int k = 0; k < C; ++k) {
      q[k] = __half2float(a.q[(int64_t)r * a.q_stride + (int64_t)h * D + lane * C + k]);
      o[k] = 0.f;
    }
    // 64 slots at a time, whose sums then join the others: one by one, 32,000 weights of
    // e^-15 added to a sum of 1 would each be off by a sixth
    for (int s0 = low; s0 <= last; s0 += 64) {
      float mc = -INFINITY, lc = 0.f, oc[C];
#pragma unroll
      for (int k = 0; k < C; ++k) oc[k] = 0.f;
      for (int s = s0; s < s0 + 64 && s <= last; ++s) {
        const int32_t* row = s < a.prefix_len ? a.prefix_pages : a.table + (int64_t)b * a.max_blocks;
        const int64_t page = row[s >> a.page_lg];
        const bool in = page >= 0 && page < a.n_pages;
        if (!in && lane == 0) set_error(a.err, kDevPage);
        const int64_t at = in ? ((page * a.Hkv + g) << a.page_lg) + (s & ((1 << a.page_lg) - 1)) : 0;
        const float uk = in ? __low2float(kv8_unit(p.from.ks[at * C + lane * C / 32])) : 0.f;
        const float uv = in ? __low2float(kv8_unit(p.from.vs[at * C + lane * C / 32])) : 0.f;
        float x = 0.f;
#pragma unroll
        for (int k = 0; k < C; ++k) x = fmaf(q[k], (p.from.k[at * D + lane * C + k] - 128) * uk, x);
        x = warp_sum(x) * a.scale_log2;
        const float mn = fmaxf(mc, x);
        const float f = mc == -INFINITY ? 0.f : exp2f(mc - mn);
        const float w = mn == -INFINITY && x == x ? 0.f : exp2f(x - mn);
        lc = lc * f + w;
#pragma unroll
        for (int k = 0; k < C; ++k) oc[k] = oc[k] * f + w * ((p.from.v[at * D + lane * C + k] - 128) * uv);
        mc = mn;
      }
      const float mn = fmaxf(m, mc);
      const float f = m == -INFINITY ? 0.f : exp2f(m - mn), w = mc == -INFINITY ? 1.f : exp2f(mc - mn);
      l = l * f + lc * w;
#pragma unroll
      for (int k = 0; k < C; ++k) o[k] = o[k] * f + oc[k] * w;
      m = mn;
    }
    const float inv = l > 0.f ? 1.f / l : (l == l ? 0.f : l);
#pragma unroll
    for (int k = 0; k < C; ++k)
      a.out[(int64_t)r * a.out_stride + (int64_t)h * D + lane * C + k] = __float2half_rn(o[k] * inv);
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

cudaError_t launch_kv8_attn(const Kv8AttnParams& p, cudaStream_t s, bool pdl) {
  const int grid = row_grid((int64_t)p.a.N * p.a.Hq * 32, 4096);
  if (p.a.D == 128) return launch(kv8_attn_kernel<128>, grid, s, pdl, p);
  if (p.a.D == 64) return launch(kv8_attn_kernel<64>, grid, s, pdl, p);
  return cudaErrorInvalidValue;
}

}  // namespace blk
