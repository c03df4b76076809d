// Device helpers shared by the paged attention kernels.
#pragma once

#include "common.cuh"
#include "paged.h"

namespace blk {

// mbar_wait for waits that are short and follow one another closely: the timer
// (a slow read) is not consulted before the phase has been probed some times.
__device__ __forceinline__ bool mbar_wait_near(uint64_t* bar, uint32_t parity, int* err) {
#pragma unroll 1
  for (int i = 0; i < 64; ++i)
    if (mbar_try_wait(bar, parity)) return true;
  return mbar_wait(bar, parity, err);
}

// A sequence of the batch as the kernels take it: n = 0 when it has no rows
// or is refused (and then `bad`): its row range, length and pages must fit the
// batch before anything is formed from them.
struct PagedSeq {
  int r0, n, L;
  bool bad;
};
__device__ __forceinline__ PagedSeq load_seq(const PagedAttnParams& p, int b) {
  const int64_t r0 = p.row_start[b], r1 = p.row_start[b + 1], L = p.cache_lens[b];
  PagedSeq s;
  const int64_t n = r1 - r0;
  s.bad = !(r0 >= 0 && r0 <= r1 && r1 <= p.N && n <= p.max_new) ||
          (n > 0 && !(L >= p.prefix_len && L <= p.max_len - n));
  s.n = s.bad ? 0 : (int)n;
  s.r0 = s.n > 0 ? (int)r0 : 0;
  s.L = s.n > 0 ? (int)L : 0;
  return s;
}

// A row's exponents are taken against its maximum x (log2 units) less w, so that weights
// come out 2^w times their size (w: see the kernels).  Not where x is past 2^22, which fp32
// holds to half a unit or worse: there a weight is off by a factor of that size, and needs
// fp16's room for it.
__device__ __forceinline__ bool weight_plain(float x) { return fabsf(x) >= 4194304.f; }

// First slot that a row in slot `last` sees, and first slot that the rows from slot
// `first` on see here (the prefix's slots only where it has no launch of its own).
__device__ __forceinline__ int paged_window(const PagedAttnParams& p, int last) {
  return p.window > 0 && last >= p.window ? last - p.window + 1 : 0;
}
__device__ __forceinline__ int paged_lo(const PagedAttnParams& p, int first) {
  return max(paged_window(p, first), p.own_lo);
}

// T * i / n, the CTA of n that has tile x of T (the greatest i with T * i / n <= x), and
// x / y, of non-negative values, in 32 bits where they fit (a 64-bit division takes
// some 100 clocks or more, and every CTA begins with a few).
__device__ __forceinline__ int64_t range_of(int64_t T, int i, int n) {
  return T < (1 << 20) ? (int64_t)((uint32_t)((uint32_t)T * (uint32_t)i) / (uint32_t)n) : T * i / n;
}
__device__ __forceinline__ int cta_of(int64_t T, int64_t x, int n) {
  return T < (1 << 20) ? (int)(((uint32_t)(x + 1) * (uint32_t)n - 1) / (uint32_t)T)
                       : (int)(((x + 1) * n - 1) / T);
}
__device__ __forceinline__ int small_div(int64_t x, int64_t y) {
  return ((x | y) >> 31) == 0 ? (int)((uint32_t)x / (uint32_t)y) : (int)(x / y);
}

}  // namespace blk
