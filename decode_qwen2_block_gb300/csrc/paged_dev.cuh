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

// First slot that the rows from slot `first` on see here (the shared prefix's
// slots are not a sequence's own).
__device__ __forceinline__ int paged_lo(const PagedAttnParams& p, int first) {
  const int64_t w = window_lo(p.window, first);
  return (int)(w > p.prefix_len ? w : p.prefix_len);
}

}  // namespace blk
