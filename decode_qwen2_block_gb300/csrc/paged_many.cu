// The many-row attention kernels over fp16 pools (paged_many.cuh).
#include "paged_many.cuh"

namespace blk {

cudaError_t launch_paged_many(const PagedManyParams& p, cudaStream_t s, bool pdl) {
  if (p.a.nc < 1 || p.a.nc > 512 || (p.prefix && p.units < 1)) return cudaErrorInvalidValue;
  if (p.a.D == 128)
    return p.prefix ? launch_many<128, true, false>(p, s, pdl) : launch_many<128, false, false>(p, s, pdl);
  if (p.a.D == 64)
    return p.prefix ? launch_many<64, true, false>(p, s, pdl) : launch_many<64, false, false>(p, s, pdl);
  return cudaErrorInvalidValue;
}

cudaError_t configure_paged_many(bool* usable) {
  *usable = true;
  cudaError_t e = configure_one<128, true, false>(usable);
  if (e == cudaSuccess) e = configure_one<128, false, false>(usable);
  if (e == cudaSuccess) e = configure_one<64, true, false>(usable);
  if (e == cudaSuccess) e = configure_one<64, false, false>(usable);
  return e;
}

}  // namespace blk
