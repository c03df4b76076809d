// The many-row attention kernels over 8-bit pools (paged_many.cuh).
#include "paged_many.cuh"

namespace blk {

cudaError_t launch_paged_many_kv8(const PagedMany8Params& p, cudaStream_t s, bool pdl) {
  if (p.a.nc < 1 || p.a.nc > 512 || (p.prefix && p.units < 1)) return cudaErrorInvalidValue;
  if (p.a.D == 128)
    return p.prefix ? launch_many<128, true, true>(p, s, pdl) : launch_many<128, false, true>(p, s, pdl);
  if (p.a.D == 64)
    return p.prefix ? launch_many<64, true, true>(p, s, pdl) : launch_many<64, false, true>(p, s, pdl);
  return cudaErrorInvalidValue;
}

cudaError_t configure_paged_many_kv8(bool* usable) {
  *usable = true;
  cudaError_t e = configure_one<128, true, true>(usable);
  if (e == cudaSuccess) e = configure_one<128, false, true>(usable);
  if (e == cudaSuccess) e = configure_one<64, true, true>(usable);
  if (e == cudaSuccess) e = configure_one<64, false, true>(usable);
  return e;
}

}  // namespace blk
