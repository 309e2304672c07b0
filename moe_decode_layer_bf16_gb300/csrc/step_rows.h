// Whether rows [start, stop) of a step's `total` lie among them.  The two come from
// device memory and may be anything: they are compared before their difference is
// taken, which then fits.
#pragma once

#ifdef __CUDACC__
#define MOE_HOST_DEV __host__ __device__ __forceinline__
#else
#define MOE_HOST_DEV inline
#endif

namespace moe {

MOE_HOST_DEV bool step_rows_ok(int start, int stop, int total) {
  return start >= 0 && stop >= start && stop <= total;
}

}  // namespace moe
