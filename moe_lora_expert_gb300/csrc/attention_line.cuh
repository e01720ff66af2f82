// What the two attention kernels share: a line of work cut into equal
// stretches, and the end of a wait.  These are called once a unit, or when
// there is nothing else to do, and are not inlined: the kernels' loops need
// the instruction cache.
#pragma once

#include "attention.cuh"
#include "ptx.cuh"

namespace moe {

// The line of ``total`` places in ``ctas`` equal stretches: where one begins, and which holds place y.
static __device__ __noinline__ int stretch_begin(int total, int ctas, int cta) {
  return static_cast<int>(static_cast<int64_t>(total) * cta / ctas);
}
static __device__ __noinline__ int stretch_of(int total, int ctas, int y) {
  int cta = static_cast<int>(static_cast<int64_t>(y) * ctas / total);
  while (cta + 1 < ctas && stretch_begin(total, ctas, cta + 1) <= y) ++cta;
  while (stretch_begin(total, ctas, cta) > y) --cta;
  return cta;
}
static __device__ __noinline__ bool wait_long(uint64_t* bar, uint32_t parity, uint64_t limit_ns, int* status, int* abort_flag) {
  if (*static_cast<volatile int*>(abort_flag) != 0) return false;
  if (mbar_wait(bar, parity, limit_ns)) return true;
  set_status(status, MOE_ERR_DEVICE_TIMEOUT);
  *static_cast<volatile int*>(abort_flag) = 1;
  return false;
}

}  // namespace moe
