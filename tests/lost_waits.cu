// A kernel source of the library (MOLORA_SOURCE) in which the waits of one warp of one CTA complete and then
// say that their time ran out: what a caller sees after a lost wait can be tested with nothing left in flight.
// MOLORA_SET names the exported function that picks the CTA and the warp (-1: none).
#include "common.cuh"
#include "kernels.h"

namespace molora {
namespace {

struct Lost {
  int cta, warp;
};
__device__ Lost lost = {-1, -1};

__device__ __forceinline__ bool is_lost() {
  return (int)blockIdx.x == lost.cta && (int)(threadIdx.x >> 5) == lost.warp;
}
__device__ __forceinline__ bool lost_wait(uint64_t* bar, uint32_t parity) {
  return mbar_wait(bar, parity) && !is_lost();
}
__device__ __forceinline__ bool lost_wait_spin(uint64_t* bar, uint32_t parity, volatile int32_t* abort) {
  if (!mbar_wait_spin(bar, parity, abort)) return false;
  if (!is_lost()) return true;
  *abort = 1;
  return false;
}

}  // namespace
}  // namespace molora

#define mbar_wait lost_wait
#define mbar_wait_spin lost_wait_spin
#include MOLORA_SOURCE
#undef mbar_wait
#undef mbar_wait_spin

extern "C" MOLORA_API int MOLORA_SET(int cta, int warp) {
  const molora::Lost l = {cta, warp};
  return (int)cudaMemcpyToSymbol(molora::lost, &l, sizeof l);
}
