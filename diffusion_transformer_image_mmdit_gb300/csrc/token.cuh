// Device helpers of the token step's kernels (token_linear.cu, kv_cache.cu).
#pragma once

#include "common.cuh"

namespace mmdit {

// Two values to e4m3 codes, the first in the low byte.
__device__ __forceinline__ uint16_t f8x2_e4m3(float lo, float hi) {
  uint16_t d;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
  return d;
}

// A kernel launched by launch_after (capi_util.h) may be on the SMs before the
// one in front of it in the stream has ended.  It begins with `grid_wait`,
// before its first access to global memory: everything in front has ended and
// is visible then.  Only behind that does it let the next kernel start
// (`grid_release`), so that whatever comes on early finds all but its direct
// predecessor ended.
// What such a kernel reads may thus be written while it is resident: it uses no
// non-coherent loads (__ldg, ld.global.nc), which are for data that nobody
// writes during the whole kernel and which the compiler may raise above the
// wait.
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_release() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

}  // namespace mmdit
