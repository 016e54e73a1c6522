// How long a wait inside a kernel has run.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define ROPE_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define ROPE_HOST_DEVICE inline
#endif

namespace rope {

constexpr uint32_t kWaitLimitNs = 2000000000u;  // 2 s; a wait is a few microseconds
constexpr uint32_t kWaitStepNs = 50000000u;

// The limit is of time in which the waiting thread ran.  The clock goes on while the context is
// suspended (another process' turn, a debugger), so between two looks at it no more than kWaitStepNs
// count: a suspension of any length is one step, and a wait runs out after 40 looks at the least.  (32 bits of the
// clock do: what a step of more than 4.2 s loses would not count.)
struct WaitClock {
  uint32_t last, waited;

  ROPE_HOST_DEVICE explicit WaitClock(uint32_t now) : last(now), waited(0) {}

  ROPE_HOST_DEVICE bool expired(uint32_t now) {
    const uint32_t step = now - last;
    waited += step < kWaitStepNs ? step : kWaitStepNs;
    last = now;
    return waited > kWaitLimitNs;
  }
};

}  // namespace rope
