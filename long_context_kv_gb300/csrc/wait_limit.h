// How long a wait inside a kernel may go on.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define PARIS_HD __host__ __device__ __forceinline__
#else
#define PARIS_HD inline
#endif

namespace paris {

constexpr uint32_t kWaitNs = 4000000000u;  // a wait that takes this long gives up
constexpr uint32_t kLookNs = 20000000u;    // between two looks no more than this counts

// The time that a wait has spent, by the lower half of the nanosecond timer at
// each look.  A block looks every few microseconds while it runs; a longer gap
// means that its process was off the GPU (time slices, a debugger), which says
// nothing of what it waits for.  32 bits hold the limit and one more look.
struct WaitLimit {
  uint32_t last, spent;
  PARIS_HD explicit WaitLimit(uint32_t now) : last(now), spent(0) {}
  PARIS_HD bool over(uint32_t now) {
    const uint32_t gap = now - last;
    spent += gap < kLookNs ? gap : kLookNs;
    last = now;
    return spent > kWaitNs;
  }
};

}  // namespace paris
