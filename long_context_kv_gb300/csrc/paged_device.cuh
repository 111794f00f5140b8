// Taking free pages in ascending order, for the kernels that plan.
#pragma once

#include "paged_internal.cuh"

namespace paris {
namespace {

constexpr int kPlanThreads = 1024;

// The `want` lowest free pages (at most those there are): f(r, page) for the
// r-th of them, by any thread, one thread's in ascending order; their bits are
// cleared.  The whole block; tmp: 33 words of shared memory; first: the thread's
// word of the first 1024.
__device__ __forceinline__ uint32_t first_bits(const Paged& c) {
  return (int)threadIdx.x < (c.n_pages + 31) / 32 ? c.bits[threadIdx.x] : 0u;
}
template <typename F>
__device__ __forceinline__ void take_free(const Paged& c, uint32_t want, uint32_t first, uint32_t* tmp, F&& f) {
  const int words = (c.n_pages + 31) / 32;
  uint32_t before = 0, next = first;
  for (int w0 = 0; w0 < words && before < want; w0 += kPlanThreads) {
    const int w = w0 + threadIdx.x;
    const uint32_t word = next;
    next = w + kPlanThreads < words ? c.bits[w + kPlanThreads] : 0u;
    uint32_t total, r = block_excl_scan(__popc(word), tmp, &total) + before;
    uint32_t left = word;
    while (left != 0 && r < want) {
      const int page = 32 * w + __ffs(left) - 1;
      if (page < c.n_pages) f(r, page);
      left &= left - 1;
      ++r;
    }
    if (left != word) c.bits[w] = left;
    before += total;
  }
}

}  // namespace
}  // namespace paris
