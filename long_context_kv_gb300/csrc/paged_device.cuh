// Taking free pages in ascending order, for the kernels that plan.
#pragma once

#include "paged_internal.cuh"

namespace paris {
namespace {

constexpr int kPlanThreads = 1024;

// The `want` lowest free pages (at most those there are): f(r, page) for the
// r-th of them, by any thread, one thread's in ascending order; their bits are
// cleared.  Returns how many there were: fewer than wanted if n_used says that
// more are free than free_bits has (bits past n_pages are no pages).  The whole
// block; tmp: 33 words of shared memory; first: the thread's word of the first
// 1024.
__device__ __forceinline__ uint32_t page_bits(const Paged& c, int w) {
  if (w >= (c.n_pages + 31) / 32) return 0u;
  return c.bits[w] & (32 * w + 32 <= c.n_pages ? kFull : (1u << (c.n_pages & 31)) - 1u);
}
__device__ __forceinline__ uint32_t first_bits(const Paged& c) { return page_bits(c, (int)threadIdx.x); }
template <typename F>
__device__ __forceinline__ uint32_t take_free(const Paged& c, uint32_t want, uint32_t first, uint32_t* tmp, F&& f) {
  const int words = (c.n_pages + 31) / 32;
  uint32_t before = 0, next = first;
  for (int w0 = 0; w0 < words && before < want; w0 += kPlanThreads) {
    const int w = w0 + threadIdx.x;
    const uint32_t word = next;
    next = page_bits(c, w + kPlanThreads);
    uint32_t total, r = block_excl_scan(__popc(word), tmp, &total) + before;
    uint32_t left = word;
    for (; left != 0 && r < want; left &= left - 1) f(r++, 32 * w + __ffs(left) - 1);
    if (left != word) c.bits[w] = left;
    before += total;
  }
  return min(before, want);
}

}  // namespace
}  // namespace paris
