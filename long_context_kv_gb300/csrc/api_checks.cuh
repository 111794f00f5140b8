// What the entry points without a context share: their errors and the checks
// of what several of them take.
#pragma once

#include <atomic>
#include <cstdarg>
#include <cstdio>

#include "../../include/paris.h"
#include "kv4_internal.cuh"

namespace paris {
namespace {

inline paris_status fail(paris_status st, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  set_thread_error(buf);
  return st;
}

inline paris_status launched(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return PARIS_OK;
  cudaGetLastError();  // reported here, not by the caller's next call
  return fail(PARIS_ECUDA, "%s: %s", what, cudaGetErrorString(e));
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline int sm_count() {
  // asked once per device: the attribute cannot change
  static std::atomic<int> cached[64];
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return 148;
  if (dev < 64 && cached[dev] > 0) return cached[dev];
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    cudaGetLastError();
    return 148;
  }
  if (dev < 64) cached[dev] = n;
  return n;
}

// Strides of an axis of more than one entry have to be positive multiples of
// 8 elements; those of an axis of one entry mean nothing and are replaced.
inline paris_status take_strides(const paris_strides& s, int64_t tokens, int heads, int seqs, const char* name, Strides* out) {
  const struct { int64_t stride, n; const char* axis; int64_t* to; } axes[3] = {
      {s.token, tokens, "token", &out->token}, {s.head, heads, "head", &out->head}, {s.seq, seqs, "seq", &out->seq}};
  for (const auto& x : axes) {
    if (x.n <= 1) {
      *x.to = kDim;
      continue;
    }
    // sequences may be further apart: tensor maps take 2^40 bytes
    const int64_t most = x.to == &out->seq ? (int64_t)1 << 38 : (int64_t)1 << 31;
    if (x.stride < kDim || x.stride % 8 || x.stride >= most)
      return fail(PARIS_EINVAL, "%s: the %s stride must be a multiple of 8 elements, from %d to below %lld (got %lld)", name,
                  x.axis, kDim, (long long)most, (long long)x.stride);
    *x.to = x.stride;
  }
  return PARIS_OK;
}

inline paris_status check_dtype(paris_dtype t) {
  return t == PARIS_F32 || t == PARIS_BF16 ? PARIS_OK : fail(PARIS_EINVAL, "dtype must be PARIS_F32 or PARIS_BF16");
}

}  // namespace
}  // namespace paris
