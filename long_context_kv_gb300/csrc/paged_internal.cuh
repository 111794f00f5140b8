// Internal declarations of the paged cache (include/paris.h, "A cache of
// pages").
#pragma once

#include "kv4_internal.cuh"

namespace paris {

constexpr int kMaxPagedSeqs = 4096;
constexpr int kMaxPagesLog = 21;  // pages of a pool: 2^21
constexpr uint32_t kStatusWrongSeq = 2u;

struct PageStrides {
  int64_t layer, page, head, row;  // bytes
};

// Device view of paris_paged.
struct Paged {
  int n_seqs, layers, hkv, e4m3;
  int shift;  // page_rows = 1 << shift
  int n_pages, width;
  uint8_t *k, *v;
  PageStrides sk, sv;
  uint8_t *ks, *vs;
  int32_t *table, *lens, *starts, *refs;
  uint32_t* bits;
  int32_t* n_used;
  uint32_t* status;
};

__device__ __forceinline__ int paged_cap(const Paged& c) { return c.width << c.shift; }
__device__ __forceinline__ int paged_len(const Paged& c, int s) { return min(max(c.lens[s], 0), paged_cap(c)); }
// Pages of so many rows.
__device__ __forceinline__ int pages_of(const Paged& c, int rows) {
  return (int)(((uint32_t)rows + (1u << c.shift) - 1u) >> c.shift);
}
__device__ __forceinline__ int clamp_page(const Paged& c, int p) { return min(max(p, 0), c.n_pages - 1); }
__device__ __forceinline__ int page_at(const Paged& c, int s, int j) { return clamp_page(c, c.table[(int64_t)s * c.width + j]); }
// A row's scale byte.
__device__ __forceinline__ int64_t scale_at(const Paged& c, int layer, int page, int head, int row) {
  return ((((int64_t)layer * c.n_pages + page) * c.hkv + head) << c.shift) + row;
}

// Two e4m3 codes, of a word's lower or upper half, as halves; every code is
// exact in them.
__device__ __forceinline__ uint32_t e4m3_lo(uint32_t codes) {
  uint32_t y;
  asm("{\n .reg .b16 lo, hi;\n mov.b32 {lo, hi}, %1;\n cvt.rn.f16x2.e4m3x2 %0, lo;\n}\n" : "=r"(y) : "r"(codes));
  return y;
}
__device__ __forceinline__ uint32_t e4m3_hi(uint32_t codes) {
  uint32_t y;
  asm("{\n .reg .b16 lo, hi;\n mov.b32 {lo, hi}, %1;\n cvt.rn.f16x2.e4m3x2 %0, hi;\n}\n" : "=r"(y) : "r"(codes));
  return y;
}

cudaError_t launch_paged_grow(const Paged& c, const int32_t* tokens, cudaStream_t st);

// Rows of a call next to the cache: packed by cu or along a seq stride.
struct PagedRows {
  Paged c;
  int layer, dtype;  // PARIS_F32 or PARIS_BF16
  uint8_t *k, *v;
  Strides ks, vs;  // elements
  int64_t rows, max_rows;
  const int32_t* cu;
};
cudaError_t launch_paged_store(const PagedRows& a, int sm_count, cudaStream_t st);
cudaError_t launch_paged_read(const PagedRows& a, int sm_count, cudaStream_t st);

// An entry of a fork: what the planning kernel tells the applying one.
struct ForkEntry {
  int dst;         // -1: left out
  int src;
  int full;        // pages shared with src
  int last;        // the page behind them that is the destination's own, or -1
  int from, rows;  // its rows [0, rows) are copied from page `from`; rows = 0: nothing is
  int old_pages;   // pages that dst held
  int pad;
};

struct ForkArgs {
  Paged c;
  const int32_t *src, *dst, *rows;
  int n, zero;         // zero: cut to 0 rows where rows is null
  int32_t* entries;    // [n][width] the sources' pages, as they were before the call
  ForkEntry* plan;     // [n]
};
cudaError_t launch_paged_fork(const ForkArgs& a, cudaStream_t st);

struct CompactArgs {
  Paged c;
  int32_t *from, *to;  // [n_pages] the moves
  int32_t* rank;       // [n_pages] a page's move
  int32_t* moves;      // [1] their number
};
cudaError_t launch_paged_compact(const CompactArgs& a, int sm_count, cudaStream_t st);

// A sequence whose attention is computed in several units.
struct PgSplit {
  int s, slot, units, pad;
};
struct PagedAttendPlan {
  int groups, blocks, slots, max_splits;
  size_t part_bytes, bytes;
};
PagedAttendPlan paged_attend_plan(const Paged& c, int hq, int sm_count);

struct PagedAttendArgs {
  Paged c;
  int layer, hq, g;
  int window;  // 0: none
  const __nv_bfloat16* q;
  __nv_bfloat16* out;
  float* lse;  // may be null
  int groups, nblocks, slots, max_splits;
  float* part;       // [slots][hq][kPartStride]
  PgSplit* splits;   // [max_splits]
  uint32_t* counts;  // the queue's next job; sequences of several units; rows to be computed again; blocks that are done with it
};
cudaError_t launch_paged_attend(const PagedAttendArgs& a, cudaStream_t st);
cudaError_t paged_attend_error(uint32_t* bits);

}  // namespace paris
