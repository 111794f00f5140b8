// Internal declarations of the 4-bit cache and the prompt calls
// (include/paris.h, "The prompt's own attention, and a cache in 4 bits").
#pragma once

#include "paris_device.cuh"

namespace paris {

constexpr int kGroup4 = 32;            // channels that share a scale
constexpr int kCode4 = kDim / 2;       // code bytes of a row
constexpr int kScale4 = kDim / kGroup4;  // scale bytes of a row
constexpr float kLimit4 = 1680.f;      // 7 x 240: the largest value a row holds
constexpr uint32_t kStatusNoRoom = 1u;

// Device view of paris_kv4.
struct Kv4 {
  int batch, hkv;
  int64_t rmax;
  uint8_t *kc, *vc, *ks, *vs;
  float* w;
  int32_t *pos, *lens, *next;
  uint32_t *counters, *status;
};

struct Strides {
  int64_t token, head, seq;
};

__device__ __forceinline__ int64_t kv4_len(const Kv4& c, int b) {
  return min64(max64(c.lens[b], 0), c.rmax);
}

// Rows [start, start + len) of sequence s on a token axis of `rows` rows;
// starts outside the axis, or before the start in front, are clamped.
__device__ __forceinline__ void seq_rows(const int32_t* cu, int s, int64_t rows, int64_t& start, int64_t& len) {
  if (cu == nullptr) {
    start = 0;
    len = rows;
    return;
  }
  start = min64(max64(cu[s], 0), rows);
  len = min64(max64(cu[s + 1], start), rows) - start;
}

// 32 N sequences (N a lane) of so many tiles each are cut into chunks of as
// few tiles as `most` chunks allow: chunk x's sequence (-1: there is no such
// chunk), the first of that sequence's chunks and their number.  A whole warp;
// `most` is at least the number of sequences that have tiles, and all tiles
// together are below 2^32.
template <int N>
__device__ __forceinline__ int3 cut_tiles(const uint32_t (&tiles)[N], uint32_t most, uint32_t x) {
  const int lane = threadIdx.x & 31;
  uint32_t all = 0, longest = 0, seqs = 0, used = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    all += tiles[i];
    longest = max(longest, tiles[i]);
    const uint32_t has = __ballot_sync(kFull, tiles[i] > 0);
    seqs += __popc(has);
    if (has != 0) used |= 1u << i;
  }
  all = __reduce_add_sync(kFull, all);
  longest = __reduce_max_sync(kFull, longest);
  // an even share may be too little, as every sequence has a chunk that is not
  // full; the longest sequence's tiles, or an even share of the other chunks,
  // are enough
  uint32_t lo = max(1u, (all + most - 1) / most), hi = max(lo, longest);
  if (most > seqs) hi = max(lo, min(hi, (all + most - seqs - 1) / (most - seqs)));
  while (lo < hi) {
    const uint32_t mid = lo + (hi - lo) / 2;
    uint32_t n = 0;
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (used >> i & 1u) n += (tiles[i] + mid - 1) / mid;
    if (__reduce_add_sync(kFull, n) <= most) hi = mid;
    else lo = mid + 1;
  }
  uint32_t before = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if ((used >> i & 1u) == 0) continue;
    const uint32_t n = (tiles[i] + lo - 1) / lo;
    const uint32_t inc = warp_incl_scan(n, lane) + before;
    const uint32_t in = __ballot_sync(kFull, x >= inc - n && x < inc);
    if (in != 0) {
      const int src = __ffs(in) - 1;
      return make_int3(32 * i + src, (int)__shfl_sync(kFull, inc - n, src), (int)__shfl_sync(kFull, n, src));
    }
    before = __shfl_sync(kFull, inc, 31);
  }
  return make_int3(-1, 0, 0);
}

struct StoreArgs {
  Kv4 c;
  const void *k, *v;
  int dtype;
  Strides ks, vs;
  int64_t rows, max_new;
  const int32_t* cu;
  const float* weights;
};
cudaError_t launch_kv4_store(const StoreArgs& a, cudaStream_t st);

struct Attend4Args {
  Kv4 c;
  const void* q;
  int dtype, hq, g, accumulate;
  int nblocks;             // chunks of the batch's rows, at most
  float* part;             // [hq][nblocks][kPartStride]
  int2* chunks;            // [batch] first chunk and number of chunks
  float* scores;           // [batch * hq][rmax], base-2 logits (accumulate)
  __nv_bfloat16* out;
};
int kv4_blocks(int batch, int hkv, int g, int64_t rmax, int sm_count);
cudaError_t launch_kv4_attend(const Attend4Args& a, cudaStream_t st);

struct EvictArgs {
  Kv4 c;
  int64_t keep, sink, recent;
  int32_t* list;  // [batch * hkv][2][rmax]: dropped rows below keep, kept rows above
};
cudaError_t launch_kv4_evict(const EvictArgs& a, cudaStream_t st);

cudaError_t launch_kv4_read(const Kv4& c, __nv_bfloat16* k_out, __nv_bfloat16* v_out, int64_t rows, cudaStream_t st);

// The sequences of a prompt call (paris_prompt without its pointers' types).
struct PromptArgs {
  int n_seqs, hq, hkv, g;
  int64_t rows_q, rows_k;
  const int32_t *cu_q, *cu_k;
  int64_t max_q, max_k;
  Strides sq, sk, sv, so;
  const __nv_bfloat16 *q, *k, *v;
  __nv_bfloat16* out;
  float* lse;  // may be null
  float* ws;   // partials of shared units
  int nsplit;  // blocks that may share a unit of rows; 1: none do
};
cudaError_t launch_prompt_attend(const PromptArgs& a, int sm_count, cudaStream_t st);
size_t prompt_workspace_bytes(PromptArgs& a, int sm_count);  // sets a.nsplit

// Whether a wait of the kernels gave up (read and cleared).
cudaError_t prompt_attend_error(uint32_t* bits);
cudaError_t prompt_weights_error(uint32_t* bits);

struct PromptWeightArgs {
  PromptArgs p;
  const float* lse;
  int window;
  float* weights;
};
cudaError_t launch_prompt_weights(const PromptWeightArgs& a, int sm_count, cudaStream_t st);

// Text of the last error without a context (paris_last_error(NULL)).
void set_thread_error(const char* text);

}  // namespace paris
