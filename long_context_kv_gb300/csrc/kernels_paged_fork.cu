// The paged cache: sequences that fork, end or are cut, and a pool that is
// closed up.
//
// What a fork reads (the sources' pages) may be what it changes, so it has
// three steps: the first shares the full pages and notes the sources' entries,
// the second decides on the pages that are not full and takes free ones for
// their copies, the third gives back what the destinations held, writes their
// entries and copies rows.  Counts change by sums only, so their order does not
// matter.  All of it is bound by latency: small forks are one block that takes
// the steps in turn (one sequence to four: 8.3 us, 9.8 as three kernels),
// larger ones a kernel a step (64 beams: 11.3 us), and sequences that end need
// none of the first two (3 us).
#include "paged_device.cuh"

namespace paris {
namespace {

constexpr int kSegment = 1024;  // entries of a block
constexpr int kForkThreads = 256;

__device__ __forceinline__ bool in_range(const Paged& c, int s) { return s >= 0 && s < c.n_seqs; }

__device__ __forceinline__ int fork_rows(const ForkArgs& a, int i, int src) {
  const int len = paged_len(a.c, src);
  return a.rows != nullptr ? min(len, max(a.rows[i], 0)) : a.zero ? 0 : len;
}

// Pages [j0, j1) of entry i's source, by `lanes` threads: those that are full
// are shared.  (Of a sequence that stays itself nothing is shared and nothing
// given back.)
__device__ __forceinline__ void share_pages(const ForkArgs& a, int i, int src, int full, int j0, int j1, int lane, int lanes) {
#pragma unroll 4
  for (int j = j0 + lane; j < j1; j += lanes) {
    const int p = page_at(a.c, src, j);
    a.entries[(int64_t)i * a.c.width + j] = p;
    if (j < full) atomicAdd(&a.c.refs[p], 1);
  }
}

__global__ void __launch_bounds__(kForkThreads) k_paged_fork_share(ForkArgs a) {
  pdl_wait();
  pdl_trigger();
  const int i = blockIdx.x, src = a.src[i], dst = a.dst[i];
  if (!in_range(a.c, src) || !in_range(a.c, dst)) return;
  const int rows = fork_rows(a, i, src), pages = pages_of(a.c, rows), j0 = blockIdx.y * kSegment;
  if (src == dst || j0 >= pages) return;
  bool twice = false;
  for (int t = threadIdx.x; t < i; t += kForkThreads) twice |= a.dst[t] == dst && in_range(a.c, a.src[t]);
  if (__syncthreads_or(twice)) return;
  share_pages(a, i, src, rows >> a.c.shift, j0, min(j0 + kSegment, pages), threadIdx.x, kForkThreads);
}

// Entries [j0, j1) of a destination, by `lanes` threads: what they held is
// given back; the number of pages that nobody holds any more.
__device__ __forceinline__ int replace_pages(const ForkArgs& a, int i, const ForkEntry& e, int j0, int j1, int lane, int lanes) {
  const bool self = e.src == e.dst;
  int gone = 0;
#pragma unroll 4
  for (int j = (self ? max(j0, e.full) : j0) + lane; j < min(j1, max(e.old_pages, e.full + 1)); j += lanes) {
    int32_t* entry = a.c.table + (int64_t)e.dst * a.c.width + j;
    const int old = clamp_page(a.c, *entry);
    if (self && j == e.full && e.last == old) continue;  // it stays
    if (j < e.full) *entry = a.entries[(int64_t)i * a.c.width + j];
    else if (j == e.full && e.last >= 0) *entry = e.last;
    if (j < e.old_pages && atomicSub(&a.c.refs[old], 1) == 1) {
      atomicOr(&a.c.bits[old >> 5], 1u << (old & 31));
      ++gone;
    }
  }
  return gone;
}

// Four rows [r0, min(r0 + 4, rows)) of one layer, head and side (keys 0, values
// 1) from a page to another: 16 lanes, 8 channels each, all loads before the
// stores.
__device__ __forceinline__ void copy_four(const Paged& c, int layer, int head, int side, int from, int to, int r0, int rows, int l16) {
  const PageStrides& st = side ? c.sv : c.sk;
  uint8_t* p = (side ? c.v : c.k) + layer * st.layer + head * st.head + r0 * st.row;
  const uint8_t* x = p + from * st.page;
  uint8_t* y = p + to * st.page;
  if (!c.e4m3) {
    uint4 w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (r0 + i < rows) w[i] = reinterpret_cast<const uint4*>(x + i * st.row)[l16];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (r0 + i < rows) reinterpret_cast<uint4*>(y + i * st.row)[l16] = w[i];
    return;
  }
  uint8_t* s = side ? c.vs : c.ks;
  const int64_t sx = scale_at(c, layer, from, head, r0), sy = scale_at(c, layer, to, head, r0);
  uint2 w[4];
  uint8_t byte = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (r0 + i < rows) w[i] = reinterpret_cast<const uint2*>(x + i * st.row)[l16];
  if (l16 < 4 && r0 + l16 < rows) byte = s[sx + l16];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (r0 + i < rows) reinterpret_cast<uint2*>(y + i * st.row)[l16] = w[i];
  if (l16 < 4 && r0 + l16 < rows) s[sy + l16] = byte;
}

// The rows of entry e's last page in one layer, by `groups` groups of 16 lanes.
__device__ __forceinline__ void copy_rows(const ForkArgs& a, const ForkEntry& e, int layer, int group, int groups) {
  const int fours = (e.rows + 3) / 4, items = 2 * a.c.hkv * fours;
  for (int it = group; it < items; it += groups) {
    const int hv = it / fours;
    copy_four(a.c, layer, hv >> 1, hv & 1, e.from, e.last, 4 * (it - hv * fours), e.rows, threadIdx.x & 15);
  }
}

// kAll: the whole of a small fork.
template <bool kAll>
__global__ void __launch_bounds__(kPlanThreads) k_paged_fork_plan(ForkArgs a) {
  __shared__ int owner[kMaxPagedSeqs];  // the first entry of a destination; then the entries that take a page, in order
  __shared__ uint32_t tmp[33];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t n_free = (uint32_t)max(a.c.n_pages - max(a.c.n_used[0], 0), 0);
  const uint32_t bits = first_bits(a.c);
  for (int s = tid; s < a.c.n_seqs; s += kPlanThreads) owner[s] = 0x7fffffff;
  __syncthreads();
  bool wrong = false, short_of = false;
  for (int i = tid; i < a.n; i += kPlanThreads) {
    const bool ok = in_range(a.c, a.src[i]) && in_range(a.c, a.dst[i]);
    if (ok) atomicMin(&owner[a.dst[i]], i);
    wrong |= !ok;
  }
  __syncthreads();
  if constexpr (kAll) {
    if (a.src != a.dst) {
      for (int i = warp; i < a.n; i += kPlanThreads / 32) {
        const int src = a.src[i], dst = a.dst[i];
        if (!in_range(a.c, src) || !in_range(a.c, dst) || src == dst || owner[dst] != i) continue;
        const int rows = fork_rows(a, i, src);
        share_pages(a, i, src, rows >> a.c.shift, 0, pages_of(a.c, rows), lane, 32);
      }
      __syncthreads();
    }
  }
  uint32_t copies = 0;
  int lens[kMaxPagedSeqs / kPlanThreads], takes[kMaxPagedSeqs / kPlanThreads];  // of this thread's entries
#pragma unroll
  for (int u = 0; u < kMaxPagedSeqs / kPlanThreads; ++u) {
    const int i = u * kPlanThreads + tid;
    if (u * kPlanThreads >= a.n) break;
    ForkEntry e = {-1, -1, 0, -1, 0, 0, 0, 0};
    bool copy = false;
    int rows = 0;
    if (i < a.n) {
      const int src = a.src[i], dst = a.dst[i];
      if (in_range(a.c, src) && in_range(a.c, dst) && owner[dst] == i) {
        rows = fork_rows(a, i, src);
        e.dst = dst;
        e.src = src;
        e.full = rows >> a.c.shift;
        e.rows = rows & ((1 << a.c.shift) - 1);
        e.old_pages = pages_of(a.c, paged_len(a.c, dst));
        if (e.rows != 0) {
          e.from = page_at(a.c, src, e.full);
          if (src == dst && a.c.refs[e.from] == 1) {
            e.last = e.from;  // it stays where it is
            e.rows = 0;
          } else {
            copy = true;
          }
        }
      }
    }
    uint32_t total;
    const uint32_t r = block_excl_scan(copy ? 1u : 0u, tmp, &total) + copies;
    if (copy && r >= n_free) {
      rows = e.full << a.c.shift;
      e.rows = 0;
      copy = false;
      short_of = true;
    }
    if (i < a.n) a.plan[i] = e;
    lens[u] = rows;
    takes[u] = copy ? (int)r : -1;
    copies += total;
  }
  __syncthreads();  // every length and owner has been read
#pragma unroll
  for (int u = 0; u < kMaxPagedSeqs / kPlanThreads; ++u) {
    const int i = u * kPlanThreads + tid;
    if (i >= a.n) break;
    const int dst = a.plan[i].dst;
    if (dst >= 0) a.c.lens[dst] = a.c.starts[dst] = lens[u];
    if (takes[u] >= 0) owner[takes[u]] = i;
  }
  if (wrong) atomicOr(a.c.status, kStatusWrongSeq);
  if (short_of) atomicOr(a.c.status, kStatusNoRoom);
  const uint32_t wanted = min(copies, n_free);
  uint32_t taken = 0;
  if (wanted != 0) {
    __syncthreads();
    taken = take_free(a.c, wanted, bits, tmp, [&](uint32_t r, int page) {
      a.plan[owner[r]].last = page;
      a.c.refs[page] = 1;
    });
  }
  if (taken < wanted) {  // n_used and free_bits do not agree: the entries that got no page keep their full ones
#pragma unroll
    for (int u = 0; u < kMaxPagedSeqs / kPlanThreads; ++u) {
      const int i = u * kPlanThreads + tid;
      if (i >= a.n) break;
      if (takes[u] < (int)taken) continue;
      a.plan[i].rows = 0;
      a.c.lens[a.plan[i].dst] = a.c.starts[a.plan[i].dst] = a.plan[i].full << a.c.shift;
    }
    if (tid == 0) atomicOr(a.c.status, kStatusNoRoom);
  }
  if constexpr (!kAll) {
    if (tid == 0 && taken != 0) a.c.n_used[0] = max(a.c.n_used[0], 0) + (int)taken;
  } else {
    __shared__ int gone;
    if (tid == 0) gone = 0;
    __syncthreads();
    int mine = 0;
    for (int i = warp; i < a.n; i += kPlanThreads / 32) {
      const ForkEntry e = a.plan[i];
      if (e.dst >= 0) mine += replace_pages(a, i, e, 0, a.c.width, lane, 32);
    }
    if (mine != 0) atomicAdd(&gone, mine);
    if (taken != 0) {
      // (entry, layer) items over the warps, the last ones first as the others have entries to replace; several warps an
      // item where there are fewer of them
      const int items = a.n * a.c.layers, each = max(kPlanThreads / 32 / items, 1), w = kPlanThreads / 32 - 1 - warp;
      for (int il = w / each; il < items; il += kPlanThreads / 32) {
        const ForkEntry e = a.plan[il / a.c.layers];
        if (e.dst >= 0 && e.rows != 0) copy_rows(a, e, il % a.c.layers, w % each * 2 + (lane >> 4), 2 * each);
      }
    }
    __syncthreads();
    if (tid == 0) a.c.n_used[0] = max(a.c.n_used[0], 0) + (int)taken - gone;
  }
}

// Blocks [0, n segs): entries; behind them `per` blocks for each (entry,
// layer) copy rows.
__global__ void __launch_bounds__(kForkThreads) k_paged_fork_apply(ForkArgs a, int segs, int per) {
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x;
  if ((int)blockIdx.x < a.n * segs) {
    const int i = blockIdx.x / segs, j0 = (blockIdx.x - i * segs) * kSegment;
    const ForkEntry e = a.plan[i];
    if (e.dst < 0) return;
    const int gone = __reduce_add_sync(kFull, replace_pages(a, i, e, j0, min(j0 + kSegment, a.c.width), tid, kForkThreads));
    if ((tid & 31) == 0 && gone != 0) atomicSub(a.c.n_used, gone);
    return;
  }
  const int x = blockIdx.x - a.n * segs, il = x / per, i = il / a.c.layers;
  const ForkEntry e = a.plan[i];
  if (e.dst < 0 || e.rows == 0) return;
  copy_rows(a, e, il - i * a.c.layers, (x - il * per) * (kForkThreads / 16) + (tid >> 4), per * (kForkThreads / 16));
}

// Sequences that end: a block each.
__global__ void __launch_bounds__(kForkThreads) k_paged_end(ForkArgs a) {
  pdl_wait();
  pdl_trigger();
  const int i = blockIdx.x, tid = threadIdx.x, dst = a.dst[i];
  if (!in_range(a.c, dst)) {
    if (tid == 0) atomicOr(a.c.status, kStatusWrongSeq);
    return;
  }
  bool twice = false;
  for (int t = tid; t < i; t += kForkThreads) twice |= a.dst[t] == dst;
  ForkEntry e = {dst, dst, 0, -1, 0, 0, pages_of(a.c, paged_len(a.c, dst)), 0};
  if (__syncthreads_or(twice)) return;  // (and its length has been read)
  const int gone = __reduce_add_sync(kFull, replace_pages(a, i, e, 0, a.c.width, tid, kForkThreads));
  if ((tid & 31) == 0 && gone != 0) atomicSub(a.c.n_used, gone);
  if (tid == 0) a.c.lens[dst] = a.c.starts[dst] = 0;
}

// One block: the pages in use are counted, as free_bits has them; then those past
// their number and the free ones below it, in ascending order, by one scan of both
// counts (at most 2^15 a round, in the halves of a word); the bits as they are
// afterwards.
__global__ void __launch_bounds__(kPlanThreads) k_paged_compact_plan(CompactArgs a) {
  __shared__ uint32_t tmp[33], counts[kPlanThreads / 32];
  pdl_wait();
  pdl_trigger();
  const int words = (a.c.n_pages + 31) / 32, lane = threadIdx.x & 31;
  const uint32_t first = first_bits(a.c);
  uint32_t mine = __popc(first);
  for (int w = kPlanThreads + threadIdx.x; w < words; w += kPlanThreads) mine += __popc(page_bits(a.c, w));
  mine = __reduce_add_sync(kFull, mine);
  if (lane == 0) counts[threadIdx.x >> 5] = mine;
  __syncthreads();
  const int used = a.c.n_pages - (int)__reduce_add_sync(kFull, counts[lane]);
  uint32_t low = 0, high = 0;
  for (int w0 = 0; w0 < words; w0 += kPlanThreads) {
    const int w = w0 + threadIdx.x, p0 = 32 * w;
    const uint32_t is_page = p0 + 32 <= a.c.n_pages ? kFull : p0 < a.c.n_pages ? (1u << (a.c.n_pages - p0)) - 1u : 0u;
    const uint32_t below = p0 + 32 <= used ? kFull : p0 < used ? (1u << (used - p0)) - 1u : 0u;
    const uint32_t free = w0 == 0 ? first : page_bits(a.c, w);
    uint32_t l = free & below, h = ~free & is_page & ~below, total;
    const uint32_t at = block_excl_scan((uint32_t)__popc(l) | (uint32_t)__popc(h) << 16, tmp, &total);
    uint32_t rl = low + (at & 0xffffu), rh = high + (at >> 16);
    for (; l != 0; l &= l - 1) a.to[rl++] = p0 + __ffs(l) - 1;
    for (; h != 0; h &= h - 1) {
      const int p = p0 + __ffs(h) - 1;
      a.rank[p] = (int)rh;
      a.from[rh++] = p;
    }
    if (w < words) a.c.bits[w] = is_page & ~below;
    low += total & 0xffffu;
    high += total >> 16;
  }
  if (threadIdx.x == 0) a.c.n_used[0] = used;
  if (threadIdx.x == 0) a.moves[0] = (int)min(low, high);
}

// The moves, four rows an item of 16 threads; counts and entries follow.  Bound
// by the bytes: 2000 pages of 64 KB in two layers (517 MB read and written)
// 75 us, 6.9 TB/s; one row at a time 88.
__global__ void __launch_bounds__(kForkThreads) k_paged_compact_move(CompactArgs a) {
  pdl_wait();
  pdl_trigger();
  const int moves = a.moves[0], tid = threadIdx.x, l16 = tid & 15;
  if (moves == 0) return;
  const int64_t threads = (int64_t)gridDim.x * kForkThreads, me = (int64_t)blockIdx.x * kForkThreads + tid;
  const int used = min(max(a.c.n_used[0], 0), a.c.n_pages);
  for (int64_t i = me; i < moves; i += threads) {
    const int p = a.from[i];
    a.c.refs[a.to[i]] = a.c.refs[p];
    a.c.refs[p] = 0;
  }
  for (int64_t i = me; i < (int64_t)a.c.n_seqs * a.c.width; i += threads) {
    const int s = (int)(i / a.c.width);
    if (i - (int64_t)s * a.c.width >= pages_of(a.c, paged_len(a.c, s))) continue;
    const int p = clamp_page(a.c, a.c.table[i]);
    if (p < used) continue;
    const int r = a.rank[p];  // of a page that is not held anything
    if (r >= 0 && r < moves && a.from[r] == p) a.c.table[i] = a.to[r];
  }
  // four rows an item
  const int part = a.c.shift - 2;
  const int64_t items = ((int64_t)moves * a.c.layers * 2 * a.c.hkv) << part;
  for (int64_t it = me >> 4; it < items; it += threads >> 4) {
    const int64_t u = it >> part, lm = u / (2 * a.c.hkv);
    const int hv = (int)(u - lm * 2 * a.c.hkv), m = (int)(lm / a.c.layers);
    copy_four(a.c, (int)(lm - (int64_t)m * a.c.layers), hv >> 1, hv & 1, a.from[m], a.to[m], 4 * ((int)it & ((1 << part) - 1)),
              1 << a.c.shift, l16);
  }
}

}  // namespace

cudaError_t launch_paged_fork(const ForkArgs& a, cudaStream_t st) {
  if (a.zero && a.rows == nullptr) return launch_pdl(k_paged_end, dim3(a.n), dim3(kForkThreads), 0, st, a);
  // One block where that has few entries and rows to go through.
  const int64_t bytes = (((int64_t)a.n * a.c.layers * a.c.hkv * 2) << a.c.shift) * kDim * 2;
  if ((int64_t)a.n * a.c.width <= 8192 && bytes <= 1 << 19)
    return launch_pdl(k_paged_fork_plan<true>, dim3(1), dim3(kPlanThreads), 0, st, a);
  const int segs = (a.c.width + kSegment - 1) / kSegment;
  const int per = (((2 * a.c.hkv) << a.c.shift) / 4 + kForkThreads - 1) / kForkThreads;
  const int64_t blocks = (int64_t)a.n * segs + (int64_t)a.n * a.c.layers * per;
  if (segs > 65535 || blocks > 0x7fffffff) return cudaErrorInvalidValue;
  cudaError_t e = cudaSuccess;
  if (a.src != a.dst) e = launch_pdl(k_paged_fork_share, dim3(a.n, segs), dim3(kForkThreads), 0, st, a);
  if (e == cudaSuccess) e = launch_pdl(k_paged_fork_plan<false>, dim3(1), dim3(kPlanThreads), 0, st, a);
  if (e == cudaSuccess) e = launch_pdl(k_paged_fork_apply, dim3((unsigned)blocks), dim3(kForkThreads), 0, st, a, segs, per);
  return e;
}

cudaError_t launch_paged_compact(const CompactArgs& a, int sm_count, cudaStream_t st) {
  cudaError_t e = launch_pdl(k_paged_compact_plan, dim3(1), dim3(kPlanThreads), 0, st, a);
  if (e == cudaSuccess) e = launch_pdl(k_paged_compact_move, dim3(8 * sm_count), dim3(kForkThreads), 0, st, a);
  return e;
}

}  // namespace paris
