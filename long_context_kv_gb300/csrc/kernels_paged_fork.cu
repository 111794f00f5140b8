// The paged cache: sequences that fork, end or are cut, and a pool that is
// closed up.
//
// A fork is three kernels, since what it reads (the sources' pages) may be
// what it changes: the first shares the full pages and notes the sources'
// entries, the second, one block, decides on the pages that are not full and
// takes free ones for their copies, the third gives back what the
// destinations held, writes their entries and copies rows.  Counts change by
// sums only, so their order does not matter.
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

__global__ void __launch_bounds__(kForkThreads) k_paged_fork_share(ForkArgs a) {
  pdl_wait();
  pdl_trigger();
  const int i = blockIdx.x, src = a.src[i], dst = a.dst[i];
  if (!in_range(a.c, src) || !in_range(a.c, dst)) return;
  const int rows = fork_rows(a, i, src), full = rows >> a.c.shift, pages = pages_of(a.c, rows);
  // of a sequence that stays itself nothing is shared and nothing given back
  const int j0 = blockIdx.y * kSegment;
  if (src == dst || j0 >= pages) return;
  bool twice = false;
  for (int t = threadIdx.x; t < i; t += kForkThreads) twice |= a.dst[t] == dst && in_range(a.c, a.src[t]);
  if (__syncthreads_or(twice)) return;
#pragma unroll
  for (int u = 0; u < kSegment / kForkThreads; ++u) {
    const int j = j0 + u * kForkThreads + threadIdx.x;
    if (j >= pages) break;
    const int p = page_at(a.c, src, j);
    a.entries[(int64_t)i * a.c.width + j] = p;
    if (j < full) atomicAdd(&a.c.refs[p], 1);
  }
}

__global__ void __launch_bounds__(kPlanThreads) k_paged_fork_plan(ForkArgs a) {
  __shared__ int owner[kMaxPagedSeqs];  // the first entry of a destination; then the entries that take a page, in order
  __shared__ uint32_t tmp[33];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x;
  for (int s = tid; s < a.c.n_seqs; s += kPlanThreads) owner[s] = 0x7fffffff;
  __syncthreads();
  bool wrong = false, short_of = false;
  for (int i = tid; i < a.n; i += kPlanThreads) {
    const bool ok = in_range(a.c, a.src[i]) && in_range(a.c, a.dst[i]);
    if (ok) atomicMin(&owner[a.dst[i]], i);
    wrong |= !ok;
  }
  __syncthreads();
  const uint32_t n_free = (uint32_t)max(a.c.n_pages - max(a.c.n_used[0], 0), 0);
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
  const uint32_t taken = min(copies, n_free);
  if (taken == 0) return;
  __syncthreads();
  take_free(a.c, taken, tmp, [&](uint32_t r, int page) {
    a.plan[owner[r]].last = page;
    a.c.refs[page] = 1;
  });
  if (tid == 0) a.c.n_used[0] = max(a.c.n_used[0], 0) + (int)taken;
}

// A row of one pool to another page of it: 16 lanes, 8 channels each.
__device__ __forceinline__ void copy_row(const uint8_t* from, uint8_t* to, int l16, int e4m3) {
  if (e4m3) reinterpret_cast<uint2*>(to)[l16] = reinterpret_cast<const uint2*>(from)[l16];
  else reinterpret_cast<uint4*>(to)[l16] = reinterpret_cast<const uint4*>(from)[l16];
}

// Blocks [0, n segs): entries; behind them `per` blocks for each (entry,
// layer) copy rows.
__global__ void __launch_bounds__(kForkThreads) k_paged_fork_apply(ForkArgs a, int segs, int per) {
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x;
  if ((int)blockIdx.x < a.n * segs) {
    const int i = blockIdx.x / segs, seg = blockIdx.x - i * segs;
    const ForkEntry e = a.plan[i];
    if (e.dst < 0) return;
    int gone = 0;
    const bool self = e.src == e.dst;
#pragma unroll
    for (int u = 0; u < kSegment / kForkThreads; ++u) {
      const int j = seg * kSegment + u * kForkThreads + tid;
      if (j >= a.c.width || (j >= e.old_pages && j > e.full)) break;
      int32_t* entry = a.c.table + (int64_t)e.dst * a.c.width + j;
      const int old = clamp_page(a.c, *entry);
      const bool stays = self && (j < e.full || (j == e.full && e.last == old));
      if (!stays) {
        if (j < e.full) *entry = a.entries[(int64_t)i * a.c.width + j];
        else if (j == e.full && e.last >= 0) *entry = e.last;
        if (j < e.old_pages && atomicSub(&a.c.refs[old], 1) == 1) {
          atomicOr(&a.c.bits[old >> 5], 1u << (old & 31));
          ++gone;
        }
      }
    }
    gone = __reduce_add_sync(kFull, gone);
    if ((tid & 31) == 0 && gone != 0) atomicSub(a.c.n_used, gone);
    return;
  }
  const int x = blockIdx.x - a.n * segs, il = x / per, part = x - il * per, i = il / a.c.layers, layer = il - i * a.c.layers;
  const ForkEntry e = a.plan[i];
  if (e.dst < 0 || e.rows == 0 || e.last < 0) return;
  const int l16 = tid & 15, items = 2 * a.c.hkv * e.rows;
#pragma unroll 4
  for (int it = part * (kForkThreads / 16) + (tid >> 4); it < items; it += per * (kForkThreads / 16)) {
    const int hv = it / e.rows, r = it - hv * e.rows, h = hv >> 1;
    const PageStrides& st = hv & 1 ? a.c.sv : a.c.sk;
    uint8_t* p = (hv & 1 ? a.c.v : a.c.k) + layer * st.layer + h * st.head + r * st.row;
    copy_row(p + e.from * st.page, p + e.last * st.page, l16, a.c.e4m3);
    if (a.c.e4m3 && l16 == 0) {
      uint8_t* s = hv & 1 ? a.c.vs : a.c.ks;
      s[scale_at(a.c, layer, e.last, h, r)] = s[scale_at(a.c, layer, e.from, h, r)];
    }
  }
}

// One block: the used pages past their number and the free ones below it, in
// ascending order, by one scan of both counts (at most 2^15 a round, in the
// halves of a word); the bits as they are afterwards.
__global__ void __launch_bounds__(kPlanThreads) k_paged_compact_plan(CompactArgs a) {
  __shared__ uint32_t tmp[33];
  pdl_wait();
  pdl_trigger();
  const int used = min(max(a.c.n_used[0], 0), a.c.n_pages), words = (a.c.n_pages + 31) / 32;
  uint32_t low = 0, high = 0;
  for (int w0 = 0; w0 < words; w0 += kPlanThreads) {
    const int w = w0 + threadIdx.x, p0 = 32 * w;
    const uint32_t is_page = p0 + 32 <= a.c.n_pages ? kFull : p0 < a.c.n_pages ? (1u << (a.c.n_pages - p0)) - 1u : 0u;
    const uint32_t below = p0 + 32 <= used ? kFull : p0 < used ? (1u << (used - p0)) - 1u : 0u;
    const uint32_t free = w < words ? a.c.bits[w] & is_page : 0u;
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
  if (threadIdx.x == 0) a.moves[0] = (int)min(low, high);
}

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
  const int64_t rows = ((int64_t)moves * a.c.layers * 2 * a.c.hkv) << a.c.shift;
#pragma unroll 4
  for (int64_t it = me >> 4; it < rows; it += threads >> 4) {
    const int r = (int)it & ((1 << a.c.shift) - 1);
    const int64_t u = it >> a.c.shift, hv = u / (2 * a.c.hkv);
    const int x = (int)(u - hv * 2 * a.c.hkv), h = x >> 1, m = (int)(hv / a.c.layers), layer = (int)(hv - (int64_t)m * a.c.layers);
    const PageStrides& st = x & 1 ? a.c.sv : a.c.sk;
    uint8_t* p = (x & 1 ? a.c.v : a.c.k) + layer * st.layer + h * st.head + r * st.row;
    const int from = a.from[m], to = a.to[m];
    copy_row(p + from * st.page, p + to * st.page, l16, a.c.e4m3);
    if (a.c.e4m3 && l16 == 0) {
      uint8_t* s = x & 1 ? a.c.vs : a.c.ks;
      s[scale_at(a.c, layer, to, h, r)] = s[scale_at(a.c, layer, from, h, r)];
    }
  }
}

}  // namespace

cudaError_t launch_paged_fork(const ForkArgs& a, cudaStream_t st) {
  const int segs = (a.c.width + kSegment - 1) / kSegment;
  const int per = (((2 * a.c.hkv) << a.c.shift) + kForkThreads - 1) / kForkThreads;
  const int64_t blocks = (int64_t)a.n * segs + (int64_t)a.n * a.c.layers * per;
  if (segs > 65535 || blocks > 0x7fffffff) return cudaErrorInvalidValue;
  cudaError_t e = launch_pdl(k_paged_fork_share, dim3(a.n, segs), dim3(kForkThreads), 0, st, a);
  if (e == cudaSuccess) e = launch_pdl(k_paged_fork_plan, dim3(1), dim3(kPlanThreads), 0, st, a);
  if (e == cudaSuccess) e = launch_pdl(k_paged_fork_apply, dim3((unsigned)blocks), dim3(kForkThreads), 0, st, a, segs, per);
  return e;
}

cudaError_t launch_paged_compact(const CompactArgs& a, int sm_count, cudaStream_t st) {
  cudaError_t e = launch_pdl(k_paged_compact_plan, dim3(1), dim3(kPlanThreads), 0, st, a);
  if (e == cudaSuccess) e = launch_pdl(k_paged_compact_move, dim3(8 * sm_count), dim3(kForkThreads), 0, st, a);
  return e;
}

}  // namespace paris
