// Eviction from the 4-bit cache by accumulated weight.
//
// One block per (sequence, KV head), or a cluster of up to eight for more
// than 16384 rows; the rows' keys (bits ordered like the weights) are kept in
// shared memory, a warp has a contiguous piece of them.  Protected rows are
// counted apart.  The smallest kept key is found by narrowing a
// range of keys: the range's rows are counted in 2048 equal bins (a
// cluster's counts are read through distributed shared memory), and the bin
// in which the wanted row falls is the next range; once it holds at most 32
// rows a warp ranks them directly.  The range starts at the keys that there
// are, so one round usually settles a block, and three settle anything.
// Equal keys are split by row index.  Then dropped rows below `keep` and kept
// rows above it are listed in ascending order (ballots, and prefixes over
// warps and blocks); they are equally many, and the i-th of the second moves
// into the i-th of the first.  Sources are at index keep and above and
// targets below it, so the moves need no order, and only rows that have to
// move are read and written.
//
// Bound by latency: a row costs 8 bytes, and the rounds are barriers.  A
// cluster costs some 2000 cycles a barrier and round of remote reads, which
// is why it starts only where the keys would no longer fit.  The code is kept
// short for the same reason: it runs once, and with the keys in registers and
// every loop unrolled (46 KB) it waited for its instructions longest.  32 heads
// of 8704 rows, 512 dropped of each: 18.8 us from cold caches.
#include <atomic>
#include <cooperative_groups.h>

#include "kv4_internal.cuh"

namespace cg = cooperative_groups;

namespace paris {
namespace {

constexpr int kMaxWarps = 32;
constexpr int kEvictMaxBlocks = 8;
constexpr int kBins = 2048;
constexpr int kHeldRows = 16384;  // rows of a block whose keys are in shared memory; further ones are read again
constexpr int kMoves = 16;     // rows that a warp moves at once

struct EvictShared {
  uint32_t hist[3][kBins];
  uint32_t warp_a[kMaxWarps], warp_b[kMaxWarps];
  uint32_t few[32];
  uint32_t nfew;
  uint32_t lo, hi, held;        // this block's least and greatest key, its protected rows
  uint32_t all_lo, all_hi, all_held;
  uint32_t drop;                // one row to drop: its index + 1, if it may be in this block
  uint32_t bin, above, in_bin;
  uint32_t count[3];            // this block's rows with the threshold key; its holes; its tails
  uint32_t blocks[3][kEvictMaxBlocks];
};
constexpr uint32_t kProtected = 0xFFFFFFFFu;  // above every weight's key

__device__ __forceinline__ uint32_t evict_key(float w, int32_t pos, int64_t sink, int64_t recent_from) {
  if (pos < sink || pos >= recent_from) return kProtected;
  return w == w ? order_key(w) : 0u;
}

template <bool kCluster, int kThreads>
__global__ void __launch_bounds__(kThreads, kThreads == 512 ? 2 : 1) k_kv4_evict(EvictArgs a) {
  constexpr int kWarps = kThreads / 32;
  constexpr int kBinsPer = kBins / kThreads < 4 ? 4 : kBins / kThreads;  // bins of a thread
  extern __shared__ uint32_t keys[];
  __shared__ __align__(16) EvictShared sh;
  cg::cluster_group cluster = cg::this_cluster();
  auto sync_all = [&]() {
    if (kCluster) cluster.sync();
    else __syncthreads();
  };
  const int nb = kCluster ? (int)cluster.num_blocks() : 1, rank = kCluster ? (int)cluster.block_rank() : 0;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int i = tid; i < 3 * kBins; i += kThreads) (&sh.hist[0][0])[i] = 0;
  if (tid == 0) {
    sh.lo = 0xFFFFFFFFu;
    sh.hi = sh.held = sh.nfew = sh.drop = 0;
  }
  if (tid < kMaxWarps) sh.warp_a[tid] = sh.warp_b[tid] = 0;  // what warps that are not there count
  pdl_wait();
  pdl_trigger();
  const int bh = blockIdx.x / nb;
  const int b = bh / a.c.hkv;
  const int32_t next = a.c.next[b];
  const int n = (int)kv4_len(a.c, b), keep = (int)a.keep;
  const int64_t base = (int64_t)bh * a.c.rmax;
  if (n > keep) {  // the same for the whole cluster
    const int64_t recent_from = (int64_t)next - a.recent;
    const int slice = kCluster ? (int)(((int64_t)n + nb - 1) / nb) : n;
    const int r0 = kCluster ? (int)min64(n, (int64_t)rank * slice) : 0, r1 = r0 + min(n - r0, slice);
    const float* w = a.c.w + base;
    const int32_t* pos = a.c.pos + base;
    // the warp's rows: 32 x [0, mine) from first on
    const int mine = (int)(((uint32_t)(r1 - r0) + kThreads - 1) / kThreads);
    const int64_t first = r0 + (int64_t)warp * mine * 32;
    const int end = (int)max64(min64(r1 - first, (int64_t)mine * 32), 0);  // the warp's rows that are there: < end
    const int room = (int)max64(min64(keep - first, (int64_t)mine * 32), 0);  // and below keep: < room
    const int heldi = min(mine, kHeldRows / kThreads);
    uint32_t* mykeys = keys + warp * heldi * 32;
    uint32_t lo = 0xFFFFFFFFu, hi = 0, prot = 0, lo_at = 0;  // lo_at: the last row with the key lo
    auto take = [&](uint32_t key, uint32_t row) {  // a thread's rows ascend
      if (key == kProtected) ++prot;
      else {
        if (key <= lo) lo_at = row;
        lo = min(lo, key);
        hi = max(hi, key);
      }
    };
    constexpr int kAhead = 8;  // rows of a thread on their way at once
#pragma unroll 1
    for (int i0 = 0; i0 < heldi; i0 += kAhead) {
      float wv[kAhead];
      int32_t pv[kAhead];
      const float* wp = w + first + 32 * i0 + lane;
      const int32_t* pp = pos + first + 32 * i0 + lane;
      const int here = min(min(heldi - i0, kAhead), (end - 32 * i0 - lane + 31) >> 5);  // the thread's rows of these
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
        if (u < here) {
          wv[u] = __ldcg(wp + 32 * u);
          pv[u] = __ldcg(pp + 32 * u);
        }
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
        if (u < here) {
          const uint32_t key = evict_key(wv[u], pv[u], a.sink, recent_from);
          mykeys[32 * (i0 + u) + lane] = key;
          take(key, (uint32_t)first + 32 * (i0 + u) + lane);
        }
    }
    auto some = [&](int i0, int i1, auto&& f) {  // f(i, key, whether the row is there): whole warps, rows ascending
#pragma unroll 1
      for (int i = i0; i < i1; ++i) {
        const int x = 32 * i + lane;
        const bool in = x < end;
        uint32_t key = 0;
        if (in) key = i < heldi ? mykeys[x] : evict_key(w[first + x], pos[first + x], a.sink, recent_from);
        f(i, key, in);
      }
    };
    auto each = [&](auto&& f) { some(0, mine, f); };
#pragma unroll 1
    for (int i = heldi; i < mine; ++i) {
      const int x = 32 * i + lane;
      if (x < end) take(evict_key(w[first + x], pos[first + x], a.sink, recent_from), (uint32_t)first + x);
    }
    const uint32_t warp_lo = __reduce_min_sync(kFull, lo);
    lo_at = __reduce_max_sync(kFull, lo == warp_lo ? lo_at : 0u);
    hi = __reduce_max_sync(kFull, hi);
    prot = __reduce_add_sync(kFull, prot);
    __syncthreads();
    if (lane == 0) {
      sh.warp_a[warp] = warp_lo;
      sh.warp_b[warp] = lo_at;
      atomicMin(&sh.lo, warp_lo);
      atomicMax(&sh.hi, hi);
      atomicAdd(&sh.held, prot);
    }
    sync_all();
    if (kCluster) {
      if (warp == 0) {
        uint32_t x = 0xFFFFFFFFu, y = 0, z = 0;
        if (lane < nb) {
          x = *cluster.map_shared_rank(&sh.lo, lane);
          y = *cluster.map_shared_rank(&sh.hi, lane);
          z = *cluster.map_shared_rank(&sh.held, lane);
        }
        x = __reduce_min_sync(kFull, x);
        y = __reduce_max_sync(kFull, y);
        z = __reduce_add_sync(kFull, z);
        if (lane == 0) {
          sh.all_lo = x;
          sh.all_hi = y;
          sh.all_held = z;
        }
      }
      __syncthreads();
    }
    lo = kCluster ? sh.all_lo : sh.lo;
    hi = kCluster ? sh.all_hi : sh.hi;
    const uint32_t protected_rows = kCluster ? sh.all_held : sh.held;
    // Rows stay whose key is above `least`, and the first `want` of those
    // with it.  With more protected rows than room, the protected ones are
    // the rows with the threshold key and no other stays.
    const bool crowded = protected_rows >= (uint32_t)keep;
    uint32_t want = crowded ? keep : keep - protected_rows;
    uint32_t equal = crowded ? protected_rows : n - protected_rows;  // rows in the range
    uint32_t moves, drop = 0;
    // A decode step drops one row, the last of those with the least key, and
    // the one row above `keep` takes its place: neither rounds nor lists
    // (a step of 2049 rows 18.5 -> 15.8 us, of 32 x 4097 67.2 -> 62.5).
    const bool one = n - keep == 1 && !crowded;
    if (one) {
      if (lane == 0 && sh.warp_a[warp] == lo) atomicMax(&sh.drop, sh.warp_b[warp] + 1);
      sync_all();
      drop = (kCluster ? __reduce_max_sync(kFull, lane < nb ? *cluster.map_shared_rank(&sh.drop, lane) : 0u) : sh.drop) - 1;
      moves = drop != (uint32_t)keep;
    } else {
#pragma unroll 1
      for (int d = 0; d < 3 && !crowded && lo < hi; ++d) {
        if (!kCluster && equal <= 32) {
          // few rows in the range: a warp ranks them
          each([&](int, uint32_t key, bool in) {
            if (in && key >= lo && key <= hi) sh.few[atomicAdd(&sh.nfew, 1u)] = key;
          });
          __syncthreads();
          if (warp == 0) {
            const uint32_t own = lane < equal ? sh.few[lane] : 0u;
            uint32_t larger = 0, same = 0;
            for (uint32_t i = 0; i < equal; ++i) {
              const uint32_t k = __shfl_sync(kFull, own, i);
              larger += k > own;
              same += k == own;
            }
            // the key that the wanted row has
            if (lane < equal && larger < want && larger + same >= want) {
              sh.bin = own;
              sh.above = larger;
              sh.in_bin = same;
            }
          }
          __syncthreads();
          lo = hi = sh.bin;
          want -= sh.above;
          equal = sh.in_bin;
          break;
        }
        // keys lo .. hi in bins of 2^shift
        const int shift = max(0, 32 - __clz(hi - lo) - 11);
        each([&](int, uint32_t key, bool in) {
          if (in && key >= lo && key <= hi) atomicAdd(&sh.hist[d][(key - lo) >> shift], 1u);
        });
        sync_all();
        // a thread's bins, from the top
        uint32_t c[kBinsPer];
#pragma unroll
        for (int i = 0; i < kBinsPer; ++i) c[i] = 0;
        const int b0 = kBins - kBinsPer - kBinsPer * tid;
        if (tid < kBins / kBinsPer) {
#pragma unroll
          for (int q = 0; q < kBinsPer; q += 4) {
            const uint32_t* bins = &sh.hist[d][b0 + kBinsPer - 4 - q];
            uint4 v[kCluster ? kEvictMaxBlocks : 1];
#pragma unroll
            for (int i = 0; i < (kCluster ? kEvictMaxBlocks : 1); ++i)
              v[i] = !kCluster ? *reinterpret_cast<const uint4*>(bins)
                     : i < nb ? *reinterpret_cast<const uint4*>(cluster.map_shared_rank(bins, i)) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int i = 0; i < (kCluster ? kEvictMaxBlocks : 1); ++i) {
              c[q] += v[i].w;
              c[q + 1] += v[i].z;
              c[q + 2] += v[i].y;
              c[q + 3] += v[i].x;
            }
          }
        }
        uint32_t sum = 0;
#pragma unroll
        for (int i = 0; i < kBinsPer; ++i) sum += c[i];
        const uint32_t inc = warp_incl_scan(sum, lane);
        if (lane == 31) sh.warp_a[warp] = inc;
        __syncthreads();
        uint32_t before = __reduce_add_sync(kFull, lane < warp ? sh.warp_a[lane] : 0u) + inc - sum;
#pragma unroll
        for (int i = 0; i < kBinsPer; ++i) {
          if (before < want && before + c[i] >= want) {
            sh.bin = b0 + kBinsPer - 1 - i;
            sh.above = before;
            sh.in_bin = c[i];
          }
          before += c[i];
        }
        __syncthreads();
        const uint32_t bin_lo = lo + (sh.bin << shift);
        hi = min(hi, bin_lo + ((1u << shift) - 1u));
        lo = bin_lo;
        want -= sh.above;
        equal = sh.in_bin;
      }
      // the threshold: rows above it stay, and the first `want` of those on it
      const uint32_t least = crowded ? kProtected : lo;
      const uint32_t below = (1u << lane) - 1u;
      uint32_t eq_at = 0;
      const bool split_tie = equal > want;  // not all of them stay: the first by row
      if (split_tie) {
        uint32_t eq = 0;
        each([&](int, uint32_t key, bool in) { eq += __popc(__ballot_sync(kFull, in && key == least)); });
        __syncthreads();
        if (lane == 0) sh.warp_a[warp] = eq;
        __syncthreads();
        const uint32_t v = sh.warp_a[lane];
        eq_at = __reduce_add_sync(kFull, lane < warp ? v : 0u);
        if (kCluster) {
          const uint32_t all = __reduce_add_sync(kFull, v);
          if (tid == 0) sh.count[0] = all;
          cluster.sync();
          eq_at += __reduce_add_sync(kFull, lane < rank ? *cluster.map_shared_rank(&sh.count[0], min(lane, nb - 1)) : 0u);
        }
      }
      // Holes and tails of 32 x 32 rows as bits, those of 32 rows in a lane;
      // then each lane lists its own, of up to 32 x 32 rows a warp without
      // sorting them out again (512 of 8704 rows dropped, with the store and the
      // read: 57.0 -> 55.4 us).
      uint32_t hs = 0, ts = 0;
      auto sort_out = [&](int i0) {
        hs = ts = 0;
        some(i0, min(mine, i0 + 32), [&](int i, uint32_t key, bool in) {
          bool k = key >= least;
          if (split_tie) {
            const uint32_t eqs = __ballot_sync(kFull, in && key == least);
            k = key > least || (key == least && eq_at + __popc(eqs & below) < want);
            eq_at += __popc(eqs);
          }
          const bool low = 32 * i + lane < room;
          const uint32_t h = __ballot_sync(kFull, in && !k && low), t = __ballot_sync(kFull, in && k && !low);
          if (lane == i - i0) {
            hs = h;
            ts = t;
          }
        });
      };
      uint32_t holes = 0, tails = 0;
      const uint32_t eq_start = eq_at;
#pragma unroll 1
      for (int i0 = 0; i0 < mine; i0 += 32) {
        sort_out(i0);
        holes += __reduce_add_sync(kFull, __popc(hs));
        tails += __reduce_add_sync(kFull, __popc(ts));
      }
      __syncthreads();
      if (lane == 0) {
        sh.warp_a[warp] = holes;
        sh.warp_b[warp] = tails;
      }
      __syncthreads();
      const uint32_t ha = sh.warp_a[lane], ta = sh.warp_b[lane];
      uint32_t hole_at = __reduce_add_sync(kFull, lane < warp ? ha : 0u), tail_at = __reduce_add_sync(kFull, lane < warp ? ta : 0u);
      const uint32_t block_holes = __reduce_add_sync(kFull, ha), block_tails = __reduce_add_sync(kFull, ta);
      if (tid == 0) {
        sh.count[1] = block_holes;
        sh.count[2] = block_tails;
      }
      eq_at = eq_start;
      int32_t* list = a.list + (int64_t)bh * 2 * a.c.rmax;
      if (holes + tails > 0) {  // of the warp
#pragma unroll 1
        for (int i0 = 0; i0 < mine; i0 += 32) {
          if (mine > 32) sort_out(i0);
          auto put = [&](uint32_t bits, uint32_t& at, int32_t* to) {
            const uint32_t inc = warp_incl_scan((uint32_t)__popc(bits), lane);
            int32_t* p = to + (at + inc - __popc(bits));
            for (; bits != 0; bits &= bits - 1) *p++ = (int32_t)first + 32 * (i0 + lane) + __ffs(bits) - 1;
            at += __shfl_sync(kFull, inc, 31);
          };
          put(hs, hole_at, list + r0);
          put(ts, tail_at, list + a.c.rmax + r0);
        }
      }
      __threadfence();
      sync_all();
      moves = block_holes;
      if (kCluster) {
        if (tid < kEvictMaxBlocks) {
          sh.blocks[1][tid] = tid < nb ? *cluster.map_shared_rank(&sh.count[1], tid) : 0u;
          sh.blocks[2][tid] = tid < nb ? *cluster.map_shared_rank(&sh.count[2], tid) : 0u;
        }
        __syncthreads();
        moves = 0;
        for (int i = 0; i < nb; ++i) moves += sh.blocks[1][i];
      }
    }
    // move i of the cluster: tail i into hole i
    // entry i of a list whose pieces start at the blocks' slices
    auto entry = [&](int which, uint32_t i) -> int32_t {
      const int32_t* l = a.list + ((int64_t)bh * 2 + (which == 2)) * a.c.rmax;
      if (kCluster) {
        int blk = 0;
        for (; blk + 1 < nb && i >= sh.blocks[which][blk]; ++blk) i -= sh.blocks[which][blk];
        l += min64(n, (int64_t)blk * slice);
      }
      return __ldcg(l + i);
    };
    // a warp moves kMoves rows at once: of each its codes, four bytes a lane,
    // and of eight together their scales, weights and positions
    uint8_t* const codes_at = (lane < 16 ? a.c.kc : a.c.vc) + base * kCode4 + 4 * (lane & 15);
    const int what = lane & 3;
    uint32_t* const rest_at = (what == 0 ? reinterpret_cast<uint32_t*>(a.c.ks) : what == 1 ? reinterpret_cast<uint32_t*>(a.c.vs)
                               : what == 2 ? reinterpret_cast<uint32_t*>(a.c.w) : reinterpret_cast<uint32_t*>(a.c.pos)) + base;
#pragma unroll 1
    for (uint32_t i0 = (rank * kWarps + warp) * kMoves; i0 < moves; i0 += nb * kWarps * kMoves) {
      const int here = (int)min(moves - i0, (uint32_t)kMoves);
      int32_t to = 0, from = 0;
      if (lane < here) {
        to = one ? (int32_t)drop : entry(1, i0 + lane);
        from = one ? keep : entry(2, i0 + lane);
      }
      uint32_t x[kMoves], y[kMoves / 8];
#pragma unroll
      for (int u = 0; u < kMoves; ++u) {
        const int32_t src = __shfl_sync(kFull, from, u);
        if (u < here) x[u] = *reinterpret_cast<const uint32_t*>(codes_at + (int64_t)src * kCode4);
      }
#pragma unroll
      for (int u = 0; u < kMoves / 8; ++u) {
        const int32_t src = __shfl_sync(kFull, from, 8 * u + (lane >> 2));
        if (8 * u + (lane >> 2) < here) y[u] = rest_at[src];
      }
#pragma unroll
      for (int u = 0; u < kMoves; ++u) {
        const int32_t dst = __shfl_sync(kFull, to, u);
        if (u < here) *reinterpret_cast<uint32_t*>(codes_at + (int64_t)dst * kCode4) = x[u];
      }
#pragma unroll
      for (int u = 0; u < kMoves / 8; ++u) {
        const int32_t dst = __shfl_sync(kFull, to, 8 * u + (lane >> 2));
        if (8 * u + (lane >> 2) < here) rest_at[dst] = y[u];
      }
    }
  }
  sync_all();  // no block leaves while another reads its shared memory
  // the last KV head of the sequence to finish shortens it
  if (rank == 0 && tid == 0) {
    __threadfence();
    if (atomicInc(&a.c.counters[b], (uint32_t)(a.c.hkv - 1)) == (uint32_t)(a.c.hkv - 1) && n > keep)
      a.c.lens[b] = (int32_t)a.keep;
  }
}

}  // namespace

namespace {

template <bool kCluster, int kThreads>
cudaError_t launch_evict(const EvictArgs& a, int nb, cudaStream_t st) {
  const int64_t per_block = ((a.c.rmax + nb - 1) / nb + kThreads - 1) / kThreads * kThreads;
  const size_t smem = (size_t)min64(kHeldRows, per_block) * sizeof(uint32_t);
  static std::atomic<bool> done[64];  // the limit belongs to the device; setting it twice is harmless
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess && !(dev >= 0 && dev < 64 && done[dev])) {
    e = cudaFuncSetAttribute((const void*)k_kv4_evict<kCluster, kThreads>, cudaFuncAttributeMaxDynamicSharedMemorySize, kHeldRows * 4);
    if (e == cudaSuccess && dev >= 0 && dev < 64) done[dev] = true;
  }
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.c.batch * a.c.hkv * nb);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = nb;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = kCluster ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, k_kv4_evict<kCluster, kThreads>, a);
}

}  // namespace

cudaError_t launch_kv4_evict(const EvictArgs& a, cudaStream_t st) {
  // Two blocks of 512 threads an SM, or one of 1024.  With few heads the smaller
  // block's barriers win while its rows are few and lose as they grow (8 heads,
  // 512 rows dropped of 2049: 5.0 against 5.4 us; of 6144: 7.2 against 6.9; of
  // 8192: 8.0 against 7.5); with more heads than SMs two blocks an SM win at any
  // size (256 heads of 6144 rows: 9.3 against 12.8 us), but a cache of larger
  // capacity seldom has as many.
  if (a.c.rmax <= 6144) return launch_evict<false, 512>(a, 1, st);
  int nb = 1;
  while (nb < kEvictMaxBlocks && (int64_t)nb * kHeldRows < a.c.rmax) nb *= 2;
  return nb == 1 ? launch_evict<false, 1024>(a, 1, st) : launch_evict<true, 1024>(a, nb, st);
}

}  // namespace paris
