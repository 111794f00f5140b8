// Eviction from the 4-bit cache by accumulated weight.
//
// One block per (sequence, KV head), or a cluster of up to eight for more
// than 16384 rows; a thread keeps its rows' keys in registers (bits ordered
// like the weights), a warp has a contiguous piece of the rows.  Protected
// rows are counted apart.  The smallest kept key is found by narrowing a
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
// is why it starts only where a thread's keys would no longer fit.
#include <cooperative_groups.h>

#include "kv4_internal.cuh"

namespace cg = cooperative_groups;

namespace paris {
namespace {

constexpr int kEvictThreads = 1024;
constexpr int kEvictWarps = kEvictThreads / 32;
constexpr int kEvictMaxBlocks = 8;
constexpr int kBins = 2048;
constexpr int kHeldKeys = 16;  // keys of a thread in registers; further ones are read again
constexpr int kMoves = 4;      // moves of 16 threads in flight

struct EvictShared {
  uint32_t hist[3][kBins];
  uint32_t warp_a[kEvictWarps], warp_b[kEvictWarps];
  uint32_t few[32];
  uint32_t nfew;
  uint32_t lo, hi, held;        // this block's least and greatest key, its protected rows
  uint32_t all_lo, all_hi, all_held;
  uint32_t bin, above, in_bin;
  uint32_t count[3];            // this block's rows with the threshold key; its holes; its tails
  uint32_t blocks[3][kEvictMaxBlocks];
};

// Key of an unprotected row (protected: false).
__device__ __forceinline__ bool evict_key(float w, int32_t pos, int64_t sink, int64_t recent_from, uint32_t& key) {
  key = w == w ? order_key(w) : 0u;
  return !(pos < sink || pos >= recent_from);
}

template <bool kCluster>
__global__ void __launch_bounds__(kEvictThreads) k_kv4_evict(EvictArgs a) {
  __shared__ __align__(16) EvictShared sh;
  cg::cluster_group cluster = cg::this_cluster();
  auto sync_all = [&]() {
    if (kCluster) cluster.sync();
    else __syncthreads();
  };
  const int nb = kCluster ? (int)cluster.num_blocks() : 1, rank = kCluster ? (int)cluster.block_rank() : 0;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int i = tid; i < 3 * kBins; i += kEvictThreads) (&sh.hist[0][0])[i] = 0;
  if (tid == 0) {
    sh.lo = 0xFFFFFFFFu;
    sh.hi = sh.held = sh.nfew = 0;
  }
  pdl_wait();
  pdl_trigger();
  const int bh = blockIdx.x / nb;
  const int b = bh / a.c.hkv;
  const int32_t next = a.c.next[b];
  const int64_t n = kv4_len(a.c, b);
  const int64_t base = (int64_t)bh * a.c.rmax;
  if (n > a.keep) {  // the same for the whole cluster
    const int64_t recent_from = (int64_t)next - a.recent;
    const int64_t slice = (n + nb - 1) / nb;
    const int64_t r0 = min64(n, rank * slice), r1 = min64(n, r0 + slice);
    const float* w = a.c.w + base;
    const int32_t* pos = a.c.pos + base;
    // the warp's rows: 32 x [0, mine) from first on
    const int mine = (int)((r1 - r0 + kEvictThreads - 1) / kEvictThreads);
    const int64_t first = r0 + (int64_t)warp * mine * 32;
    const int64_t left = r1 - first - lane;  // row i of the lane is there if 32 i < left
    uint32_t held[kHeldKeys];
    uint32_t flags = 0;  // bit 2i: row i is there; bit 2i + 1: and not protected
    {
      float wv[kHeldKeys];
      int32_t pv[kHeldKeys];
#pragma unroll
      for (int i = 0; i < kHeldKeys; ++i)
        if (i < mine && 32 * i < left) {
          wv[i] = w[first + 32 * i + lane];
          pv[i] = pos[first + 32 * i + lane];
        }
#pragma unroll
      for (int i = 0; i < kHeldKeys; ++i) {
        held[i] = 0;
        if (i < mine && 32 * i < left) flags |= (evict_key(wv[i], pv[i], a.sink, recent_from, held[i]) ? 3u : 1u) << (2 * i);
      }
    }
    auto each = [&](auto&& f) {  // f(i, key, state): 0 not there, 1 protected, 3 neither; whole warps, rows ascending
#pragma unroll
      for (int i = 0; i < kHeldKeys; ++i) {
        if (i >= mine) break;
        f(i, held[i], (flags >> (2 * i)) & 3u);
      }
      for (int i = kHeldKeys; i < mine; ++i) {
        uint32_t key = 0, st = 0;
        if (32 * (int64_t)i < left)
          st = evict_key(w[first + 32 * (int64_t)i + lane], pos[first + 32 * (int64_t)i + lane], a.sink, recent_from, key) ? 3u : 1u;
        f(i, key, st);
      }
    };
    uint32_t lo = 0xFFFFFFFFu, hi = 0, prot = 0;
    each([&](int, uint32_t key, uint32_t st) {
      if (st == 3u) {
        lo = min(lo, key);
        hi = max(hi, key);
      }
      prot += st == 1u;
    });
    lo = __reduce_min_sync(kFull, lo);
    hi = __reduce_max_sync(kFull, hi);
    prot = __reduce_add_sync(kFull, prot);
    __syncthreads();
    if (lane == 0) {
      atomicMin(&sh.lo, lo);
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
    const int64_t protected_rows = kCluster ? sh.all_held : sh.held;
    // Rows stay whose key is above `least`, and the first `want` of those
    // with it.  With more protected rows than room, the protected ones are
    // the rows with the threshold key and no other stays.
    const bool crowded = protected_rows >= a.keep;
    int64_t want = crowded ? a.keep : a.keep - protected_rows;
    int64_t equal = crowded ? protected_rows : n - protected_rows;  // rows in the range
#pragma unroll 1
    for (int d = 0; d < 3 && !crowded && lo < hi; ++d) {
      if (!kCluster && equal <= 32) {
        // few rows in the range: a warp ranks them
        each([&](int, uint32_t key, uint32_t st) {
          if (st == 3u && key >= lo && key <= hi) sh.few[atomicAdd(&sh.nfew, 1u)] = key;
        });
        __syncthreads();
        const uint32_t mine_key = lane < equal ? sh.few[lane] : 0u;
        uint32_t larger = 0, same = 0;
        for (int i = 0; i < equal; ++i) {
          const uint32_t k = __shfl_sync(kFull, mine_key, i);
          larger += k > mine_key;
          same += k == mine_key;
        }
        // the key that the wanted row has
        const uint32_t hit = __ballot_sync(kFull, lane < equal && larger < want && larger + same >= want);
        const int src = __ffs(hit) - 1;
        lo = hi = __shfl_sync(kFull, mine_key, src);
        want -= __shfl_sync(kFull, larger, src);
        equal = __shfl_sync(kFull, same, src);
        break;
      }
      // keys lo .. hi in bins of 2^shift
      const int shift = max(0, 32 - __clz(hi - lo) - 11);
      each([&](int, uint32_t key, uint32_t st) {
        if (st == 3u && key >= lo && key <= hi) atomicAdd(&sh.hist[d][(key - lo) >> shift], 1u);
      });
      sync_all();
      // four bins a thread of the first half, from the top
      uint32_t c[4] = {0, 0, 0, 0};
      const int b0 = kBins - 4 - 4 * tid;
      if (tid < kBins / 4) {
        if (kCluster) {
          uint4 v[kEvictMaxBlocks];
#pragma unroll
          for (int i = 0; i < kEvictMaxBlocks; ++i)
            v[i] = i < nb ? *reinterpret_cast<const uint4*>(cluster.map_shared_rank(&sh.hist[d][b0], i)) : make_uint4(0, 0, 0, 0);
#pragma unroll
          for (int i = 0; i < kEvictMaxBlocks; ++i) {
            c[0] += v[i].w;
            c[1] += v[i].z;
            c[2] += v[i].y;
            c[3] += v[i].x;
          }
        } else {
          const uint4 v = *reinterpret_cast<const uint4*>(&sh.hist[d][b0]);
          c[0] = v.w;
          c[1] = v.z;
          c[2] = v.y;
          c[3] = v.x;
        }
      }
      const uint32_t sum = c[0] + c[1] + c[2] + c[3], inc = warp_incl_scan(sum, lane);
      if (lane == 31) sh.warp_a[warp] = inc;
      __syncthreads();
      uint32_t before = __reduce_add_sync(kFull, lane < warp ? sh.warp_a[lane] : 0u) + inc - sum;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (before < want && before + c[i] >= want) {
          sh.bin = b0 + 3 - i;
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
    const uint32_t least = lo;
    const uint32_t tied = crowded ? 1u : 3u;  // state of the rows that share the last places
    auto is_tied = [&](uint32_t key, uint32_t st) { return st == tied && (crowded || key == least); };
    const uint32_t below = (1u << lane) - 1u;
    uint32_t eq_at = 0;
    const bool split_tie = equal > want;  // not all of them stay: the first by row
    if (split_tie) {
      uint32_t eq = 0;
      each([&](int, uint32_t key, uint32_t st) { eq += __popc(__ballot_sync(kFull, is_tied(key, st))); });
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
    // holes and tails of 32 rows as bits
    auto sort_out = [&](int i, uint32_t key, uint32_t st, uint32_t& hs, uint32_t& ts) {
      bool k;
      const bool tie = is_tied(key, st);
      if (split_tie) {
        const uint32_t eqs = __ballot_sync(kFull, tie);
        k = (tie && eq_at + __popc(eqs & below) < want) || (!crowded && (st == 1u || (st == 3u && key > least)));
        eq_at += __popc(eqs);
      } else {
        k = tie || (!crowded && (st == 1u || (st == 3u && key > least)));
      }
      const bool low = first + 32 * (int64_t)i + lane < a.keep;
      hs = __ballot_sync(kFull, st != 0u && !k && low);
      ts = __ballot_sync(kFull, k && !low);
    };
    uint32_t holes = 0, tails = 0;
    const uint32_t eq_start = eq_at;
    each([&](int i, uint32_t key, uint32_t st) {
      uint32_t hs, ts;
      sort_out(i, key, st, hs, ts);
      holes += __popc(hs);
      tails += __popc(ts);
    });
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
    int32_t* list = a.list + (int64_t)bh * 2 * a.c.rmax;
    eq_at = eq_start;
    if (block_holes + block_tails > 0)
      each([&](int i, uint32_t key, uint32_t st) {
        uint32_t hs, ts;
        sort_out(i, key, st, hs, ts);
        const int32_t r = (int32_t)(first + 32 * (int64_t)i + lane);
        if (hs >> lane & 1u) list[r0 + hole_at + __popc(hs & below)] = r;
        if (ts >> lane & 1u) list[a.c.rmax + r0 + tail_at + __popc(ts & below)] = r;
        hole_at += __popc(hs);
        tail_at += __popc(ts);
      });
    __threadfence();
    sync_all();
    // move i of the cluster: tail i into hole i; 16 threads a move
    uint32_t moves = block_holes;
    if (kCluster) {
      if (tid < kEvictMaxBlocks) {
        sh.blocks[1][tid] = tid < nb ? *cluster.map_shared_rank(&sh.count[1], tid) : 0u;
        sh.blocks[2][tid] = tid < nb ? *cluster.map_shared_rank(&sh.count[2], tid) : 0u;
      }
      __syncthreads();
      moves = 0;
      for (int i = 0; i < nb; ++i) moves += sh.blocks[1][i];
    }
    // entry i of a list whose pieces start at the blocks' slices
    auto entry = [&](int which, uint32_t i) -> int64_t {
      const int32_t* l = list + (which == 2 ? a.c.rmax : 0);
      if (kCluster) {
        int blk = 0;
        for (; blk + 1 < nb && i >= sh.blocks[which][blk]; ++blk) i -= sh.blocks[which][blk];
        l += min64(n, blk * slice);
      }
      return base + __ldcg(l + i);
    };
    const int l16 = tid & 15;
    const uint32_t stride = nb * (kEvictThreads / 16);
    for (uint32_t i0 = rank * (kEvictThreads / 16) + (tid >> 4); i0 < moves; i0 += kMoves * stride) {
      int64_t dst[kMoves], src[kMoves];
      uint4 v[kMoves];
#pragma unroll
      for (int u = 0; u < kMoves; ++u)
        if (i0 + u * stride < moves) {
          dst[u] = entry(1, i0 + u * stride);
          src[u] = entry(2, i0 + u * stride);
        }
#pragma unroll
      for (int u = 0; u < kMoves; ++u) {
        if (i0 + u * stride >= moves) continue;
        if (l16 < 8) v[u] = reinterpret_cast<const uint4*>((l16 < 4 ? a.c.kc : a.c.vc) + src[u] * kCode4)[l16 & 3];
        else if (l16 < 12) v[u].x = (l16 == 8 ? reinterpret_cast<const uint32_t*>(a.c.ks) : l16 == 9 ? reinterpret_cast<const uint32_t*>(a.c.vs)
                                     : l16 == 10 ? reinterpret_cast<const uint32_t*>(a.c.w) : reinterpret_cast<const uint32_t*>(a.c.pos))[src[u]];
      }
#pragma unroll
      for (int u = 0; u < kMoves; ++u) {
        if (i0 + u * stride >= moves) continue;
        if (l16 < 8) reinterpret_cast<uint4*>((l16 < 4 ? a.c.kc : a.c.vc) + dst[u] * kCode4)[l16 & 3] = v[u];
        else if (l16 < 12) (l16 == 8 ? reinterpret_cast<uint32_t*>(a.c.ks) : l16 == 9 ? reinterpret_cast<uint32_t*>(a.c.vs)
                            : l16 == 10 ? reinterpret_cast<uint32_t*>(a.c.w) : reinterpret_cast<uint32_t*>(a.c.pos))[dst[u]] = v[u].x;
      }
    }
  }
  sync_all();  // no block leaves while another reads its shared memory
  // the last KV head of the sequence to finish shortens it
  if (rank == 0 && tid == 0) {
    __threadfence();
    if (atomicInc(&a.c.counters[b], (uint32_t)(a.c.hkv - 1)) == (uint32_t)(a.c.hkv - 1) && n > a.keep)
      a.c.lens[b] = (int32_t)a.keep;
  }
}

}  // namespace

cudaError_t launch_kv4_evict(const EvictArgs& a, cudaStream_t st) {
  int nb = 1;
  while (nb < kEvictMaxBlocks && nb * kHeldKeys * kEvictThreads < a.c.rmax) nb *= 2;
  if (nb == 1) return launch_pdl(k_kv4_evict<false>, dim3(a.c.batch * a.c.hkv), dim3(kEvictThreads), 0, st, a);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.c.batch * a.c.hkv * nb);
  cfg.blockDim = dim3(kEvictThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = nb;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, k_kv4_evict<true>, a);
}

}  // namespace paris
