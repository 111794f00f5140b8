// Eviction from the 4-bit cache by accumulated weight.
//
// One cluster per (sequence, KV head), a contiguous slice of its rows per
// block.  A row's key orders rows by weight (protected rows above all); the
// keep-th largest key is found digit by digit from the top, eight bits at a
// time: each block counts its rows' digits, the cluster's counts are read
// through distributed shared memory, and every block takes the same digit.
// Equal keys are split by row index.  Then dropped rows below `keep` and
// kept rows above it are listed in ascending order; they are equally many,
// and the i-th of the second moves into the i-th of the first.  Sources are
// at index keep and above and targets below it, so the moves need no order,
// and only rows that have to move are read and written.
#include <cooperative_groups.h>

#include "kv4_internal.cuh"

namespace cg = cooperative_groups;

namespace paris {
namespace {

constexpr int kEvictThreads = 1024;
constexpr int kEvictMaxBlocks = 8;

struct EvictShared {
  uint32_t hist[4][256];
  uint32_t tmp[33];
  uint32_t sum[256];
  uint32_t digit, above;
  uint32_t count[3];  // this block's rows with the threshold key; its holes; its tails
};

__device__ __forceinline__ uint32_t evict_key(float w, int32_t pos, int64_t sink, int64_t recent_from) {
  if (pos < sink || pos >= recent_from) return 0xFFFFFFFFu;
  return w == w ? order_key(w) : 0u;
}

__global__ void __launch_bounds__(kEvictThreads) k_kv4_evict(EvictArgs a) {
  __shared__ EvictShared sh;
  cg::cluster_group cluster = cg::this_cluster();
  pdl_wait();
  pdl_trigger();
  const int nb = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int bh = blockIdx.x / nb;
  const int b = bh / a.c.hkv;
  const int tid = threadIdx.x;
  const int64_t n = kv4_len(a.c, b);
  const int64_t base = (int64_t)bh * a.c.rmax;
  if (n > a.keep) {  // the same for the whole cluster
    const int64_t recent_from = (int64_t)a.c.next[b] - a.recent;
    const int64_t slice = (n + nb - 1) / nb;
    const int64_t r0 = min64(n, rank * slice), r1 = min64(n, r0 + slice);
    const float* w = a.c.w + base;
    const int32_t* pos = a.c.pos + base;
    for (int i = tid; i < 4 * 256; i += kEvictThreads) (&sh.hist[0][0])[i] = 0;
    __syncthreads();
    uint32_t prefix = 0;
    int64_t want = a.keep;  // rows still wanted among those with the prefix
#pragma unroll 1
    for (int d = 0; d < 4; ++d) {
      const int shift = 24 - 8 * d;
      for (int64_t r = r0 + tid; r < r1; r += kEvictThreads) {
        const uint32_t key = evict_key(w[r], pos[r], a.sink, recent_from);
        if (d == 0 || (key >> (shift + 8)) == prefix) atomicAdd(&sh.hist[d][(key >> shift) & 255u], 1u);
      }
      cluster.sync();
      if (tid < 256) {
        uint32_t c = 0;
        for (int i = 0; i < nb; ++i) c += *cluster.map_shared_rank(&sh.hist[d][tid], i);
        sh.sum[tid] = c;
      }
      __syncthreads();
      // the largest digit with at least `want` rows at it or above
      const uint32_t mine = tid < 256 ? sh.sum[255 - tid] : 0u;
      uint32_t total;
      const uint32_t before = block_excl_scan(mine, sh.tmp, &total);
      if (tid < 256 && before < (uint32_t)want && before + mine >= (uint32_t)want) {
        sh.digit = 255 - tid;
        sh.above = before;
      }
      __syncthreads();
      prefix = (prefix << 8) | sh.digit;
      want -= sh.above;
    }
    // prefix is the smallest kept key; `want` of the rows that have it stay
    if (tid == 0) sh.count[0] = sh.hist[3][prefix & 255u];
    cluster.sync();
    int64_t eq0 = 0;  // rows with the threshold key in the blocks in front
    for (int i = 0; i < rank; ++i) eq0 += *cluster.map_shared_rank(&sh.count[0], i);
    int32_t* list = a.list + (int64_t)bh * 2 * a.c.rmax;
    int32_t* holes = list + r0;
    int32_t* tails = list + a.c.rmax + r0;
    uint32_t nholes = 0, ntails = 0;
    for (int64_t c0 = r0; c0 < r1; c0 += kEvictThreads) {
      const int64_t r = c0 + tid;
      const bool in = r < r1;
      const uint32_t key = in ? evict_key(w[r], pos[r], a.sink, recent_from) : 0u;
      uint32_t total;
      const uint32_t eq = in && key == prefix ? 1u : 0u;
      const uint32_t eq_before = block_excl_scan(eq, sh.tmp, &total);
      const bool kept = in && (key > prefix || (eq && eq0 + eq_before < want));
      eq0 += total;
      const uint32_t hole = in && !kept && r < a.keep ? 1u : 0u, tail = kept && r >= a.keep ? 1u : 0u;
      // holes and tails fit 16 bits of a block's 1024 rows each
      const uint32_t at = block_excl_scan(hole | (tail << 16), sh.tmp, &total);
      if (hole) holes[nholes + (at & 0xffffu)] = (int32_t)r;
      if (tail) tails[ntails + (at >> 16)] = (int32_t)r;
      nholes += total & 0xffffu;
      ntails += total >> 16;
    }
    if (tid == 0) {
      sh.count[1] = nholes;
      sh.count[2] = ntails;
    }
    __threadfence();
    cluster.sync();
    // move i of the cluster: tail i into hole i; 16 threads a move
    int64_t moves = 0;
    for (int i = 0; i < nb; ++i) moves += *cluster.map_shared_rank(&sh.count[1], i);
    const int l16 = tid & 15;
    for (int64_t i = (int64_t)rank * (kEvictThreads / 16) + (tid >> 4); i < moves; i += nb * (kEvictThreads / 16)) {
      int64_t hi = i, ti = i;
      int hb = 0, tb = 0;
      for (; hb + 1 < nb; ++hb) {
        const uint32_t c = *cluster.map_shared_rank(&sh.count[1], hb);
        if (hi < c) break;
        hi -= c;
      }
      for (; tb + 1 < nb; ++tb) {
        const uint32_t c = *cluster.map_shared_rank(&sh.count[2], tb);
        if (ti < c) break;
        ti -= c;
      }
      const int64_t dst = base + __ldcg(list + min64(n, hb * slice) + hi);
      const int64_t src = base + __ldcg(list + a.c.rmax + min64(n, tb * slice) + ti);
      if (l16 < 4) {
        reinterpret_cast<uint4*>(a.c.kc + dst * kCode4)[l16] = reinterpret_cast<const uint4*>(a.c.kc + src * kCode4)[l16];
      } else if (l16 < 8) {
        reinterpret_cast<uint4*>(a.c.vc + dst * kCode4)[l16 - 4] =
            reinterpret_cast<const uint4*>(a.c.vc + src * kCode4)[l16 - 4];
      } else if (l16 == 8) {
        *reinterpret_cast<uint32_t*>(a.c.ks + dst * kScale4) = *reinterpret_cast<const uint32_t*>(a.c.ks + src * kScale4);
      } else if (l16 == 9) {
        *reinterpret_cast<uint32_t*>(a.c.vs + dst * kScale4) = *reinterpret_cast<const uint32_t*>(a.c.vs + src * kScale4);
      } else if (l16 == 10) {
        a.c.w[dst] = a.c.w[src];
      } else if (l16 == 11) {
        a.c.pos[dst] = a.c.pos[src];
      }
    }
  }
  cluster.sync();  // no block leaves while another reads its shared memory
  // the last KV head of the sequence to finish shortens it
  if (rank == 0 && tid == 0) {
    __threadfence();
    if (atomicInc(&a.c.counters[b], (uint32_t)(a.c.hkv - 1)) == (uint32_t)(a.c.hkv - 1) && n > a.keep)
      a.c.lens[b] = (int32_t)a.keep;
  }
}

}  // namespace

cudaError_t launch_kv4_evict(const EvictArgs& a, cudaStream_t st) {
  // a block per 4096 rows: below that a cluster's barriers cost more than
  // the rows do
  int nb = 1;
  while (nb < kEvictMaxBlocks && nb * 4096 < a.c.rmax) nb *= 2;
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
  return cudaLaunchKernelEx(&cfg, k_kv4_evict, a);
}

}  // namespace paris
