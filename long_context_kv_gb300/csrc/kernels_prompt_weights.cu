// The weights that the last queries of each prompt give to its keys:
// w_j = sum over the window's (query, query head) rows n of exp(s_nj - lse_n).
//
// The product is taken with the keys as rows, S = K Q^T, so that a key is a
// lane of tensor memory and its sum stays in one thread: no reduction across
// threads, no atomics.  A block holds up to 256 window rows of a KV head
// (all of a 64-query window of four heads) in shared memory and walks a
// range of 128-key tiles; a producing warp keeps K tiles coming by TMA, an
// issuing warp runs a tile's product into one of two 256-column halves of
// tensor memory, and two groups of four warps take the exponentials of half of
// the columns each and add, while the tensor cores fill the other half of
// tensor memory.  Longer windows go by in chunks of 256 rows, each adding to
// the sums before.
//
// Bound by the read of K where the window is short, and at 256 rows by the
// exponentials and by shared memory, which the products read at 96 of its 128
// bytes a cycle (with a product of 128 columns a time it was all 128, and the
// copies of K waited for it: 23.3 us for 32K keys of 8 KV heads, against 21.3).
// Now 20.4 us there (67 MB, 3.3 TB/s), of which 5 are the start.
#include <atomic>
#include <algorithm>

#include "tc_device.cuh"

namespace paris {
namespace {

constexpr int kWStages = 4;
constexpr int kWRows = 256;            // window rows of a chunk
constexpr int kWThreads = 384;
// Up to this many sequences' tiles are cut by their lengths; more of them, or
// more KV heads of them than SMs, are a block each (and KV head).
constexpr int kCutSeqs = 160;
constexpr int kKeyBytes = kTile * kDim * 2;
constexpr int kQHalf = kWRows * 128;   // 64 channels of a chunk
constexpr size_t kWSmem = (size_t)kWStages * kKeyBytes + 2 * kQHalf + 1024;

struct WeightShared {
  uint64_t q_full, q_empty, k_full[kWStages], k_empty[kWStages], s_full[2], s_empty[2], part_full[4], drained;
  uint32_t tmem, gave_up;
  uint32_t none[2];  // of this chunk and the next: a row's lse is -inf
  float part[4][kTile];  // the second group's sums
  __align__(16) float lse[kWRows];  // base 2, negative
  int tok[kWRows];  // the row's query, counted from the chunk's first; kNoRow: it adds nothing
};

constexpr int kNoRow = -0x7fffffff - 1;  // before every key

struct WeightMaps {
  CUtensorMap q, k;
};

__global__ void __launch_bounds__(kWThreads, 1)
    k_prompt_weights(const __grid_constant__ PromptWeightArgs wa, const __grid_constant__ WeightMaps maps, int chunks) {
  extern __shared__ uint8_t dyn[];
  __shared__ __align__(16) WeightShared sh;
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(kFull, tid >> 5, 0);
  const uint32_t base = (smem_u32(dyn) + 1023u) & ~1023u, qb = base + kWStages * kKeyBytes;
  const uint32_t q_full = smem_u32(&sh.q_full), q_empty = smem_u32(&sh.q_empty), k_full = smem_u32(&sh.k_full[0]),
                 k_empty = smem_u32(&sh.k_empty[0]), s_full = smem_u32(&sh.s_full[0]), s_empty = smem_u32(&sh.s_empty[0]), part_full = smem_u32(&sh.part_full[0]);
  if (tid == 0) {
    sh.gave_up = sh.none[0] = sh.none[1] = 0;
    bar_init(q_full, 1);
    bar_init(q_empty, 1);
    bar_init(smem_u32(&sh.drained), 1);
    for (int i = 0; i < kWStages; ++i) {
      bar_init(k_full + 8 * i, 1);
      bar_init(k_empty + 8 * i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      bar_init(s_full + 8 * i, 1);
      bar_init(s_empty + 8 * i, 2 * kTile);
    }
    for (int i = 0; i < 4; ++i) bar_init(part_full + 8 * i, kTile);
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  if (warp == 8) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;\n" ::"r"(smem_u32(&sh.tmem)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::: "memory");
    tm_fence_before();
  }
  __syncthreads();
  tm_fence_after();
  const uint32_t tmem = __shfl_sync(kFull, *(volatile uint32_t*)&sh.tmem, 0);
  volatile uint32_t* gave_up = &sh.gave_up;
  auto free_tmem = [&]() {
    if (warp == 8) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;\n" ::"r"(tmem) : "memory");
  };
  pdl_wait();
  pdl_trigger();
  const PromptArgs& a = wa.p;
  // the block's part of a sequence's key tiles
  const int place = blockIdx.x / a.hkv, kvh = blockIdx.x - place * a.hkv;
  int s = place, part = 0, parts = 1;
  if (chunks > 0 && a.n_seqs == 1) {
    s = 0;
    part = place;
    parts = chunks;
  } else if (chunks > 0) {
    uint32_t tiles[kCutSeqs / 32];
#pragma unroll
    for (int i = 0; i < kCutSeqs / 32; ++i) {
      int64_t start = 0, len = 0;
      if (32 * i + lane < a.n_seqs) seq_rows(a.cu_k, 32 * i + lane, a.rows_k, start, len);
      tiles[i] = (uint32_t)((min64(len, a.max_k) + kTile - 1) / kTile);
    }
    const int3 cut = cut_tiles(tiles, (uint32_t)chunks, (uint32_t)place);
    if (cut.x < 0) {
      free_tmem();
      return;
    }
    s = cut.x;
    part = place - cut.y;
    parts = cut.z;
  }
  int64_t q0, lq, k0, lk;
  seq_rows(a.cu_q, s, a.rows_q, q0, lq);
  seq_rows(a.cu_k, s, a.rows_k, k0, lk);
  const int64_t lkm = min64(lk, a.max_k);
  const int all_tiles = (int)((lkm + kTile - 1) / kTile), per = (all_tiles + parts - 1) / parts;
  const int tile0 = part * per, ntile = min(per, all_tiles - tile0);
  if (ntile <= 0) {
    free_tmem();
    return;
  }
  const int win = (int)min64(wa.window, lq);      // queries of the window
  const int tq = kWRows / a.g;                    // of a chunk
  const int nchunk = (win + tq - 1) / tq;
  float* out = wa.weights + ((int64_t)(a.cu_k ? 0 : s) * a.hkv + kvh) * a.rows_k + k0;
  if (nchunk == 0) {
    for (int64_t j = (int64_t)tile0 * kTile + tid; j < min64(lkm, (int64_t)(tile0 + ntile) * kTile); j += kWThreads) out[j] = 0.f;
    free_tmem();
    return;
  }
  const int64_t first = lq - win;                 // first query of the window
  const int total = nchunk * ntile;               // products, chunk by chunk (the launch keeps it below 2^31)
  // rows of chunk c, and the product's N
  auto rows_of = [&](int c) { return min(tq, win - c * tq) * a.g; };

  if (warp == 9) {
    if (lane == 0) {
      int x = 0;
      bool ok = true;
      for (; ok && x < total; ++x) {
        const int c = x / ntile, st = x % kWStages, turn = x / kWStages;
        if (x % ntile == 0) {
          if (c > 0) ok = bar_wait(q_empty, (c - 1) & 1, gave_up);
          if (!ok) break;
          bar_expect(q_full, (uint32_t)(2 * tq * a.g * 128));
          for (int h = 0; h < 2; ++h)
            tma_load(qb + h * kQHalf, &maps.q, 64 * h, kvh * a.g, (int)(q0 + first) + c * tq, a.cu_q ? 0 : s, q_full);
        }
        if (turn > 0) ok = bar_wait(k_empty + 8 * st, (turn - 1) & 1, gave_up);
        if (!ok) break;
        bar_expect(k_full + 8 * st, kKeyBytes);
        for (int h = 0; h < 2; ++h)
          tma_load(base + st * kKeyBytes + h * (kKeyBytes / 2), &maps.k, 64 * h, (int)k0 + (tile0 + x % ntile) * kTile, kvh, a.cu_k ? 0 : s,
                   k_full + 8 * st);
      }
      if (x < total) {  // given up: what was issued lands before the block ends
        WaitLimit limit(now_ns());
        for (int y = max(0, x - kWStages); y < x; ++y)
          while (!bar_try(k_full + 8 * (y % kWStages), (y / kWStages) & 1) && !limit.over(now_ns())) {}
        while (x > 0 && !bar_try(q_full, ((x - 1) / ntile) & 1) && !limit.over(now_ns())) {}
      }
    }
  } else if (warp == 8) {
    auto wait = [&](uint32_t bar, uint32_t parity) { return (bool)__all_sync(kFull, bar_wait(bar, parity, gave_up)); };
    bool ok = true;
    for (int x = 0; ok && x < total; ++x) {
      const int c = x / ntile, st = x % kWStages, buf = x & 1;
      if (x % ntile == 0) ok = wait(q_full, c & 1);
      if (ok) ok = wait(k_full + 8 * st, (x / kWStages) & 1);
      if (ok && x > 1) ok = wait(s_empty + 8 * buf, ((x >> 1) - 1) & 1);
      if (!ok) break;
      if (elect()) {
        tm_fence_after();
        const uint32_t instr = mma_instr((uint32_t)(rows_of(c) + 15) & ~15u);
        const uint64_t kd = smem_desc(base + st * kKeyBytes, 16, 1024), qd = smem_desc(qb, 16, 1024);
#pragma unroll
        for (int d = 0; d < kDim / 16; ++d)
          mma_ss(tmem + buf * kWRows, kd + (d >> 2) * (kKeyBytes / 32) + (d & 3) * 2, qd + (d >> 2) * (kQHalf >> 4) + (d & 3) * 2, instr, d > 0);
        mma_commit(s_full + 8 * buf);
        mma_commit(k_empty + 8 * st);
        if (x % ntile == ntile - 1) mma_commit(q_empty);
      }
      __syncwarp();
    }
    mma_drain(smem_u32(&sh.drained));
  } else if (warp < 8) {
    const int grp = warp >> 2, row = tid & (kTile - 1);
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    bool ok = true;
    for (int c = 0; c < nchunk; ++c) {  // past a wait that gave up, only the barriers
      const int n = rows_of(c);
      // both groups are done with the last chunk's table before it changes
      asm volatile("bar.sync 1, 256;\n" ::: "memory");
      // A row whose lse is -inf adds nothing, whatever its product is.  Only the
      // path of the loop below that looks at every row leaves it out, and one
      // such row sends the whole chunk there.  (The flag goes through shared
      // memory: as a barrier's own reduction it took the kernel from 128 to 159
      // registers and 32K keys from 20.0 to 21.2 us.)
      if (tid == 0) sh.none[(c + 1) & 1] = 0;
      for (int r = tid; r < kWRows; r += 256) {
        const int64_t i = first + (int64_t)c * tq + r / a.g;
        const int h = kvh * a.g + r % a.g;
        const bool in = r < n;
        const float lse = in ? wa.lse[((int64_t)(a.cu_q ? 0 : s) * a.hq + h) * a.rows_q + q0 + i] : -INFINITY;
        sh.lse[r] = -lse * kLog2e;
        sh.tok[r] = lse == -INFINITY ? kNoRow : r / a.g;
        if (in && lse == -INFINITY) sh.none[c & 1] = 1;
      }
      asm volatile("bar.sync 1, 256;\n" ::: "memory");
      const bool none = sh.none[c & 1] != 0;
      // this group's columns: whole groups of 32 but for the last
      const int half = ((n + 1) / 2 + 31) & ~31, c0 = grp ? min(half, n) : 0, c1 = grp ? n : min(half, n);
      const int64_t least = first + (int64_t)c * tq + lk - lq;  // every row of the chunk sees this far
      const int64_t clear = none || (c1 - c0) % 32 ? -1 : least;  // tiles that end here take no look at rows
      for (int t = 0; t < ntile; ++t) {
        const int x = c * ntile + t, buf = x & 1;
        if (ok) ok = __all_sync(kFull, bar_wait(s_full + 8 * buf, (x >> 1) & 1, gave_up));
        if (!ok) break;
        tm_fence_after();
        const uint32_t ts = tmem + lanes + buf * kWRows;
        const int64_t j = (int64_t)(tile0 + t) * kTile + row;
        float sum = 0.f;
        if ((int64_t)(tile0 + t + 1) * kTile - 1 <= clear) {
          // 32 columns at a time, the next 32 on their way meanwhile
          uint32_t v[2][32];
          uint64_t sum2[2] = {0, 0};
          const uint64_t c2 = pair2(kScaleLog2, kScaleLog2);
          auto add32 = [&](const uint32_t (&y)[32], int r) {
#pragma unroll
            for (int u = 0; u < 32; u += 4) {
              const ulonglong2 l4 = *reinterpret_cast<const ulonglong2*>(&sh.lse[r + u]);
              float p[4];
              unpair2(fma2(pair2(__uint_as_float(y[u]), __uint_as_float(y[u + 1])), c2, l4.x), p[0], p[1]);
              unpair2(fma2(pair2(__uint_as_float(y[u + 2]), __uint_as_float(y[u + 3])), c2, l4.y), p[2], p[3]);
              sum2[0] = add2(sum2[0], pair2(ex2(p[0]), ex2(p[1])));
              sum2[1] = add2(sum2[1], pair2(ex2(p[2]), ex2(p[3])));
            }
          };
          if (c0 < c1) tm_ld32(v[0], 0, ts + c0);
          tm_wait_ld();
          for (int r = c0; r < c1; r += 64) {
            const bool second = r + 32 < c1, third = r + 64 < c1;
            if (second) tm_ld32(v[1], 0, ts + r + 32);
            add32(v[0], r);
            tm_wait_ld();
            if (second) {
              if (third) tm_ld32(v[0], 0, ts + r + 64);
              add32(v[1], r + 32);
              tm_wait_ld();
            }
          }
          float p0, p1;
          unpair2(add2(sum2[0], sum2[1]), p0, p1);
          sum = p0 + p1;
        } else {
          float part[4] = {0.f, 0.f, 0.f, 0.f};
          for (int r = c0; r < c1; r += 32) {
            uint32_t v[32];
            tm_ld32(v, 0, ts + r);
            tm_wait_ld();
#pragma unroll
            for (int u = 0; u < 32; ++u) {
              const float p = ex2(fmaf(__uint_as_float(v[u]), kScaleLog2, sh.lse[r + u]));
              part[u & 3] += j <= least + sh.tok[r + u] ? p : 0.f;
            }
          }
          sum = (part[0] + part[1]) + (part[2] + part[3]);
        }
        tm_fence_before();
        bar_arrive(s_empty + 8 * buf);
        // the first group adds the second's sum; a place is written again four
        // tiles later, when the first group has given back two more
        if (grp) {
          sh.part[x & 3][row] = sum;
          bar_arrive(part_full + 8 * (x & 3));
        } else {
          ok = __all_sync(kFull, bar_wait(part_full + 8 * (x & 3), (x >> 2) & 1, gave_up));
          if (!ok) break;
          sum += sh.part[x & 3][row];
          if (j < lkm) out[j] = c > 0 ? out[j] + sum : sum;
        }
      }
    }
    tm_fence_before();
  }
  __syncthreads();
  tm_fence_after();
  free_tmem();
}

cudaError_t raise_smem() {
  static std::atomic<bool> done[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || (dev >= 0 && dev < 64 && done[dev])) return e;
  e = cudaFuncSetAttribute((const void*)k_prompt_weights, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kWSmem);
  if (e == cudaSuccess && dev >= 0 && dev < 64) done[dev] = true;
  return e;
}

}  // namespace

cudaError_t prompt_weights_error(uint32_t* bits) { return take_gave_up(bits); }

cudaError_t launch_prompt_weights(const PromptWeightArgs& w, int sm_count, cudaStream_t st) {
  const PromptArgs& a = w.p;
  const int64_t ns = a.cu_q ? 1 : a.n_seqs;
  WeightMaps m;
  const void* q = a.rows_q > 0 ? a.q : a.k;  // no queries: nothing of them is loaded
  if (!encode(&m.q, q, a.hq, a.sq.head, std::max<int64_t>(1, a.rows_q), a.sq.token, ns, a.sq.seq, a.g, kWRows / a.g) ||
      !encode(&m.k, a.k, a.rows_k, a.sk.token, a.hkv, a.sk.head, ns, a.sk.seq, kTile, 1))
    return cudaErrorInvalidValue;
  cudaError_t e = raise_smem();
  if (e != cudaSuccess) return e;
  // A block per SM, and for each KV head as many chunks of the sequences' tiles
  // (six sequences of 7422 tokens in all: 10.0 -> 9.0 us against chunks cut by
  // the longest one's); a block for each sequence and KV head where those are
  // more.
  const int64_t units = (int64_t)a.n_seqs * a.hkv, tiles = (a.max_k + kTile - 1) / kTile;
  const bool cut = units <= sm_count && a.n_seqs <= kCutSeqs;
  const int64_t most = cut ? std::min<int64_t>(sm_count / a.hkv, a.n_seqs * tiles) : 0;
  const int64_t chunk = kWRows / a.g, chunks = (std::min<int64_t>(w.window, a.rows_q) + chunk - 1) / chunk;
  if (chunks * tiles > 0x7fffffff) return cudaErrorInvalidValue;
  return launch_pdl(k_prompt_weights, dim3((unsigned)(cut ? most * a.hkv : units)), dim3(kWThreads), kWSmem, st, w, m, (int)most);
}

}  // namespace paris
