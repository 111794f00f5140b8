// Causal attention over prompts.
//
//   s_ij = <q_i, k_j> / sqrt(d),  j <= i + len_k - len_q,
//   o_i = sum_j exp(s_ij - m_i) v_j / sum_j exp(s_ij - m_i)
//
// with the running maximum m_i of one pass over the keys.  k_prompt_attend has
// a block per SM that walks items: 256 query rows of a KV head and a range of
// its keys.  A query row is a (token, query head) pair with the heads fastest,
// so the G heads of a KV head share every key and value tile and a tile of
// rows spans only 128 / G tokens of the diagonal.  Work is split by role:
//   - a producing warp finds the items, longest first, and copies the query
//     tiles and then the 128-key tiles of K and V with TMA into a ring of
//     shared-memory stages, the next item's while this one still computes;
//   - an issuing warp runs the products on the tensor cores: S = Q K^T of both
//     128-row tiles into tensor memory, then, as soon as a tile's weights are
//     there, O += P V (P read from tensor memory, where it replaces S) and the
//     next S of the same tile;
//   - two groups of four warps, one per tile, turn S into P, a thread per row:
//     maximum, exp2, sum, all in registers.
// While one tile is in its softmax the tensor cores work for the other.  The
// products of a block run in the order of their issue, so S of step j being
// complete means that O holds steps up to j - 1: a row whose maximum grew by
// more than 2^8 rescales O right then, and the others do not touch it.
//
// Bound by the tensor cores (4 d flops a visible pair), and right under them
// by shared memory: a step of both tiles and 128 keys is 2048 cycles of
// products, whose operands and copies are 256 KB at 128 bytes a cycle, again
// 2048; it takes 2900 to 3300 (32768 tokens of 8 query heads: 1.39 ms among
// other passes, 1584 TFLOP/s, 0.81 of the measured bf16 rate in bursts and 0.93
// of the sustained one).  What the steps measured:
// operands kept in uniform registers by electing the issuing lane, 2474 ->
// 1446 us there; a block per item instead of per SM, 1468 against 1364 us; an
// eighth of the exponentials by a polynomial in the FMA units, 1406 against
// 1331 us: the special-function units are not what a step waits for.  An
// item's result takes 4000 cycles more, in which its tile's group does nothing
// else; that is 15 % of a batch of short prompts.
//
// The weights enter P V as bf16, their sum as float32: both operands of a
// product are of one type, V's, and a second product for what the rounding
// leaves would be half as many operations again on what bounds the kernel.  The
// largest error against 64 bits is 2.1e-3 to 2.3e-3 of the result's size, and
// 1.6e-3 with float32 weights, nearly all of it the result's own rounding.
//
// What a row does not see has weight 0, but 0 times an infinity or NaN in V
// is NaN: value rows past the end of a sequence are cleared in shared memory,
// and a row whose result is not finite is computed again, when the block's
// items are done, by prompt_row, which reads only what the row sees.
#include <atomic>
#include <algorithm>

#include "tc_device.cuh"

namespace paris {
namespace {

constexpr int kRowWarps = 8;

__device__ __forceinline__ float dot8(uint4 a, uint4 b, float acc) {
  const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    acc = fmaf(bf16_bits_to_float(x[i] & 0xffffu), bf16_bits_to_float(y[i] & 0xffffu), acc);
    acc = fmaf(__uint_as_float(x[i] & 0xffff0000u), __uint_as_float(y[i] & 0xffff0000u), acc);
  }
  return acc;
}

// A weight's exponent is one fma of the product, the scale and the maximum, in
// which the maximum's own rounding, 2^-24 of it, is left over.  It does no harm
// while weights stay within float32 and bf16, as a row's sum and result are off
// by the same factor; from a maximum of 2^31 on they would not, and rows past
// 2^29 are left to prompt_row, whose largest weight is 1 at any size.
__device__ __forceinline__ bool too_far(float m) { return fabsf(m) > 536870912.f && m != -INFINITY; }

// One query row by one warp: its visible keys 32 at a time, a lane per key
// for the scores, four channels per lane for the weighted sum.  Only rows
// that the query sees are read.  The sum is held as the mean so far, which
// stays within the values' range where the plain sum may not.
__device__ __noinline__ void prompt_row(const PromptArgs& a, int s, int h, int64_t q0, int64_t i, int64_t k0, int64_t visible) {
  const int lane = threadIdx.x & 31;
  const int kvh = h / a.g;
  const uint4* q = reinterpret_cast<const uint4*>(a.q + (a.cu_q ? 0 : s * a.sq.seq) + (q0 + i) * a.sq.token + h * a.sq.head);
  const __nv_bfloat16* k = a.k + (a.cu_k ? 0 : s * a.sk.seq) + k0 * a.sk.token + kvh * a.sk.head;
  const __nv_bfloat16* v = a.v + (a.cu_k ? 0 : s * a.sv.seq) + k0 * a.sv.token + kvh * a.sv.head;
  float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
  for (int64_t j0 = 0; j0 < visible; j0 += 32) {
    const int n = (int)min64(32, visible - j0);
    float sc = -INFINITY;
    if (lane < n) {
      const uint4* kr = reinterpret_cast<const uint4*>(k + (j0 + lane) * a.sk.token);
      float acc = 0.f;
#pragma unroll 4
      for (int c = 0; c < 16; ++c) acc = dot8(kr[c], __ldg(q + c), acc);
      sc = acc * kScaleLog2;
    }
    float mx = sc;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, off));
    const float mn = fmaxf(m, mx);
    const float f = m == mn ? 1.f : exp2f(m - mn);
    m = mn;
    const float p = sc == -INFINITY ? 0.f : exp2f(sc - m);  // no weight, and m may be -inf too
    float ps = p;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) ps += __shfl_xor_sync(kFull, ps, off);
    const float before = l * f;
    l = before + ps;
    const float per = l != 0.f ? 1.f / l : 0.f, share = p * per, old = before * per;  // l is 1 at least, or 0
#pragma unroll
    for (int c = 0; c < 4; ++c) o[c] *= old;
    for (int j = 0; j < n; ++j) {
      const float pj = __shfl_sync(kFull, share, j);
      float vy[4];
      load4(v + (j0 + j) * a.sv.token, 1, 4 * lane, vy);
#pragma unroll
      for (int c = 0; c < 4; ++c) o[c] = fmaf(pj, vy[c], o[c]);
    }
  }
  __nv_bfloat16* out = a.out + (a.cu_q ? 0 : s * a.so.seq) + (q0 + i) * a.so.token + h * a.so.head;
  *reinterpret_cast<uint2*>(out + 4 * lane) = make_uint2(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]));
  if (a.lse != nullptr && lane == 0)
    a.lse[((int64_t)(a.cu_q ? 0 : s) * a.hq + h) * a.rows_q + q0 + i] = visible > 0 ? (m + log2f(l)) * kLn2 : -INFINITY;
}

// ------------------------------------------------------------ the tensor-core kernel
constexpr int kTiles = 2;             // query tiles of a block
constexpr int kStages = 5;            // K and V tiles in flight
constexpr int kTileBytes = kTile * kDim * 2;
constexpr int kHalfBytes = kTileBytes / 2;  // 64 channels of a tile: rows of 128 bytes, swizzled
constexpr int kPromptThreads = 384;   // two softmax groups; a group with the issuing and the producing warp
// Registers of a thread: 168 at launch (65536 / 384); the third group gives
// up what the softmax groups, with a whole row of S each, need:
// 2 x 216 + 72 = 3 x 168.
constexpr int kSoftmaxRegs = 216, kIssueRegs = 72;
constexpr int kPartRow = kDim + 4;    // partial of a row: maximum, sum, number of its parts, -, o
constexpr float kGrowth = 8.f;        // a row's maximum may lag this far (base 2): weights stay below 2^8
constexpr size_t kPromptSmem = (size_t)(kTiles + kStages) * kTileBytes + 1024;

struct PromptMaps {
  CUtensorMap q, k, v;
};

// A block's piece of work: 256 query rows of a KV head and a range of keys.
struct PromptItem {
  int s, kvh, qb;
  int part, parts;      // of the keys, where several blocks share them
  int q0, lq, k0, lk;
  int t0;               // first token of tile 0
  int jb, end[kTiles];  // key blocks [jb, end) of each tile
};

constexpr int kItems = 4;

struct PromptShared {
  uint64_t q_full, q_empty, full[kStages], empty[kStages], s_full[kTiles], p_full[2 * kTiles], o_full[kTiles], o_empty[kTiles];
  uint64_t item_full[kItems], item_empty[kItems], drained;
  PromptItem items[kItems];  // s < 0: no more
  uint32_t tmem;
  uint32_t gave_up;
};

__device__ __forceinline__ int blocks_of(int64_t lq, int tokens) { return (int)((lq + tokens - 1) / tokens); }

// Up to this many packed sequences are walked by query block, with a few
// looks at every length for each item; more of them one after the other.
constexpr int kFewSeqs = 64;

// What a producing warp keeps from item to item: of few sequences a lane's
// two numbers of query blocks; of many, where the walk over them has come to
// (those before s0 have `before` query blocks).
struct PromptCursor {
  int64_t units;  // (query block, sequence, KV head)s in all
  int few[kFewSeqs / 32];
  int s0;
  int64_t before;
};

// Query blocks of sequence s (0: there is no such sequence).
__device__ __forceinline__ int seq_blocks(const PromptArgs& a, int s, int tokens) {
  if (s >= a.n_seqs) return 0;
  int64_t q0, lq;
  seq_rows(a.cu_q, s, a.rows_q, q0, lq);
  return blocks_of(min64(lq, a.max_q), tokens);
}

__device__ __forceinline__ PromptCursor first_cursor(const PromptArgs& a) {
  const int lane = threadIdx.x & 31, tokens = kTiles * (kTile / a.g);
  PromptCursor cur{};
  if (a.cu_q == nullptr) {
    cur.units = (int64_t)blocks_of(a.max_q, tokens) * a.n_seqs;
  } else {
#pragma unroll
    for (int i = 0; i < kFewSeqs / 32; ++i) {
      cur.few[i] = seq_blocks(a, 32 * i + lane, tokens);
      cur.units += __reduce_add_sync(kFull, (uint32_t)cur.few[i]);
    }
    for (int s0 = kFewSeqs; s0 < a.n_seqs; s0 += 32) cur.units += __reduce_add_sync(kFull, (uint32_t)seq_blocks(a, s0 + lane, tokens));
  }
  cur.units *= a.hkv;
  return cur;
}

// Item `it` of this block (a warp computes it).  False: there is no such item.
//
// Units are numbered by query block in descending order, so that those that
// see most keys come first, and for each the sequences that have it and the KV
// heads; of more than kFewSeqs sequences, their query blocks in turn.  Where
// there are units for all blocks, a block takes one of every turn of the grid,
// every other turn backwards: who had the longest of one turn has the
// shortest of the next.  Where there are fewer (nsplit > 1), block c of G
// takes the c-th G-th part of all the units' keys, taken to be equally many:
// the end of one unit, maybe whole ones, and the beginning of another.
__device__ __forceinline__ bool prompt_item(const PromptArgs& a, int it, PromptCursor& cur, PromptItem& w) {
  const int lane = threadIdx.x & 31;
  const int tq = kTile / a.g, tokens = kTiles * tq;
  int64_t x, from_part = 0, to_part = 1, blocks = 1;  // the unit; its keys from from_part / blocks to to_part / blocks
  w.part = 0;
  w.parts = 1;
  if (a.nsplit > 1) {
    const int64_t c = blockIdx.x, u = cur.units;
    blocks = min64(gridDim.x, u * (a.nsplit - 1));
    if (c >= blocks) return false;
    const int64_t lo = c * u, hi = lo + u;  // in blocks-ths of a unit
    x = lo / blocks + it;
    if (x * blocks >= hi) return false;
    from_part = max64(lo - x * blocks, 0);
    to_part = min64(hi - x * blocks, blocks);
    const int64_t first = x * blocks / u, last = ((x + 1) * blocks - 1) / u;
    w.part = (int)(c - first);
    w.parts = (int)(last - first + 1);
  } else {
    x = (int64_t)it * gridDim.x + (it & 1 ? (int)gridDim.x - 1 - (int)blockIdx.x : (int)blockIdx.x);
    if (x >= cur.units) return false;
  }
  const int64_t y = x / a.hkv;  // (query block, sequence)
  w.kvh = (int)(x - y * a.hkv);
  if (a.cu_q == nullptr) {
    const int nqb = blocks_of(a.max_q, tokens);
    w.qb = nqb - 1 - (int)(y / a.n_seqs);
    w.s = (int)(y % a.n_seqs);
  } else {
    if (a.n_seqs > kFewSeqs) {
      for (;; cur.s0 += 32) {
        if (cur.s0 >= a.n_seqs) return false;  // not for a unit
        const int n = seq_blocks(a, cur.s0 + lane, tokens);
        const uint32_t inc = warp_incl_scan((uint32_t)n, lane), all = __shfl_sync(kFull, inc, 31);
        const int64_t j = y - cur.before;
        if (j < all) {
          const int src = __popc(__ballot_sync(kFull, inc <= j));  // the lanes before it
          w.s = cur.s0 + src;
          // the longest of a sequence's blocks first
          w.qb = (int)(__shfl_sync(kFull, inc, src) - 1 - j);
          break;
        }
        cur.before += all;
      }
    } else {
      // number of (block, sequence) pairs with block >= level
      auto from = [&](int level) -> int64_t {
        int64_t n = 0;
#pragma unroll
        for (int i = 0; i < kFewSeqs / 32; ++i) n += __reduce_add_sync(kFull, (uint32_t)max(0, cur.few[i] - level));
        return n;
      };
      int lo = 0, hi = blocks_of(a.max_q, tokens);  // from(lo) > y >= from(hi)
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (from(mid) > y) lo = mid;
        else hi = mid;
      }
      int64_t j = y - from(lo + 1);  // among the sequences that have block lo
      w.qb = lo;
      w.s = 0;
#pragma unroll
      for (int i = 0; i < kFewSeqs / 32; ++i) {
        const uint32_t has = __ballot_sync(kFull, cur.few[i] > lo);
        const int n = __popc(has);
        if (j < n) {
          uint32_t m = has;
          for (int x = 0; x < j; ++x) m &= m - 1;
          w.s = 32 * i + __ffs(m) - 1;
          break;
        }
        j -= n;
      }
    }
  }
  int64_t q0, lq, k0, lk;
  seq_rows(a.cu_q, w.s, a.rows_q, q0, lq);
  seq_rows(a.cu_k, w.s, a.rows_k, k0, lk);
  w.q0 = (int)q0;
  w.lq = (int)lq;
  w.k0 = (int)k0;
  w.lk = (int)lk;
  w.t0 = w.qb * tokens;
  const int64_t rows = min64(lq, a.max_q);
  // keys of each tile: up to what its last token sees
  int n[kTiles], most = 0;
#pragma unroll
  for (int i = 0; i < kTiles; ++i) {
    const int64_t first = w.t0 + i * tq, last = min64(first + tq, rows) - 1;
    const int64_t seen = first <= last ? min64(lk, last + lk - lq + 1) : 0;
    n[i] = seen > 0 ? (int)((seen + kTile - 1) / kTile) : 0;
    most = max(most, n[i]);
  }
  w.jb = (int)(most * from_part / blocks);
  const int to = (int)(most * to_part / blocks);
#pragma unroll
  for (int i = 0; i < kTiles; ++i) w.end[i] = max(w.jb, min(n[i], to));
  return true;
}

// A softmax warp's rows of all the block's items once more: those whose result
// is not finite are computed again.  That takes as long as there are keys
// (32 rows of each of eight warps that see 65536 keys: 0.35 s), so it waits
// until every item is done and no role waits for another: what is in V decides
// how long it takes, and no wait's limit may depend on that.
__device__ __noinline__ void prompt_again(const PromptArgs& a) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int tq = kTile / a.g, first = (warp & 3) * 32;
  PromptCursor cur = first_cursor(a);
  PromptItem w;
  __syncwarp();  // a row was stored by several lanes, and is read by all
  for (int it = 0; prompt_item(a, it, cur, w); ++it) {
    const int n = (int)min64(w.lq, a.max_q);
    for (int r = first; r < min(first + 32, tq * a.g); ++r) {
      const int tok = w.t0 + (warp >> 2) * tq + r / a.g, h = w.kvh * a.g + r % a.g;
      if (tok >= n) break;
      const __nv_bfloat16* out = a.out + (a.cu_q ? 0 : w.s * a.so.seq) + (int64_t)(w.q0 + tok) * a.so.token + h * a.so.head;
      const uint2 y = *reinterpret_cast<const uint2*>(out + 4 * lane);
      const uint32_t x = y.x & 0x7f807f80u, z = y.y & 0x7f807f80u;  // exponents; all ones: infinities and NaN
      const bool bad = (x & 0xffffu) == 0x7f80u || x >> 16 == 0x7f80u || (z & 0xffffu) == 0x7f80u || z >> 16 == 0x7f80u;
      if (__any_sync(kFull, bad)) prompt_row(a, w.s, h, w.q0, tok, w.k0, min(w.lk, tok + w.lk - w.lq + 1));
    }
  }
}

__global__ void __launch_bounds__(kPromptThreads, 1)
    k_prompt_attend(const __grid_constant__ PromptArgs a, const __grid_constant__ PromptMaps maps) {
  extern __shared__ uint8_t dyn[];
  __shared__ PromptShared sh;
  const uint32_t base = (smem_u32(dyn) + 1023u) & ~1023u;
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(kFull, tid >> 5, 0);  // the same for the warp, and known to be
  const uint32_t q_full = smem_u32(&sh.q_full), q_empty = smem_u32(&sh.q_empty), full = smem_u32(&sh.full[0]), empty = smem_u32(&sh.empty[0]);
  const uint32_t s_full = smem_u32(&sh.s_full[0]), p_full = smem_u32(&sh.p_full[0]), o_full = smem_u32(&sh.o_full[0]),
                 o_empty = smem_u32(&sh.o_empty[0]), item_full = smem_u32(&sh.item_full[0]), item_empty = smem_u32(&sh.item_empty[0]);
  if (tid == 0) {
    sh.gave_up = 0;
    bar_init(q_full, 1);
    bar_init(q_empty, 1);
    for (int i = 0; i < kStages; ++i) {
      bar_init(full + 8 * i, 1);
      bar_init(empty + 8 * i, 1);
    }
    for (int i = 0; i < kTiles; ++i) {
      bar_init(s_full + 8 * i, 1);
      bar_init(p_full + 16 * i, kTile);
      bar_init(p_full + 16 * i + 8, kTile);
      bar_init(o_full + 8 * i, 1);
      bar_init(o_empty + 8 * i, kTile);
    }
    bar_init(smem_u32(&sh.drained), 1);
    for (int i = 0; i < kItems; ++i) {
      bar_init(item_full + 8 * i, 1);
      bar_init(item_empty + 8 * i, 9);  // the issuing warp and eight softmax warps
    }
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  if (warp == 8) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;\n" ::"r"(smem_u32(&sh.tmem)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::: "memory");
    tm_fence_before();
  }
  __syncthreads();
  tm_fence_after();
  pdl_wait();
  pdl_trigger();
  const uint32_t tmem = __shfl_sync(kFull, *(volatile uint32_t*)&sh.tmem, 0);
  volatile uint32_t* gave_up = &sh.gave_up;
  const uint32_t ring = base + kTiles * kTileBytes;

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kIssueRegs));
    auto wait = [&](uint32_t bar, uint32_t parity) { return (bool)__all_sync(kFull, bar_wait(bar, parity, gave_up)); };
    if (warp == 9) {
      // ---- producer: items, queries, keys and values
      const int tq = kTile / a.g;
      int nq = 0, x = 0;  // query loads, ring loads so far
      bool ok = true;
      PromptCursor cur = first_cursor(a);
      auto item = [&](int it, PromptItem& w) { return prompt_item(a, it, cur, w); };
      PromptItem w, next;
      bool more = item(0, next);
      for (int it = 0; ok; ++it) {
        w = next;
        if (!more) w.s = -1;
        if (it >= kItems) ok = wait(item_empty + 8 * (it % kItems), (it / kItems - 1) & 1);
        if (!ok) break;
        if (lane == 0) {
          sh.items[it % kItems] = w;
          bar_arrive(item_full + 8 * (it % kItems));
        }
        if (!more) break;
        const int jb = w.jb, e = max(w.end[0], w.end[1]), loads = 2 * (e - jb);
        if (loads == 0) {
          more = item(it + 1, next);
          continue;
        }
        if (nq > 0) ok = wait(q_empty, (nq - 1) & 1);
        if (!ok) break;
        const int qseq = a.cu_q ? 0 : w.s, kseq = a.cu_k ? 0 : w.s;
        if (lane == 0) {
          bar_expect(q_full, (uint32_t)(kTiles * 2 * tq * a.g * 128));
          for (int i = 0; i < kTiles; ++i)
            for (int h = 0; h < 2; ++h)
              tma_load(base + i * kTileBytes + h * kHalfBytes, &maps.q, 64 * h, w.kvh * a.g, w.q0 + w.t0 + i * tq, qseq, q_full);
        }
        ++nq;
        for (int j = 0; ok && j < loads; ++j) {
          const int st = x % kStages, turn = x / kStages;
          if (turn > 0) ok = wait(empty + 8 * st, (turn - 1) & 1);
          if (!ok) break;
          if (lane == 0) {
            bar_expect(full + 8 * st, kTileBytes);
            const CUtensorMap* m = (j & 1) ? &maps.v : &maps.k;
            const int row = w.k0 + (jb + (j >> 1)) * kTile;
            for (int h = 0; h < 2; ++h) tma_load(ring + st * kTileBytes + h * kHalfBytes, m, 64 * h, row, w.kvh, kseq, full + 8 * st);
          }
          ++x;
          // the ring is full for now: time to find the next item
          if (j == min(loads, kStages) - 1) more = item(it + 1, next);
        }
      }
      if (!ok && lane == 0) {  // given up: what was issued lands before the block ends
        WaitLimit limit(now_ns());
        while (nq > 0 && !bar_try(q_full, (nq - 1) & 1) && !limit.over(now_ns())) {}
        for (int y = max(0, x - kStages); y < x; ++y)
          while (!bar_try(full + 8 * (y % kStages), (y / kStages) & 1) && !limit.over(now_ns())) {}
      }
    } else if (warp == 8) {
      // ---- products (the whole warp walks; one lane issues)
      bool ok = true;
      int nq = 0, x = 0;              // items with keys, ring stages so far
      int ns[kTiles] = {0, 0};        // steps of each tile so far
      int no[kTiles] = {0, 0};        // results of each tile so far
      auto scores = [&](int i, int xs) {  // S_i = Q_i K^T with the key tile in stage xs
        const uint32_t qa = base + i * kTileBytes, kb = ring + (xs % kStages) * kTileBytes;
        const uint64_t qd = smem_desc(qa, 16, 1024), kd = smem_desc(kb, 16, 1024);
#pragma unroll
        for (int c = 0; c < kDim / 16; ++c) {
          const uint32_t off = (c >> 2) * (kHalfBytes >> 4) + (c & 3) * 2;
          mma_ss(tmem + i * kTile, qd + off, kd + off, mma_instr(kTile), c > 0);
        }
        mma_commit(s_full + 8 * i);
      };
      for (int it = 0; ok; ++it) {
        ok = wait(item_full + 8 * (it % kItems), (it / kItems) & 1);
        if (!ok) break;
        const volatile PromptItem& w = sh.items[it % kItems];
        if (__shfl_sync(kFull, w.s, 0) < 0) break;
        const int jb = __shfl_sync(kFull, w.jb, 0), lk = __shfl_sync(kFull, w.lk, 0);  // every lane has read it
        const int ends[kTiles] = {__shfl_sync(kFull, w.end[0], 0), __shfl_sync(kFull, w.end[1], 0)};
        const int e = max(ends[0], ends[1]);
        if (lane == 0) bar_arrive(item_empty + 8 * (it % kItems));
        if (e == jb) continue;
        ok = wait(q_full, nq & 1);
        ++nq;
        if (ok) ok = wait(full + 8 * (x % kStages), (x / kStages) & 1);
        if (ok && elect()) {
          tm_fence_after();
          for (int i = 0; i < kTiles; ++i)
            if (jb < ends[i]) scores(i, x);
          mma_commit(empty + 8 * (x % kStages));
          if (e == jb + 1) mma_commit(q_empty);
        }
        __syncwarp();
        const int tail = lk % kTile;  // keys of the sequence's last, unfilled block
        for (int j = jb; ok && j < e; ++j) {
          const int xv = x + 1, xk = x + 2;
          ok = wait(full + 8 * (xv % kStages), (xv / kStages) & 1);
          if (ok && j + 1 < e) ok = wait(full + 8 * (xk % kStages), (xk / kStages) & 1);
          if (!ok) break;
          const uint32_t vb = ring + (xv % kStages) * kTileBytes;
          if (tail && j == lk / kTile) {
            // value rows past the sequence's end: anything times weight 0 is 0
            for (int y = tail * 8 + lane; y < kTile * 8; y += 32)
              for (int h = 0; h < 2; ++h)
                asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};\n" ::"r"(vb + h * kHalfBytes + y * 16), "r"(0) : "memory");
            asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
            __syncwarp();
          }
#pragma unroll
          for (int i = 0; i < kTiles; ++i) {
            const bool mine = j < ends[i];
            // 16 keys a product: 8 columns of weights, 16 rows of V
            const uint64_t vd = smem_desc(vb, kHalfBytes, 1024);
            auto values = [&](int c) {
              mma_ts(tmem + (2 + i) * kTile, tmem + i * kTile + 8 * c, vd + c * 128, mma_instr(kTile) | kMmaBN, j > jb || c > 0);
            };
            // the last result has been read before the first product replaces it
            if (ok && mine && j == jb && no[i] > 0) ok = wait(o_empty + 8 * i, (no[i] - 1) & 1);
            if (ok && mine) ok = wait(p_full + 16 * i, ns[i] & 1);
            if (ok && mine && elect()) {
              tm_fence_after();
#pragma unroll
              for (int c = 0; c < 6; ++c) values(c);
            }
            __syncwarp();
            if (ok && mine) ok = wait(p_full + 16 * i + 8, ns[i] & 1);
            if (ok && mine && elect()) {
              tm_fence_after();
              values(6);
              values(7);
              if (j + 1 == ends[i]) mma_commit(o_full + 8 * i);
              if (j + 1 < ends[i]) scores(i, xk);
            }
            __syncwarp();
            if (mine) ++ns[i];
            if (mine && j + 1 == ends[i]) ++no[i];
          }
          if (ok && elect()) {
            mma_commit(empty + 8 * (xv % kStages));
            if (j + 1 < e) mma_commit(empty + 8 * (xk % kStages));
            if (j + 2 == e) mma_commit(q_empty);  // the item's last scores
          }
          __syncwarp();
          x += 2;
        }
      }
      mma_drain(smem_u32(&sh.drained));
    }
  } else {
    // ---- softmax of tile i, a row per thread
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(kSoftmaxRegs));
    const int i = warp >> 2, row = tid & (kTile - 1);
    const int tq = kTile / a.g;
    const int row_tok = row / a.g, row_head = row % a.g;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + lanes + i * kTile, to = tmem + lanes + (2 + i) * kTile;
    bool ok = true, again = false;  // again: a row's result is not finite
    uint32_t ns = 0, no = 0;  // steps and results of the tile so far
    for (int it = 0; ok; ++it) {
      ok = __all_sync(kFull, bar_wait(item_full + 8 * (it % kItems), (it / kItems) & 1, gave_up));
      if (!ok) break;
      const volatile PromptItem& w = sh.items[it % kItems];
      const int ws = __shfl_sync(kFull, w.s, 0);
      if (ws < 0) break;
      const int jb = __shfl_sync(kFull, w.jb, 0), end = __shfl_sync(kFull, w.end[i], 0);
      const int lq = w.lq, lk = w.lk, q0 = w.q0;
      const int first_tok = w.t0 + i * tq, tok = first_tok + row_tok;
      const bool live = row < tq * a.g && tok < (int)min64(lq, a.max_q);
      const int h = w.kvh * a.g + row_head;
      // the last key the row sees; rows that are not there see what the first does
      const int last_key = min(lk, (live ? tok : first_tok) + lk - lq + 1) - 1;
      const int tile_key = min(lk, first_tok + lk - lq + 1) - 1;  // every row of the tile sees this far
      float* part = nullptr;
      if (a.nsplit > 1) {
        const int64_t nqb = (a.max_q + kTiles * tq - 1) / (kTiles * tq);
        part = a.ws + (((((int64_t)ws * a.hkv + w.kvh) * nqb + w.qb) * a.nsplit + w.part) * (kTiles * kTile) + i * kTile + row) * kPartRow;
      }
      if (part != nullptr && live) part[2] = __int_as_float(w.parts);
      __syncwarp();
      if (lane == 0) bar_arrive(item_empty + 8 * (it % kItems));
      float m = -INFINITY, l = 0.f;  // base 2
      for (int j = jb; j < end; ++j) {
        ok = __all_sync(kFull, bar_wait(s_full + 8 * i, ns & 1, gave_up));
        if (!ok) break;
        ++ns;
        tm_fence_after();
        uint32_t s[kTile];
        tm_ld32(s, 0, ts);
        tm_wait_ld();
        tm_ld32(s, 32, ts + 32);
        tm_ld32(s, 64, ts + 64);
        tm_ld32(s, 96, ts + 96);
        const bool cut = (j + 1) * kTile - 1 > tile_key;
        const int left = last_key - j * kTile;  // last visible column
        if (cut) {
#pragma unroll
          for (int c = 0; c < 32; ++c)
            if (c > left) s[c] = 0xff800000u;  // -inf
        }
        // The first weights are taken with the maximum so far, while the other
        // scores are on their way and before the block's own maximum is found;
        // only a row that grew past kGrowth does them again.
        const uint64_t c2 = pair2(kScaleLog2, kScaleLog2);
        uint64_t sum0 = 0, sum1 = 0;
        auto four = [&](int c, uint64_t n2, uint32_t& lo, uint32_t& hi) {
          float x0, x1, x2, x3;
          unpair2(fma2(pair2(__uint_as_float(s[c]), __uint_as_float(s[c + 1])), c2, n2), x0, x1);
          unpair2(fma2(pair2(__uint_as_float(s[c + 2]), __uint_as_float(s[c + 3])), c2, n2), x2, x3);
          x0 = ex2(x0);
          x1 = ex2(x1);
          x2 = ex2(x2);
          x3 = ex2(x3);
          sum0 = add2(sum0, pair2(x0, x1));
          sum1 = add2(sum1, pair2(x2, x3));
          lo = pack_bf16x2(x0, x1);
          hi = pack_bf16x2(x2, x3);
        };
        uint32_t first[16];
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        float neg = m == -INFINITY ? 0.f : -m;
#pragma unroll
        for (int c = 0; c < 32; c += 4) {
          four(c, pair2(neg, neg), first[c / 2], first[c / 2 + 1]);
          mx[0] = fmaxf(mx[0], fmaxf(__uint_as_float(s[c]), __uint_as_float(s[c + 1])));
          mx[1] = fmaxf(mx[1], fmaxf(__uint_as_float(s[c + 2]), __uint_as_float(s[c + 3])));
        }
        tm_wait_ld();
        hold32(s, 32);
        hold32(s, 64);
        hold32(s, 96);
        if (cut) {
#pragma unroll
          for (int c = 32; c < kTile; ++c)
            if (c > left) s[c] = 0xff800000u;
        }
#pragma unroll
        for (int u = 16; u < 64; ++u)
          mx[u & 3] = fmaxf(mx[u & 3], fmaxf(__uint_as_float(s[2 * u]), __uint_as_float(s[2 * u + 1])));
        const float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * kScaleLog2;
        const bool grew = mt > m + kGrowth;
        if (__any_sync(kFull, grew)) {
          const float f = grew ? ex2(m - mt) : 1.f;
          if (j > jb) {
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
              uint32_t o[32];
              tm_ld32(o, 0, to + 32 * c);
              tm_wait_ld();
#pragma unroll
              for (int u = 0; u < 32; ++u) o[u] = __float_as_uint(__uint_as_float(o[u]) * f);
              tm_st32(to + 32 * c, o, 0);
            }
          }
          l *= f;
          if (grew) m = mt;
          neg = m == -INFINITY ? 0.f : -m;
          sum0 = sum1 = 0;
#pragma unroll
          for (int c = 0; c < 32; c += 4) four(c, pair2(neg, neg), first[c / 2], first[c / 2 + 1]);
        }
        const uint64_t n2 = pair2(neg, neg);
#pragma unroll
        for (int c = 0; c < 16; ++c) s[c] = first[c];
#pragma unroll
        for (int c = 32; c < 64; c += 4) four(c, n2, s[c / 2], s[c / 2 + 1]);
        tm_st32(ts, s, 0);
#pragma unroll
        for (int c = 64; c < 96; c += 4) four(c, n2, s[c / 2], s[c / 2 + 1]);
        tm_st16(ts + 32, s, 32);
        tm_wait_st();
        tm_fence_before();
        bar_arrive(p_full + 16 * i);  // the products may start on 96 keys
#pragma unroll
        for (int c = 96; c < 128; c += 4) four(c, n2, s[c / 2], s[c / 2 + 1]);
        tm_st16(ts + 48, s, 48);
        tm_wait_st();
        tm_fence_before();
        bar_arrive(p_full + 16 * i + 8);
        float a0, a1;
        unpair2(add2(sum0, sum1), a0, a1);
        l += a0 + a1;
      }
      // ---- result
      const bool any = end > jb;
      if (any && ok) ok = bar_wait(o_full + 8 * i, no & 1, gave_up);
      ok = __all_sync(kFull, ok);
      if (!ok) break;
      if (any) {
        ++no;
        tm_fence_after();
      }
      const float inv = too_far(m) ? NAN : l != 0.f ? 1.f / l : 0.f;  // a row that sees nothing: 0
      // 0 times every value, added up: 0 but for infinities and NaN
      uint64_t none = 0;
      const uint64_t inv2 = pair2(inv, inv);
      // A lane has a row; stored like that, a warp's 16-byte pieces lie in 32
      // lines (4500 cycles an item).  So eight lanes exchange 128 bytes of
      // their eight rows at a time, and four whole lines are stored at once.
      char* to_row = nullptr;
      if (live) to_row = part != nullptr ? reinterpret_cast<char*>(part + 4)
                                         : reinterpret_cast<char*>(a.out + (a.cu_q ? 0 : ws * a.so.seq) + (int64_t)(q0 + tok) * a.so.token + h * a.so.head);
      auto store_lines = [&](uint32_t (&v)[32], int at) {  // 128 bytes of every row, `at` bytes into it
        // eight by eight pieces: (lane, piece) and (piece, lane) change places
        // where bit b of the two differs, for one b after the other
#pragma unroll
        for (int b = 1; b < 8; b <<= 1) {
          const bool up = lane & b;
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            if (c & b) continue;
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              uint32_t &p = v[4 * c + x], &q = v[4 * (c | b) + x];
              const uint32_t got = __shfl_xor_sync(kFull, up ? p : q, b);
              if (up) p = got;
              else q = got;
            }
          }
        }
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          char* to = reinterpret_cast<char*>(__shfl_sync(kFull, reinterpret_cast<unsigned long long>(to_row), (lane & ~7) + c));
          if (to != nullptr) *reinterpret_cast<uint4*>(to + at + 16 * (lane & 7)) = make_uint4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
        }
      };
      // one copy of the code: it runs once an item and is fetched anew
      const int cols = part != nullptr ? 32 : 64;  // columns in 128 bytes
#pragma unroll 1
      for (int c = 0; c < kDim; c += cols) {
        uint32_t v[32];
        if (!any) {
#pragma unroll
          for (int u = 0; u < 32; ++u) v[u] = 0;
        } else if (part != nullptr) {
          tm_ld32(v, 0, to + c);
          tm_wait_ld();
        } else {
          uint32_t o[64];
          tm_ld32(o, 0, to + c);
          tm_ld32(o, 32, to + c + 32);
          tm_wait_ld();
#pragma unroll
          for (int u = 0; u < 64; u += 2) {
            const uint64_t y = mul2(pair2(__uint_as_float(o[u]), __uint_as_float(o[u + 1])), inv2);
            none = fma2(y, 0, none);
            float y0, y1;
            unpair2(y, y0, y1);
            v[u / 2] = pack_bf16x2(y0, y1);
          }
        }
        if (any && c + cols == kDim) {  // the next item's products may replace it
          tm_fence_before();
          bar_arrive(o_empty + 8 * i);
        }
        store_lines(v, c / cols * 128);
      }
      if (part != nullptr) {
        if (live) {
          part[0] = m;
          part[1] = l;
        }
      } else {
        if (live && a.lse != nullptr)
          a.lse[((int64_t)(a.cu_q ? 0 : ws) * a.hq + h) * a.rows_q + q0 + tok] = last_key >= 0 ? (m + log2f(l)) * kLn2 : -INFINITY;
        float z0, z1;
        unpair2(none, z0, z1);
        again = again || (live && !(z0 + z1 == 0.f));
      }
    }
    if (ok && __any_sync(kFull, again)) prompt_again(a);
    tm_fence_before();
  }
  __syncthreads();
  if (warp == 8) {
    tm_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;\n" ::"r"(tmem) : "memory");
  }
}

// A warp per query row: join the partials.  Bound by latency: the first four
// parts are on their way, from places that are there whether they are used or
// not, before the row's number of parts and its sequence's length are known
// (512 queries over 32768 keys, 3 to 4 parts a row: 18.5 -> 11.0 us).
__global__ void __launch_bounds__(32 * kRowWarps) k_prompt_join(PromptArgs a, int nqb) {
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h = blockIdx.y, s = blockIdx.z, kvh = h / a.g;
  const int64_t tok = (int64_t)blockIdx.x * kRowWarps + warp;
  if (tok >= a.max_q) return;
  const int tq = kTile / a.g;
  const int64_t qb = tok / (kTiles * tq);
  const int in = (int)(tok - qb * kTiles * tq), row = in / tq * kTile + in % tq * a.g + h % a.g;
  const float* part = a.ws + ((((int64_t)s * a.hkv + kvh) * nqb + qb) * a.nsplit * (kTiles * kTile) + row) * kPartRow;
  const int64_t step = (int64_t)(kTiles * kTile) * kPartRow;
  constexpr int kAhead = 4;
  float2 ml[kAhead];
  float4 v[kAhead];
#pragma unroll
  for (int x = 0; x < kAhead; ++x)
    if (x < a.nsplit) {
      ml[x] = *reinterpret_cast<const float2*>(part + x * step);
      v[x] = *reinterpret_cast<const float4*>(part + x * step + 4 + 4 * lane);
    }
  const int parts = __float_as_int(part[2]);  // at most nsplit
  int64_t q0, lq, k0, lk;
  seq_rows(a.cu_q, s, a.rows_q, q0, lq);
  seq_rows(a.cu_k, s, a.rows_k, k0, lk);
  if (tok >= lq) return;
  float M = -INFINITY;
#pragma unroll
  for (int x = 0; x < kAhead; ++x)
    if (x < parts) M = fmaxf(M, ml[x].x);
  for (int x = kAhead; x < parts; ++x) M = fmaxf(M, part[x * step]);
  float L = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
  auto add = [&](const float2& ml, const float4& v) {
    if (ml.y == 0.f) return;  // no weight at all, and M may be -inf
    const float f = ml.x == M ? 1.f : exp2f(ml.x - M);
    L += ml.y * f;
    o[0] = fmaf(v.x, f, o[0]);
    o[1] = fmaf(v.y, f, o[1]);
    o[2] = fmaf(v.z, f, o[2]);
    o[3] = fmaf(v.w, f, o[3]);
  };
#pragma unroll
  for (int x = 0; x < kAhead; ++x)
    if (x < parts) add(ml[x], v[x]);
#pragma unroll 4
  for (int x = kAhead; x < parts; ++x)
    add(*reinterpret_cast<const float2*>(part + x * step), *reinterpret_cast<const float4*>(part + x * step + 4 + 4 * lane));
  const float inv = L != 0.f ? 1.f / L : 0.f;
  bool finite = true;
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    o[c] *= inv;
    finite = finite && fabsf(o[c]) < INFINITY;
  }
  finite = finite && !too_far(M);
  const int64_t visible = max64(0, min64(lk, tok + lk - lq + 1));
  if (!__all_sync(kFull, finite)) {
    prompt_row(a, s, h, q0, tok, k0, visible);
    return;
  }
  __nv_bfloat16* out = a.out + (a.cu_q ? 0 : s * a.so.seq) + (q0 + tok) * a.so.token + h * a.so.head;
  *reinterpret_cast<uint2*>(out + 4 * lane) = make_uint2(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]));
  if (a.lse != nullptr && lane == 0)
    a.lse[((int64_t)(a.cu_q ? 0 : s) * a.hq + h) * a.rows_q + q0 + tok] = visible > 0 ? (M + log2f(L)) * kLn2 : -INFINITY;
}

}  // namespace

namespace {

int64_t prompt_blocks(const PromptArgs& a) {  // blocks of query rows of the longest sequence
  const int64_t tokens = kTiles * (kTile / a.g);
  return (a.max_q + tokens - 1) / tokens;
}

// The kernel's shared-memory limit belongs to the device and is set once on
// each (a second thread doing the same is harmless).
cudaError_t raise_smem() {
  static std::atomic<bool> done[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || (dev >= 0 && dev < 64 && done[dev])) return e;
  e = cudaFuncSetAttribute((const void*)k_prompt_attend, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kPromptSmem);
  if (e == cudaSuccess && dev >= 0 && dev < 64) done[dev] = true;
  return e;
}

}  // namespace

size_t prompt_workspace_bytes(PromptArgs& a, int sm_count) {
  // Units that do not fill the GPU are shared among blocks, at least four key
  // blocks to each; a unit's keys then lie in up to nsplit blocks.
  const int64_t units = prompt_blocks(a) * a.n_seqs * a.hkv;
  const int64_t most = std::max<int64_t>(1, (a.max_k + 4 * kTile - 1) / (4 * kTile));
  const int64_t share = std::min<int64_t>({most, (sm_count + units - 1) / units, 63});
  a.nsplit = units < sm_count && share > 1 ? (int)share + 1 : 1;
  return a.nsplit > 1 ? (size_t)units * a.nsplit * kTiles * kTile * kPartRow * sizeof(float) : 0;
}

cudaError_t launch_prompt_attend(const PromptArgs& a, int sm_count, cudaStream_t st) {
  PromptMaps m;
  const int64_t ns = a.cu_q ? 1 : a.n_seqs;
  const int tq = kTile / a.g;
  // no keys at all: nothing is loaded, and any valid address will do
  const void* k = a.rows_k > 0 ? a.k : a.q;
  const void* v = a.rows_k > 0 ? a.v : a.q;
  const int64_t rows_k = std::max<int64_t>(1, a.rows_k);
  if (!encode(&m.q, a.q, a.hq, a.sq.head, a.rows_q, a.sq.token, ns, a.sq.seq, a.g, tq) ||
      !encode(&m.k, k, rows_k, a.sk.token, a.hkv, a.sk.head, ns, a.sk.seq, kTile, 1) ||
      !encode(&m.v, v, rows_k, a.sv.token, a.hkv, a.sv.head, ns, a.sv.seq, kTile, 1))
    return cudaErrorInvalidValue;
  cudaError_t e = raise_smem();
  if (e != cudaSuccess) return e;
  // a block per SM walks the items; no more blocks than there can be items
  const int64_t nqb = prompt_blocks(a), tokens = kTiles * (kTile / a.g);
  const int64_t pairs = a.cu_q ? std::min(nqb * a.n_seqs, a.rows_q / tokens + a.n_seqs) : nqb * a.n_seqs;
  const int64_t blocks = std::min<int64_t>(sm_count, pairs * a.hkv * std::max(1, a.nsplit - 1));
  e = launch_pdl(k_prompt_attend, dim3((unsigned)blocks), dim3(kPromptThreads), kPromptSmem, st, a, m);
  if (e != cudaSuccess || a.nsplit == 1) return e;
  const dim3 grid((unsigned)((a.max_q + kRowWarps - 1) / kRowWarps), a.hq, a.n_seqs);
  return launch_pdl(k_prompt_join, grid, dim3(32 * kRowWarps), 0, st, a, (int)nqb);
}

cudaError_t prompt_attend_error(uint32_t* bits) { return take_gave_up(bits); }

}  // namespace paris
