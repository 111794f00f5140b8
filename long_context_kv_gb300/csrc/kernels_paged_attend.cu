// Attention of one new token over a paged cache.
//
// Bound by the read of the rows in use: 512 bytes for each row and KV head
// in bf16, 258 in 8 bits.  What that asks for:
//
// - All SMs read to the end.  The tiles of all sequences form one line, which
//   the blocks of a KV head cut into equal parts; a part may end one sequence
//   and begin the next.  A sequence that several blocks share leaves partial
//   sums (maximum, sum, unnormalised result) in the workspace, and the block
//   that finishes last joins them, in the blocks' order.
// - Copies are always under way.  A warp takes steps of 8 KB of its own (16
//   bf16 rows of keys and values, or 32 in 8 bits) through a ring in shared
//   memory that TMA fills, two steps ahead and across the ends of sequences;
//   no warp waits for another but at those.  The tensor maps' swizzle makes
//   the reads below free of bank conflicts, and their strides take any order
//   of the pages' dimensions.
// - The arithmetic stays out of the way.  Both products have the cache's rows
//   on their M side, S^T = K Q^T and O^T = V^T P^T (m16n8k16, float32 sums), so
//   that the eight columns are what there are few of.  For up to four query
//   heads the columns hold each head twice, and P's upper and lower part; for
//   more, bf16 weights take a second product for their lower parts.  Values
//   of 8-bit rows are converted to halves, in which they are exact, and their
//   scales stay outside the products: a key row's multiplies its scores, a
//   value row's joins the exponent.
//
// Weights are p = 2^(s - m) of base-2 scores, m a maximum so far that may lag
// by 2^8.  With a value row's scale 2^e, what enters the product with V is
// 2^(s + e - m), m the maximum of s + e, and the sum takes 2^-e of it.  m is kept
// as a row's own product and e, and both are subtracted before the scale, so
// that weights are right at any size of the scores.
#include <cuda_fp16.h>

#include <algorithm>
#include <atomic>

#include "paged_internal.cuh"
#include "tc_device.cuh"

namespace paris {
namespace {

constexpr int kPgWarps = 4;
constexpr int kPgThreads = 32 * kPgWarps;
constexpr int kPgDepth = 3;
constexpr int kPgStage = 8192;  // bytes of a step: half keys, half values
constexpr int kPgScale = 64;    // a step's scale bytes: 32 of keys, 32 of values
constexpr int kPgOut = 8192;    // bytes through which the warps' results meet
constexpr float kPgGrowth = 8.f;
constexpr int kPgGroups = 32;   // counters of a (sequence, KV head)
constexpr int kPgSmem = 1024 + kPgWarps * kPgDepth * (kPgStage + kPgScale) + kPgOut;

template <bool kE4m3>
struct Pg {
  static constexpr int kRows = kE4m3 ? 32 : 16;  // rows of a warp's step
  static constexpr int kTile = kRows * kPgWarps;
  static constexpr int kU = kRows / 16;
};

// The rows of a sequence that count, from a multiple of a step's rows on.
struct PgSeq {
  int len, first, base;  // rows [first, len), tiles from base on
  uint32_t tiles;
};
template <bool kE4m3>
__device__ __forceinline__ PgSeq pg_seq(const PagedAttendArgs& a, int s) {
  PgSeq q;
  q.len = paged_len(a.c, s);
  q.first = a.window > 0 ? max(q.len - a.window, 0) : 0;
  q.base = q.first & ~(Pg<kE4m3>::kRows - 1);
  q.tiles = ((uint32_t)(q.len - q.base) + Pg<kE4m3>::kTile - 1) / Pg<kE4m3>::kTile;
  return q;
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
template <bool kE4m3>
__device__ __forceinline__ void mma16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (kE4m3)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(y) : "r"(x));
  return y;
}
// Two weights in the products' type, and what that leaves out.
template <bool kE4m3>
__device__ __forceinline__ uint32_t pack_weights(float a, float b, float& ra, float& rb) {
  if constexpr (kE4m3) {
    const __half2 h = __floats2half2_rn(a, b);
    const float2 f = __half22float2(h);
    ra = a - f.x;
    rb = b - f.y;
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const uint32_t h = pack_bf16x2(a, b);
    ra = a - bf16_bits_to_float(h & 0xffffu);
    rb = b - __uint_as_float(h & 0xffff0000u);
    return h;
  }
}
template <bool kE4m3>
__device__ __forceinline__ uint32_t pack_weights(float a, float b) {
  if constexpr (kE4m3) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    return pack_bf16x2(a, b);
  }
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n" ::"r"(dst), "l"(src),
               "r"(bytes), "r"(bar)
               : "memory");
}

// A maximum: a row's product d and exponent e, for scores d qs + e.
struct PgMax {
  float d, e;
};
// How far x lies above y.
__device__ __forceinline__ float above(PgMax x, PgMax y, float qs) { return fmaf(x.d - y.d, qs, x.e - y.e); }
// The larger one by k (its distance from some third one); the same on both sides of an exchange.
__device__ __forceinline__ void keep_larger(float& k, PgMax& m, float k2, PgMax m2) {
  if (k2 > k || (k2 == k && (m2.d > m.d || (m2.d == m.d && m2.e > m.e)))) {
    k = k2;
    m = m2;
  }
}

// Join the partial results of blocks [xf, xl] for nh query heads: a warp a
// head, its lanes over the partials' maxima and sums and then over the channels.
__device__ __forceinline__ void pg_join(const PagedAttendArgs& a, int b, int qh0, int nh, int xf, int xl, bool begins) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, n = xl - xf + 1;
  for (int h = warp; h < nh; h += kPgWarps) {
    const float* part = a.part + ((int64_t)(qh0 + h) * a.nblocks + xf) * 2 * kPartStride;
    // a block's first stretch lies in its first half; that of the block in which the sequence begins may not be it
    auto at = [&](int i) { return part + (2 * i + (i == 0 && !begins ? 1 : 0)) * kPartStride; };
    auto head = [&](int i) { return __ldcg(reinterpret_cast<const float4*>(at(i))); };
    PgMax m = {0.f, 0.f};
    float qs = 0.f, sum = 0.f;
#pragma unroll 1
    for (int round = 0; round < 2; ++round) {  // the second finds the largest by exact distances from about the largest
      float k = -INFINITY;
      PgMax best = {-INFINITY, -INFINITY};
      for (int i = lane; i < n; i += 32) {
        const float4 v = head(i);
        qs = v.w;
        if (v.z != 0.f) keep_larger(k, best, above({v.x, v.y}, m, v.w), {v.x, v.y});
      }
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const float k2 = __shfl_xor_sync(kFull, k, off);
        keep_larger(k, best, k2, {__shfl_xor_sync(kFull, best.d, off), __shfl_xor_sync(kFull, best.e, off)});
      }
      if (k > -INFINITY) m = best;
    }
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = 0; i0 < n; i0 += 32) {
      float f = 0.f;
      if (i0 + lane < n) {
        const float4 v = head(i0 + lane);
        if (v.z != 0.f) {  // the sum 0: no rows of weight
          f = ex2(above({v.x, v.y}, m, v.w));
          sum += v.z * f;
        }
      }
      const int most = min(32, n - i0);
#pragma unroll 8
      for (int i = 0; i < most; ++i) {
        const float fi = __shfl_sync(kFull, f, i);
        const float4 x = __ldcg(reinterpret_cast<const float4*>(at(i0 + i) + 4) + lane);
        o.x = fmaf(x.x, fi, o.x);
        o.y = fmaf(x.y, fi, o.y);
        o.z = fmaf(x.z, fi, o.z);
        o.w = fmaf(x.w, fi, o.w);
      }
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(kFull, sum, off);
    const float inv = sum != 0.f ? 1.f / sum : 0.f;
    const int64_t q = (int64_t)b * a.hq + qh0 + h;
    reinterpret_cast<uint2*>(a.out + q * kDim)[lane] = make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
    qs = __shfl_sync(kFull, qs, 0);
    if (a.lse != nullptr && lane == 0)
      a.lse[q] = sum != 0.f ? kLn2 * (fmaf(m.d, qs, m.e) + log2f(sum)) : -INFINITY;
  }
}

struct PgShared {
  uint64_t bar[kPgWarps][kPgDepth];
  float4 ml[kPgWarps][16];   // maximum (product, exponent), sum, scale of a head's scores
  float f[kPgWarps][16];     // a warp's share of the block's result
  float4 all[16];            // the block's maximum, sum and scale
  uint32_t tmp[33];
  uint32_t start_tile;
  int start_seq, last;
  uint32_t gave_up;
};

template <bool kE4m3, int kHeads>
__global__ void __launch_bounds__(kPgThreads, 2)
    k_paged_attend(PagedAttendArgs a, const __grid_constant__ CUtensorMap km, const __grid_constant__ CUtensorMap vm) {
  using G = Pg<kE4m3>;
  constexpr int kRows = G::kRows, kU = G::kU;
  constexpr int kQ = kHeads == 16 ? 2 : 1;                       // column tiles of queries
  constexpr int kParts = kHeads > 4 && !kE4m3 ? 2 : 1;           // products of weights with V for each of them
  constexpr float kUp = kE4m3 ? 7.f : 0.f, kDown = kE4m3 ? 1.f / 128.f : 1.f;  // halves have few exponents: weights are kept 2^7 up
  constexpr float kScoreScale = kScaleLog2;
  extern __shared__ uint8_t raw_mem[];
  __shared__ PgShared sh;
  const int tid = threadIdx.x, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int warp = __shfl_sync(kFull, tid >> 5, 0);
  const uint32_t ring = ((smem_u32(raw_mem) + 1023u) & ~1023u) + warp * kPgDepth * kPgStage;
  uint8_t* mem = raw_mem + ((1024u - (smem_u32(raw_mem) & 1023u)) & 1023u);
  const uint8_t* scales = mem + kPgWarps * kPgDepth * kPgStage + warp * kPgDepth * kPgScale;
  float* so = reinterpret_cast<float*>(mem + kPgWarps * kPgDepth * (kPgStage + kPgScale));
  const uint32_t bar0 = smem_u32(&sh.bar[warp][0]);
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < kPgDepth; ++i) bar_init(bar0 + 8 * i, 1);
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  if (tid == 0) sh.gave_up = 0;
  volatile uint32_t* gave_up = &sh.gave_up;
  const int kvh = blockIdx.y, h0 = blockIdx.z * kHeads, nh = min(kHeads, a.g - h0), qh0 = kvh * a.g + h0;
  const uint32_t x = blockIdx.x;
  pdl_wait();
  pdl_trigger();

  // sequences without rows: spread over the blocks
  for (int s = x; s < a.c.n_seqs; s += a.nblocks) {
    if (paged_len(a.c, s) > 0) continue;
    const int64_t q = (int64_t)s * a.hq + qh0;
    for (int i = tid; i < nh * (kDim / 8); i += kPgThreads) reinterpret_cast<uint4*>(a.out + q * kDim)[i] = make_uint4(0, 0, 0, 0);
    if (a.lse != nullptr && tid < nh) a.lse[q + tid] = -INFINITY;
  }

  // the block's part [lo, hi) of all tiles, and the sequence in which it begins
  uint32_t total, lo, hi, nb;
  {
    const int per = (a.c.n_seqs + kPgThreads - 1) / kPgThreads, s0 = tid * per, s1 = min(s0 + per, a.c.n_seqs);
    uint32_t mine = 0;
    for (int s = s0; s < s1; ++s) mine += pg_seq<kE4m3>(a, s).tiles;
    uint32_t before = block_excl_scan(mine, sh.tmp, &total);
    nb = min((uint32_t)a.nblocks, total);  // blocks with a part, of one tile at least
    if (x >= nb) return;
    lo = (uint32_t)((uint64_t)x * total / nb);
    hi = (uint32_t)((uint64_t)(x + 1) * total / nb);
    if (lo >= before && lo < before + mine) {
      for (int s = s0; s < s1; ++s) {
        const uint32_t n = pg_seq<kE4m3>(a, s).tiles;
        if (lo < before + n) {
          sh.start_seq = s;
          sh.start_tile = before;
          break;
        }
        before += n;
      }
    }
    __syncthreads();
  }

  // what the warp copies next: step `ahead.tile` of the line, in sequence ahead.s
  int c_s = sh.start_seq;
  PgSeq c_q = pg_seq<kE4m3>(a, c_s);
  uint32_t c_a = sh.start_tile;  // the sequence's first tile
  int p_s = c_s;
  PgSeq p_q = c_q;
  uint32_t p_a = c_a, p_tile = lo, issued = 0, taken = 0;
  uint32_t p_stage = 0, c_stage = 0, c_parity = 0;
  auto copy_next = [&]() {
    if (p_tile >= hi) return;
    while (p_tile >= p_a + p_q.tiles) {
      p_a += p_q.tiles;
      p_q = pg_seq<kE4m3>(a, ++p_s);
    }
    const int row = p_q.base + (int)(p_tile - p_a) * G::kTile + warp * kRows;
    ++p_tile;
    if (row >= p_q.len || __any_sync(kFull, *gave_up != 0)) return;
    const int j = row >> a.c.shift, r = row & ((1 << a.c.shift) - 1);
    const uint32_t dst = ring + p_stage * kPgStage, bar = bar0 + 8 * p_stage;
    if (elect()) {
      const int page = page_at(a.c, p_s, j);
      if constexpr (!kE4m3) {
        bar_expect(bar, kPgStage);
        tma_load(dst, &km, 0, r, kvh, page, bar);
        tma_load(dst + 2048, &km, 64, r, kvh, page, bar);
        tma_load(dst + 4096, &vm, 0, r, kvh, page, bar);
        tma_load(dst + 6144, &vm, 64, r, kvh, page, bar);
      } else {
        const uint32_t sc = smem_u32(scales) + p_stage * kPgScale;
        if (a.c.shift > 4) {
          bar_expect(bar, kPgStage + kPgScale);
          tma_load(dst, &km, 0, r, kvh, page, bar);
          tma_load(dst + 4096, &vm, 0, r, kvh, page, bar);
          const int64_t e = scale_at(a.c, a.layer, page, kvh, r);
          bulk_load(sc, a.c.ks + e, 32, bar);
          bulk_load(sc + 32, a.c.vs + e, 32, bar);
        } else {
          // two pages, the second one if it has rows
          const bool two = row + 16 < p_q.len;
          const int next = two ? page_at(a.c, p_s, j + 1) : 0;
          bar_expect(bar, (kPgStage + kPgScale) >> (two ? 0 : 1));
          tma_load(dst, &km, 0, 0, kvh, page, bar);
          tma_load(dst + 4096, &vm, 0, 0, kvh, page, bar);
          const int64_t e = scale_at(a.c, a.layer, page, kvh, 0);
          bulk_load(sc, a.c.ks + e, 16, bar);
          bulk_load(sc + 32, a.c.vs + e, 16, bar);
          if (two) {
            tma_load(dst + 2048, &km, 0, 0, kvh, next, bar);
            tma_load(dst + 6144, &vm, 0, 0, kvh, next, bar);
            const int64_t f = scale_at(a.c, a.layer, next, kvh, 0);
            bulk_load(sc + 16, a.c.ks + f, 16, bar);
            bulk_load(sc + 48, a.c.vs + f, 16, bar);
          }
        }
      }
    }
    __syncwarp();
    p_stage = p_stage + 1 == kPgDepth ? 0 : p_stage + 1;
    ++issued;
  };
#pragma unroll
  for (int i = 0; i < kPgDepth - 1; ++i) copy_next();

  // a lane's places in a step's boxes (128 bytes a row, 16-byte pieces swizzled by the row)
  const uint32_t lrow = lane & 15, lhi = lane >> 4, lsw = lane & 7;

  uint32_t tile = lo;
  while (tile < hi) {
    while (tile >= c_a + c_q.tiles) {
      c_a += c_q.tiles;
      c_q = pg_seq<kE4m3>(a, ++c_s);
    }
    const uint32_t end = min(hi, c_a + c_q.tiles);

    // the queries: column g's head (of four: twice)
    uint32_t qf[kQ][8][2];
    float qs[kQ][2];  // of a thread's columns 2 t and 2 t + 1
#pragma unroll
    for (int c = 0; c < kQ; ++c) {
      const int h = 8 * c + (kHeads == 4 ? g & 3 : g);
      const uint32_t* q = reinterpret_cast<const uint32_t*>(a.q + ((int64_t)c_s * a.hq + qh0 + h) * kDim);
      uint32_t w[8][2];
#pragma unroll
      for (int s = 0; s < 8; ++s) {
        if constexpr (!kE4m3) {
          w[s][0] = h < nh ? __ldg(q + 8 * s + t) : 0u;
          w[s][1] = h < nh ? __ldg(q + 8 * s + 4 + t) : 0u;
        } else {
          const uint2 u = h < nh ? __ldg(reinterpret_cast<const uint2*>(q + 8 * s) + t) : make_uint2(0, 0);
          w[s][0] = u.x;
          w[s][1] = u.y;
        }
      }
      if constexpr (!kE4m3) {
#pragma unroll
        for (int s = 0; s < 8; ++s) {
          qf[c][s][0] = w[s][0];
          qf[c][s][1] = w[s][1];
        }
        qs[c][0] = qs[c][1] = kScoreScale;
      } else {
        // as halves, scaled by a power of two to below 1; eight bits fit their eleven
        float amax = 0.f;
#pragma unroll
        for (int s = 0; s < 8; ++s)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            amax = fmaxf(amax, fmaxf(fabsf(bf16_bits_to_float(w[s][i] & 0xffffu)), fabsf(__uint_as_float(w[s][i] & 0xffff0000u))));
        amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 2));
        const int e = min(max((int)((__float_as_uint(amax) >> 23) & 255u) - 126, -100), 126);
        const float down = __uint_as_float((uint32_t)(127 - e) << 23), up = __uint_as_float((uint32_t)(127 + e) << 23) * kScoreScale;
#pragma unroll
        for (int s = 0; s < 8; ++s)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            qf[c][s][i] = pack_weights<true>(bf16_bits_to_float(w[s][i] & 0xffffu) * down, __uint_as_float(w[s][i] & 0xffff0000u) * down);
        qs[c][0] = __shfl_sync(kFull, up, 8 * t);
        qs[c][1] = __shfl_sync(kFull, up, 8 * t + 4);
      }
    }

    float o[8][kQ][4];
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int c = 0; c < kQ; ++c) o[j][c][0] = o[j][c][1] = o[j][c][2] = o[j][c][3] = 0.f;
    PgMax m[kQ][2];
    float l[kQ][2];
    bool live[kQ][2];  // a row of weight has set the maximum
#pragma unroll
    for (int c = 0; c < kQ; ++c)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        m[c][i] = {0.f, 0.f};
        l[c][i] = 0.f;
        live[c][i] = false;
      }

#pragma unroll 1
    for (; tile < end; ++tile) {
      copy_next();
      const int row0 = c_q.base + (int)(tile - c_a) * G::kTile + warp * kRows;
      if (row0 >= c_q.len || taken == issued) continue;  // (nothing is copied any more after a wait that gave up)
      const uint32_t kst = ring + c_stage * kPgStage, vst = kst + kPgStage / 2;
      if (!bar_wait(bar0 + 8 * c_stage, c_parity, gave_up)) {
        WaitLimit limit(now_ns());  // the copy ends before the block does
        while (!bar_try(bar0 + 8 * c_stage, c_parity) && !limit.over(now_ns())) {}
      }
      ++taken;
      const bool edge = row0 < c_q.first || row0 + kRows > c_q.len;
      if (edge) {
        // rows that do not count may hold anything, and 0 times NaN is NaN
        for (int r = lane >> 3; r < kRows; r += 4) {
          if (row0 + r >= c_q.first && row0 + r < c_q.len) continue;
          const uint32_t z = vst + r * 128 + 16 * (lane & 7);
          asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};\n" ::"r"(z), "r"(0) : "memory");
          if (!kE4m3) asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};\n" ::"r"(z + 2048), "r"(0) : "memory");
        }
        asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");  // before the next copy into the step's place
        __syncwarp();
      }

      // S^T: p[u][c][2 r + i] of row 16 u + 8 r + g, column 2 t + i
      float p[kU][kQ][4], ev[kU][2], inv[kU][2];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
#pragma unroll
        for (int c = 0; c < kQ; ++c) p[u][c][0] = p[u][c][1] = p[u][c][2] = p[u][c][3] = 0.f;
        if constexpr (!kE4m3) {
#pragma unroll
          for (int s = 0; s < 8; ++s) {
            uint32_t f[4];
            ldsm4(f, kst + (s >> 2) * 2048 + lrow * 128 + (((2 * (s & 3) + lhi) ^ lsw) << 4));
#pragma unroll
            for (int c = 0; c < kQ; ++c) mma16<false>(p[u][c], f[0], f[1], f[2], f[3], qf[c][s][0], qf[c][s][1]);
          }
        } else {
#pragma unroll
          for (int s = 0; s < 4; ++s) {
            // four neighbouring channels of a row: two at places 2 t of the product's inner axis, two at 2 t + 8
            uint32_t f[4];
            ldsm4(f, kst + (16 * u + lrow) * 128 + (((2 * s + lhi) ^ lsw) << 4));
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const uint32_t a0 = e4m3_to_f16x2(f[2 * i]), a1 = e4m3_to_f16x2(f[2 * i + 1]);
              const uint32_t a2 = e4m3_to_f16x2(f[2 * i] >> 16), a3 = e4m3_to_f16x2(f[2 * i + 1] >> 16);
#pragma unroll
              for (int c = 0; c < kQ; ++c) mma16<true>(p[u][c], a0, a1, a2, a3, qf[c][2 * s + i][0], qf[c][2 * s + i][1]);
            }
          }
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const uint8_t* sc = scales + c_stage * kPgScale + 16 * u + 8 * r + g;
            const int kb = sc[0], vb = sc[32];
            const float S = __uint_as_float((uint32_t)kb << 23);
            ev[u][r] = (float)(vb - 127);
            inv[u][r] = __uint_as_float((uint32_t)(254 - vb) << 23);
#pragma unroll
            for (int c = 0; c < kQ; ++c) {
              p[u][c][2 * r] *= S;
              p[u][c][2 * r + 1] *= S;
            }
          }
        }
      }
      if (edge) {
#pragma unroll
        for (int u = 0; u < kU; ++u)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const int row = row0 + 16 * u + 8 * r + g;
            if (row >= c_q.first && row < c_q.len) continue;
            ev[u][r] = 0.f;
            inv[u][r] = 1.f;
#pragma unroll
            for (int c = 0; c < kQ; ++c) p[u][c][2 * r] = p[u][c][2 * r + 1] = -INFINITY;
          }
      }
      auto score = [&](int u, int c, int r, int i) {
        const float d = p[u][c][2 * r + i] - m[c][i].d;
        return kE4m3 ? fmaf(d, qs[c][i], ev[u][r] - m[c][i].e) : d * qs[c][i];
      };
      bool grows = false;
#pragma unroll
      for (int u = 0; u < kU; ++u)
#pragma unroll
        for (int c = 0; c < kQ; ++c)
#pragma unroll
          for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int i = 0; i < 2; ++i)
              grows |= score(u, c, r, i) > kPgGrowth || (!live[c][i] && p[u][c][2 * r + i] > -INFINITY);
      // A maximum that is found by distances from far away may be off by their
      // rounding; the next look is from nearby.
#pragma unroll 1
      for (int look = 0; look < 3 && __any_sync(kFull, grows); ++look) {
        grows = false;
#pragma unroll
        for (int c = 0; c < kQ; ++c)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float k = -INFINITY;
            PgMax best = {-INFINITY, -INFINITY};
#pragma unroll
            for (int u = 0; u < kU; ++u)
#pragma unroll
              for (int r = 0; r < 2; ++r) {
                const PgMax v = {p[u][c][2 * r + i], kE4m3 ? ev[u][r] : 0.f};
                keep_larger(k, best, kE4m3 ? score(u, c, r, i) : v.d, v);
              }
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) {
              const float k2 = __shfl_xor_sync(kFull, k, off);
              keep_larger(k, best, k2, {__shfl_xor_sync(kFull, best.d, off), __shfl_xor_sync(kFull, best.e, off)});
            }
            const float up = above(best, m[c][i], qs[c][i]);
            if (best.d > -INFINITY && (!live[c][i] || up > 0.f)) {
              const float f = live[c][i] ? ex2(-up) : 0.f;
              l[c][i] *= f;
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                o[j][c][i] *= f;
                o[j][c][i + 2] *= f;
              }
              m[c][i] = best;
              live[c][i] = true;
            }
#pragma unroll
            for (int u = 0; u < kU; ++u)
#pragma unroll
              for (int r = 0; r < 2; ++r) grows |= score(u, c, r, i) > kPgGrowth;
          }
      }

      // P^T as the second operand: rows 16 u + 8 r, a column tile's upper and lower parts
      uint32_t pb[kU][kQ][kParts][2];
#pragma unroll
      for (int u = 0; u < kU; ++u)
#pragma unroll
        for (int c = 0; c < kQ; ++c)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float w0 = ex2(score(u, c, r, 0) + kUp), w1 = ex2(score(u, c, r, 1) + kUp);
            l[c][0] = kE4m3 ? fmaf(w0, inv[u][r], l[c][0]) : l[c][0] + w0;
            l[c][1] = kE4m3 ? fmaf(w1, inv[u][r], l[c][1]) : l[c][1] + w1;
            if constexpr (kHeads == 4) {
              float r0, r1;
              const uint32_t up = pack_weights<kE4m3>(w0, w1, r0, r1), low = pack_weights<kE4m3>(r0, r1);
              pb[u][c][0][r] = transpose8x8(t < 2 ? up : low);
            } else if constexpr (kParts == 2) {
              float r0, r1;
              pb[u][c][0][r] = transpose8x8(pack_weights<kE4m3>(w0, w1, r0, r1));
              pb[u][c][kParts - 1][r] = transpose8x8(pack_weights<kE4m3>(r0, r1));
            } else {
              pb[u][c][0][r] = transpose8x8(pack_weights<kE4m3>(w0, w1));
            }
          }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if constexpr (!kE4m3) {
          uint32_t f[4];
          // rows 0-7 and 8-15 by channels 16 j and 16 j + 8
          const uint32_t vrow = (lane & 7) + ((lane >> 4) << 3), vhi = (lane >> 3) & 1;
          ldsm4_t(f, vst + (j >> 2) * 2048 + vrow * 128 + (((2 * (j & 3) + vhi) ^ lsw) << 4));
#pragma unroll
          for (int c = 0; c < kQ; ++c)
#pragma unroll
            for (int s = 0; s < kParts; ++s) mma16<false>(o[j][c], f[0], f[1], f[2], f[3], pb[0][c][s][0], pb[0][c][s][1]);
        } else {
          uint32_t f[4];
          ldsm4_t(f, vst + lane * 128 + ((j ^ lsw) << 4));
#pragma unroll
          for (int u = 0; u < kU; ++u) {
            // two rows by two channels a word: even channels are the product's first eight rows, odd ones the others
            const uint32_t w0 = __byte_perm(f[2 * u], 0, 0x3120), w1 = __byte_perm(f[2 * u + 1], 0, 0x3120);
            const uint32_t a0 = e4m3_to_f16x2(w0), a1 = e4m3_to_f16x2(w0 >> 16), a2 = e4m3_to_f16x2(w1), a3 = e4m3_to_f16x2(w1 >> 16);
#pragma unroll
            for (int c = 0; c < kQ; ++c) mma16<true>(o[j][c], a0, a1, a2, a3, pb[u][c][0][0], pb[u][c][0][1]);
          }
        }
      }
      __syncwarp();  // the step's place may be filled again
      if (++c_stage == kPgDepth) {
        c_stage = 0;
        c_parity ^= 1;
      }
    }

    // the warps' sums
#pragma unroll
    for (int c = 0; c < kQ; ++c)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) l[c][i] += __shfl_xor_sync(kFull, l[c][i], off);
        if (g == 0 && (kHeads > 4 || t < 2)) sh.ml[warp][8 * c + 2 * t + i] = make_float4(m[c][i].d, m[c][i].e, l[c][i] * kDown, qs[c][i]);
      }
    __syncthreads();
    if (tid < kHeads) {
      PgMax best = {0.f, 0.f};
      const float scale = sh.ml[0][tid].w;
      bool any = false;
#pragma unroll
      for (int w = 0; w < kPgWarps; ++w) {
        const float4 v = sh.ml[w][tid];
        if (v.z != 0.f && (!any || above({v.x, v.y}, best, scale) > 0.f)) {
          best = {v.x, v.y};
          any = true;
        }
      }
      float sum = 0.f;
#pragma unroll
      for (int w = 0; w < kPgWarps; ++w) {
        const float4 v = sh.ml[w][tid];
        const float f = v.z != 0.f ? ex2(above({v.x, v.y}, best, scale)) : 0.f;
        sh.f[w][tid] = f * kDown;
        sum += v.z != 0.f ? v.z * f : 0.f;
      }
      sh.all[tid] = make_float4(best.d, best.e, sum, scale);
    }
    // the blocks that share the sequence
    const int xf = (int)(((uint64_t)(c_a + 1) * nb - 1) / total), xl = (int)(((uint64_t)(c_a + c_q.tiles) * nb - 1) / total);
    const bool begins = (uint32_t)((uint64_t)xf * total / nb) == c_a;  // with its first block
    const int half = (int)x == xf && !begins ? 1 : 0;
    // their results, kCh channels at a time: [warp][head][channel]
    constexpr int kCh = kPgOut / 4 / kPgWarps / kHeads, kTiles = kCh / 16;
#pragma unroll
    for (int pass = 0; pass < kDim / kCh; ++pass) {
      __syncthreads();
#pragma unroll
      for (int jj = 0; jj < kTiles; ++jj) {
        const int j = pass * kTiles + jj;
#pragma unroll
        for (int c = 0; c < kQ; ++c)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float v = o[j][c][i];
            if constexpr (kHeads == 4) v += __shfl_xor_sync(kFull, v, 2);
            const int ch = 16 * jj + (kE4m3 ? 2 * g + (i >> 1) : g + 8 * (i >> 1)), h = 8 * c + 2 * t + (i & 1);
            if (kHeads > 4 || t < 2) so[(warp * kHeads + h) * kCh + ch] = v;
          }
      }
      __syncthreads();
      const int h = tid * 4 / kCh, ch = tid * 4 % kCh;
      if (h < nh) {
        float4 r = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kPgWarps; ++w) {
          const float f = sh.f[w][h];
          const float4 v = *reinterpret_cast<const float4*>(so + (w * kHeads + h) * kCh + ch);
          if (f == 0.f) continue;  // no rows of weight
          r.x = fmaf(v.x, f, r.x);
          r.y = fmaf(v.y, f, r.y);
          r.z = fmaf(v.z, f, r.z);
          r.w = fmaf(v.w, f, r.w);
        }
        const float4 all = sh.all[h];
        const int channel = pass * kCh + ch;
        if (xf == xl) {
          const float inv = all.z != 0.f ? 1.f / all.z : 0.f;
          const int64_t q = (int64_t)c_s * a.hq + qh0 + h;
          *reinterpret_cast<uint2*>(a.out + q * kDim + channel) =
              make_uint2(pack_bf16x2(r.x * inv, r.y * inv), pack_bf16x2(r.z * inv, r.w * inv));
          if (a.lse != nullptr && channel == 0)
            a.lse[q] = all.z != 0.f ? kLn2 * (fmaf(all.x, all.w, all.y) + log2f(all.z)) : -INFINITY;
        } else {
          float* part = a.part + (((int64_t)(qh0 + h) * a.nblocks + x) * 2 + half) * kPartStride;
          *reinterpret_cast<float4*>(part + 4 + channel) = r;
          if (channel == 0) *reinterpret_cast<float4*>(part) = all;
        }
      }
    }
    if (xf != xl) {
      __syncthreads();
      if (tid == 0) {
        __threadfence();
        const uint32_t n = (uint32_t)(xl - xf);
        uint32_t* counter = a.counters + ((int64_t)c_s * a.c.hkv + kvh) * kPgGroups + blockIdx.z;
        sh.last = atomicInc(counter, n) == n;
        __threadfence();
      }
      __syncthreads();
      if (sh.last) pg_join(a, c_s, qh0, nh, xf, xl, begins);
    }
    __syncthreads();  // what the sums went through may be used again
  }
}

// box rows x 128 channels of one head and page (bf16: 64 channels, 128 bytes).
bool encode_pages(CUtensorMap* m, const Paged& c, const uint8_t* base, const PageStrides& s, int layer) {
  EncodeTiled fn = encode_tiled();
  if (fn == nullptr) return false;
  const int rows = 1 << c.shift;
  const cuuint64_t dims[4] = {(cuuint64_t)kDim, (cuuint64_t)rows, (cuuint64_t)c.hkv, (cuuint64_t)c.n_pages};
  const cuuint64_t strides[3] = {(cuuint64_t)s.row, (cuuint64_t)s.head, (cuuint64_t)s.page};
  const cuuint32_t box[4] = {c.e4m3 ? 128u : 64u, (cuuint32_t)(c.e4m3 ? std::min(rows, 32) : 16), 1, 1}, one[4] = {1, 1, 1, 1};
  return fn(m, c.e4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
            const_cast<uint8_t*>(base + layer * s.layer), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int heads_of(int g) { return g <= 4 ? 4 : g <= 8 ? 8 : 16; }

template <bool kE4m3, int kHeads>
cudaError_t launch_heads(const PagedAttendArgs& a, const CUtensorMap& km, const CUtensorMap& vm, cudaStream_t st) {
  static std::atomic<bool> done[64];  // the limit belongs to the device; setting it twice is harmless
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess && !(dev >= 0 && dev < 64 && done[dev])) {
    e = cudaFuncSetAttribute((const void*)k_paged_attend<kE4m3, kHeads>, cudaFuncAttributeMaxDynamicSharedMemorySize, kPgSmem);
    if (e == cudaSuccess && dev >= 0 && dev < 64) done[dev] = true;
  }
  if (e != cudaSuccess) return e;
  const dim3 grid(a.nblocks, a.c.hkv, (a.g + kHeads - 1) / kHeads);
  return launch_pdl(k_paged_attend<kE4m3, kHeads>, grid, dim3(kPgThreads), kPgSmem, st, a, km, vm);
}

}  // namespace

// Blocks of a KV head and head group: a wave of two an SM, and no more than
// there could be tiles.
int paged_attend_blocks(const Paged& c, int g, int sm_count) {
  const int groups = (g + heads_of(g) - 1) / heads_of(g), tile = c.e4m3 ? Pg<true>::kTile : Pg<false>::kTile;
  const int64_t wave = std::max<int64_t>(1, 2 * (int64_t)sm_count / ((int64_t)c.hkv * groups));
  const int64_t rows = (int64_t)c.width << c.shift;
  return (int)std::min(wave, c.n_seqs * ((rows + tile - 1) / tile + (rows > tile ? 1 : 0)));
}

size_t paged_attend_part_bytes(const Paged&, int hq, int nblocks) {
  return (size_t)hq * nblocks * 2 * kPartStride * sizeof(float);
}

cudaError_t paged_attend_error(uint32_t* bits) { return take_gave_up(bits); }

cudaError_t launch_paged_attend(const PagedAttendArgs& a, cudaStream_t st) {
  CUtensorMap km, vm;
  if (!encode_pages(&km, a.c, a.c.k, a.c.sk, a.layer) || !encode_pages(&vm, a.c, a.c.v, a.c.sv, a.layer)) return cudaErrorInvalidValue;
  const int heads = heads_of(a.g);
  if (a.c.e4m3)
    return heads == 4 ? launch_heads<true, 4>(a, km, vm, st) : heads == 8 ? launch_heads<true, 8>(a, km, vm, st) : launch_heads<true, 16>(a, km, vm, st);
  return heads == 4 ? launch_heads<false, 4>(a, km, vm, st) : heads == 8 ? launch_heads<false, 8>(a, km, vm, st) : launch_heads<false, 16>(a, km, vm, st);
}

}  // namespace paris
