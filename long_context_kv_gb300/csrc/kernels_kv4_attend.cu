// Decode attention over the 4-bit cache, and the accumulation of its weights.
//
// Bound by the read of the rows: 136 bytes per row and KV head (codes and
// scales of a key and a value) against 512 in bf16.  What has to stay out of
// the way is the unpacking, 256 values a row, so no value is converted
// twice and none goes through shared memory:
//
// - The products are m16n8k16 half-precision mma with float32 accumulation.
//   Which channel a fragment slot stands for is free as long as both
//   operands agree, so a thread's fragments are built from the 16 (keys) or
//   8 (values) contiguous code bytes that it loads itself.
// - A code word becomes pairs of halves with half a shift, one logic
//   operation and one fma a pair: a nibble or-ed into the mantissa of 64
//   gives 64 + u / 16 (bits 0-3) or 64 + u (bits 4-7), and the fma with S and
//   -64.5 S or -72 S gives S (u - 8) / 16 or S (u - 8).  S has four
//   significant bits, so 129 S and 9 S fit a half's eleven and every term is
//   exact; the 1/16 of the even channels is made good in the queries and in
//   the result.
// - Both products have the cache's rows on their M side, S^T = K Q^T and
//   O^T = V^T P^T, so that the eight columns are what there are few of: for up
//   to four query heads their upper and lower half-precision parts (22 bits
//   of a query or weight for the cost of 11), for up to eight two products.
//   (A bf16 query's eight bits fit the upper part and its lower one is 0; the
//   products are the same for both types.)
//   The weights go from the one's result to the other's operand by 8x8
//   transposes in registers.
//
// A warp walks its rows 32 at a time with a running maximum and sum per
// head, its next steps' rows on the way to its own ring in shared memory; no
// warp waits for another until the end.  Partials of (chunk, head) are merged
// by k_kv4_finish, which also turns the scores into weights.  More than eight
// query heads per KV head are two blocks, each reading the rows.
//
// At 131072 rows of 8 KV heads, 4 query heads each (142.6 MB): 35.6 us with the
// merge.  The copies alone in this form, with nothing computed, take 30.6: 23.5
// at 6 TB/s and 7 for the start, the first rows' way and the end.  Fewer instructions no
// longer tell (HFMA2 halved by keys as subnormals: the same), nor do more or
// fewer warps (12, 16, 20 an SM: within 2 us).
#include <atomic>
#include <float.h>

#include <cuda_fp16.h>

#include <algorithm>

#include "kv4_internal.cuh"

namespace paris {
namespace {

constexpr int kWarps4 = 4;
constexpr int kThreads4 = 32 * kWarps4;
constexpr int kRows4 = 32;                     // rows per warp and step
constexpr int kTile4 = kRows4 * kWarps4;       // rows per block and step
constexpr int kHeads4 = 8;                     // query heads per block
// Steps of a warp's ring.  Two are enough to keep the rows coming (16 warps an
// SM, 4.4 KB each on the way) and leave shared memory for the blocks of the
// kernel that follows: 37.6 us at 131072 rows, 39.5 with three.
constexpr int kDepth4 = 2;
constexpr float kGrowth4 = 8.f;                // how far a running maximum may lag, base 2
constexpr float kUp4 = 7.f, kDown4 = 1.f / 128.f;  // weights are kept 2^7 up

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
               "{%0,%1,%2,%3};\n"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t h2u(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }
__device__ __forceinline__ __half2 u2h(uint32_t u) { return *reinterpret_cast<__half2*>(&u); }

// The two lower nibbles of each half of x as pairs of halves, times their
// scales: v0 = S (first - 8) / 16, v1 = S (second - 8).  magic: 64 in each
// half.  It comes as a kernel argument because as a constant it is or-ed in
// by an instruction of its own (an instruction holds one immediate, the
// mask): twice the logic, 259 against 131 of them for 32 rows.
constexpr uint32_t kMagic4 = 0x54005400u;
__device__ __forceinline__ void unpack2(uint32_t x, uint32_t magic, __half2 S, __half2 even, __half2 odd, uint32_t& v0, uint32_t& v1) {
  uint32_t y0, y1;
  asm("lop3.b32 %0, %1, 0x000F000F, %2, 0xEA;\n" : "=r"(y0) : "r"(x), "r"(magic));
  asm("lop3.b32 %0, %1, 0x00F000F0, %2, 0xEA;\n" : "=r"(y1) : "r"(x), "r"(magic));
  v0 = h2u(__hfma2(u2h(y0), S, even));
  v1 = h2u(__hfma2(u2h(y1), S, odd));
}

// A warp's ring: kDepth4 steps of 32 rows as they are in memory.
struct Step4 {
  uint4 k[kRows4 * kCode4 / 16], v[kRows4 * kCode4 / 16];
  uint32_t ks[kRows4], vs[kRows4];
};

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;\n" ::"r"(dst), "l"(src) : "memory");
}

// What a lane copies of the warp's next step: a code piece (and those 512, 1024
// and 1536 bytes on) and a row's scales, of keys and values.
struct Next4 {
  const uint8_t *k, *v, *ks, *vs;
};

// Start the copy of a step of which `left` rows are there; past them the last
// one again (its weights are set to zero).
__device__ __forceinline__ void copy_step(uint32_t dst, Next4& p, int left, int lane) {
  if (left >= kRows4) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      copy16(dst + 16 * lane + 512 * i, p.k + 512 * i);
      copy16(dst + 2048 + 16 * lane + 512 * i, p.v + 512 * i);
    }
    copy4(dst + 4096 + 4 * lane, p.ks);
    copy4(dst + 4224 + 4 * lane, p.vs);
  } else {
#pragma unroll 1
    for (int i = 0; i < 4; ++i) {
      const int row = 8 * i + (lane >> 2), back = max(row - left + 1, 0) * kCode4 - 512 * i;
      copy16(dst + 16 * lane + 512 * i, p.k - back);
      copy16(dst + 2048 + 16 * lane + 512 * i, p.v - back);
    }
    const int back = max(lane - left + 1, 0) * kScale4;
    copy4(dst + 4096 + 4 * lane, p.ks - back);
    copy4(dst + 4224 + 4 * lane, p.vs - back);
  }
  p.k += kTile4 * kCode4;
  p.v += kTile4 * kCode4;
  p.ks += kTile4 * kScale4;
  p.vs += kTile4 * kScale4;
}

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(y) : "r"(x));
  return y;
}

// The rows of a batch are cut into chunks, a block each (per KV head and head
// group), a sequence's into equal ones.  Their size comes from the lengths as
// they are on the device, so that nblocks chunks hold every row however the
// lengths differ.  Batches of more than 128 sequences (four a lane) fill the
// GPU anyway, and are cut evenly.
constexpr int kCutSeqs = 128;

// The block's sequence (-1: none), the first of its chunks and their number.
__device__ __forceinline__ int3 chunk_of(const Attend4Args& a, int x) {
  if (a.c.batch > kCutSeqs) {
    const int n = a.nblocks / a.c.batch;
    return make_int3(x / n, x / n * n, n);
  }
  // tiles fit 31 bits: 128 x 2^31 / 128
  if (a.c.batch == 1) {
    const uint32_t all = ((uint32_t)kv4_len(a.c, 0) + kTile4 - 1) / kTile4;
    const uint32_t size = max(1u, (all + a.nblocks - 1) / a.nblocks), n = (all + size - 1) / size;
    return make_int3((uint32_t)x < n ? 0 : -1, 0, n);
  }
  const int lane = threadIdx.x & 31;
  uint32_t tiles[kCutSeqs / 32];
#pragma unroll
  for (int i = 0; i < kCutSeqs / 32; ++i)
    tiles[i] = 32 * i + lane < a.c.batch ? ((uint32_t)kv4_len(a.c, 32 * i + lane) + kTile4 - 1) / kTile4 : 0u;
  return cut_tiles(tiles, a.nblocks, x);
}

struct Shared4 {
  uint2 q[8][2][32];           // query fragments: step, column tile, lane
  float qscale[kHeads4];
  float ml[kWarps4][kHeads4][2];
};

// NT column tiles: 1 for up to four query heads (columns 0-3 their upper,
// 4-7 their lower parts), 2 for up to eight (a tile of each).
template <int NT>
__global__ void __launch_bounds__(kThreads4, NT == 1 ? 4 : 3) k_kv4_attend(Attend4Args a, uint32_t magic) {
  extern __shared__ __align__(16) uint8_t ring_mem[];
  __shared__ Shared4 sh;
  constexpr int kHeads = 4 * NT;
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int warp = __shfl_sync(kFull, tid >> 5, 0);
  const int kvh = blockIdx.y, h0 = blockIdx.z * kHeads;
  int3 chunk = chunk_of(a, blockIdx.x);
  // the same in every lane: a reduction tells the compiler, and the addresses
  // stay in uniform registers (36.4 against 33.4 us at 128K rows)
  chunk = make_int3(__reduce_max_sync(kFull, chunk.x), __reduce_max_sync(kFull, chunk.y), __reduce_max_sync(kFull, chunk.z));
  const int b = chunk.x;
  if (b < 0) return;
  const int split = (int)blockIdx.x - chunk.y, bh = b * a.c.hkv + kvh;
  // for the merging kernel; a sequence without rows has no chunk, or empty ones
  if (split == 0 && kvh == 0 && blockIdx.z == 0 && tid == 0) a.chunks[b] = make_int2(chunk.y, chunk.z);
  const int nh = min(kHeads, a.g - h0);
  const int qh0 = kvh * a.g + h0;  // first query head of the block
  const int64_t len = kv4_len(a.c, b);
  const uint32_t chunk_rows = (((uint32_t)len + kTile4 - 1) / kTile4 + chunk.z - 1) / chunk.z * kTile4;
  const int64_t r_begin = (int64_t)split * chunk_rows;
  float* part = a.part + ((int64_t)qh0 * a.nblocks + blockIdx.x) * kPartStride;
  if (r_begin >= len) {
    if (tid < nh) {
      part[(int64_t)tid * a.nblocks * kPartStride] = -INFINITY;
      part[(int64_t)tid * a.nblocks * kPartStride + 1] = 0.f;
    }
    return;
  }
  // rows of this split from its first on, and of the sequence
  const int n = __reduce_max_sync(kFull, (int)min64(len - r_begin, chunk_rows));
  const int64_t base = (int64_t)bh * a.c.rmax + r_begin;
  const Step4* ring = reinterpret_cast<const Step4*>(ring_mem) + warp * kDepth4;
  const uint32_t ring_u32 = static_cast<uint32_t>(__cvta_generic_to_shared(ring));
  int row0 = warp * kRows4;
  Next4 ahead{a.c.kc + (base + row0) * kCode4 + 16 * lane, a.c.vc + (base + row0) * kCode4 + 16 * lane,
              a.c.ks + (base + row0 + lane) * kScale4, a.c.vs + (base + row0 + lane) * kScale4};
  auto start_copy = [&](int i) {
    if (row0 + i * kTile4 < n) copy_step(ring_u32 + i * (int)sizeof(Step4), ahead, n - row0 - i * kTile4, lane);
    asm volatile("cp.async.commit_group;\n" ::: "memory");
  };

  // The query of column g's head as two half parts, scaled by a power of two
  // to at most 1 (its scores are scaled back, with log2(e) / sqrt(d)); each
  // warp makes two of the eight steps' fragments.  Its loads go out first,
  // then the first step's; the further ones, which the memory takes a while to
  // deliver to all blocks at once, do not hold up the query's.
  {
    const int h = NT == 1 ? g & 3 : g;
    const int64_t qe = ((int64_t)b * a.hq + qh0 + h) * kDim + 32 * t;
    uint4 raw[8];
    if (a.dtype == 1) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        raw[i] = h < nh ? __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) + qe) + i) : make_uint4(0, 0, 0, 0);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        raw[i] = h < nh ? __ldg(reinterpret_cast<const uint4*>(static_cast<const float*>(a.q) + qe) + i) : make_uint4(0, 0, 0, 0);
    }
    start_copy(0);
    float x[8], amax = 0.f;
    if (a.dtype == 1) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float lo = bf16_bits_to_float(w[j] & 0xffffu), hi = __uint_as_float(w[j] & 0xffff0000u);
          amax = fmaxf(amax, fmaxf(fabsf(lo), fabsf(hi)));
          if (i == warp) {
            x[2 * j] = lo;
            x[2 * j + 1] = hi;
          }
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          amax = fmaxf(amax, fabsf(__uint_as_float(w[j])));
          if (i >> 1 == warp) x[4 * (i & 1) + j] = __uint_as_float(w[j]);
        }
      }
    }
    amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 2));
    // 2^e > amax for every finite query but those of 2^126 and more, which come
    // out below 4 (64 in even channels); queries below 2^-101 are scaled by
    // less than their size asks for, and their scores are nothing in float32
    // all the same
    const int e = min(max((int)((__float_as_uint(amax) >> 23) & 255u) - 126, -100), 126);
    const float down = __uint_as_float((uint32_t)(127 - e) << 23);
    if (warp == 0 && t == 0) sh.qscale[h] = __uint_as_float((uint32_t)(127 + e) << 23) * (1.4426950408889634f * 0.08838834764831845f);
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      uint32_t hi[2], lo[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        // fragment slots of step 2 warp + s: channels c and c + 4 of the
        // warp's eight, c = 2 s + j; even channels' rows come over 16
        const float up = j == 0 ? 16.f * down : down;
        const float y0 = x[2 * s + j] * up, y1 = x[2 * s + j + 4] * up;
        const __half2 u = __floats2half2_rn(y0, y1);
        const float2 r = __half22float2(u);
        hi[j] = h2u(u);
        lo[j] = h2u(__floats2half2_rn(y0 - r.x, y1 - r.y));
      }
      const bool low = NT == 1 && g >= 4;
      sh.q[2 * warp + s][0][lane] = low ? make_uint2(lo[0], lo[1]) : make_uint2(hi[0], hi[1]);
      if (NT == 2) sh.q[2 * warp + s][1][lane] = make_uint2(lo[0], lo[1]);
    }
  }
#pragma unroll
  for (int i = 1; i < kDepth4 - 1; ++i) start_copy(i);
  __syncthreads();
  // Eight heads' fragments are read again at each use, as they would take 32 of
  // the registers that keep the loads and the unpacking apart (16 ragged
  // sequences of up to 16384 rows: 40.5 -> 38.2 us).  Four heads' stay in
  // registers (read again: 38.1 -> 39.2 us at 131072 rows).
  const uint32_t q_u32 = static_cast<uint32_t>(__cvta_generic_to_shared(&sh.q[0][0][lane]));
  uint2 q1[8];
  if constexpr (NT == 1) {
#pragma unroll
    for (int s = 0; s < 8; ++s) q1[s] = sh.q[s][0][lane];
  }
  auto qf = [&](int s, int c) {
    if constexpr (NT == 1) {
      return q1[s];
    } else {
      uint2 r;
      asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(q_u32 + (s * NT + c) * (int)sizeof(sh.q[0][0])));
      return r;
    }
  };
  // a thread's columns: heads hc and hc + 1
  const int hc = NT == 1 ? 2 * (t & 1) : 2 * t;
  const float qs[2] = {sh.qscale[hc], sh.qscale[hc + 1]};
  const __half2 c_even = __float2half2_rn(-64.5f), c_odd = __float2half2_rn(-72.f);

  float o[8][NT][4];
#pragma unroll
  for (int j = 0; j < 8; ++j)
#pragma unroll
    for (int c = 0; c < NT; ++c) o[j][c][0] = o[j][c][1] = o[j][c][2] = o[j][c][3] = 0.f;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};  // m: a product, before its scale qs
  float* sc = a.accumulate ? a.scores + ((int64_t)b * a.hq + qh0 + hc) * a.c.rmax + r_begin : nullptr;

  // Index 2x + y of an 8-row product stands for row 2x + (y ^ (x & 1)): the
  // rows of a key fragment's quarter warp then lie in different halves of
  // the banks, and of a value fragment's half warp in two.
  const int krow = (g & 6) + ((g & 1) ^ ((g >> 1) & 1));
  const int vrow[2] = {2 * t + (t & 1), 2 * t + ((t & 1) ^ 1)};
  int stage = 0;
#pragma unroll 1
  for (; row0 < n; row0 += kTile4) {
    {
      const int next = row0 + (kDepth4 - 1) * kTile4;
      const int to = stage == 0 ? kDepth4 - 1 : stage - 1;
      if (next < n) copy_step(ring_u32 + to * (int)sizeof(Step4), ahead, n - next, lane);
      asm volatile("cp.async.commit_group;\n" ::: "memory");
      asm volatile("cp.async.wait_group %0;\n" ::"n"(kDepth4 - 1) : "memory");
      __syncwarp();
    }
    const Step4& st = ring[stage];
    // p[u][r][c]: row krow + 8 r + 16 u, head hc + c
    float p[2][2][2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      float d[NT][4];
      uint4 kw[2];
      __half2 S[2], even[2], odd[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = 16 * u + 8 * i + krow;
        kw[i] = st.k[4 * r + t];
        S[i] = u2h((uint32_t) reinterpret_cast<const uint8_t*>(st.ks)[4 * r + t] * 0x00800080u);
        even[i] = __hmul2(S[i], c_even);
        odd[i] = __hmul2(S[i], c_odd);
      }
#pragma unroll
      for (int c = 0; c < NT; ++c) d[c][0] = d[c][1] = d[c][2] = d[c][3] = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t w0 = j == 0 ? kw[0].x : j == 1 ? kw[0].y : j == 2 ? kw[0].z : kw[0].w;
        const uint32_t w1 = j == 0 ? kw[1].x : j == 1 ? kw[1].y : j == 2 ? kw[1].z : kw[1].w;
        uint32_t a0, a1, a2, a3;
        unpack2(w0, magic, S[0], even[0], odd[0], a0, a2);
        unpack2(w1, magic, S[1], even[1], odd[1], a1, a3);
#pragma unroll
        for (int c = 0; c < NT; ++c) {
          const uint2 q = qf(2 * j, c);
          mma_f16(d[c], a0, a1, a2, a3, q.x, q.y);
        }
        unpack2(w0 >> 8, magic, S[0], even[0], odd[0], a0, a2);
        unpack2(w1 >> 8, magic, S[1], even[1], odd[1], a1, a3);
#pragma unroll
        for (int c = 0; c < NT; ++c) {
          const uint2 q = qf(2 * j + 1, c);
          mma_f16(d[c], a0, a1, a2, a3, q.x, q.y);
        }
      }
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          // the upper and the lower part's share
          const float x = d[0][2 * r + c];
          p[u][r][c] = NT == 1 ? x + __shfl_xor_sync(kFull, x, 2) : x + d[NT - 1][2 * r + c];
        }
    }
    if (row0 + kRows4 > n) {
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int r = 0; r < 2; ++r)
          if (row0 + 16 * u + 8 * r + krow >= n) p[u][r][0] = p[u][r][1] = -INFINITY;
    }
    if (sc != nullptr && (NT == 2 || t < 2)) {
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int x = row0 + 16 * u + 8 * r + krow;
          if (x < n) {
            if (hc < nh) sc[x] = p[u][r][0] * qs[0];
            if (hc + 1 < nh) sc[a.c.rmax + x] = p[u][r][1] * qs[1];
          }
        }
    }
    float mx[2];
#pragma unroll
    for (int c = 0; c < 2; ++c) mx[c] = fmaxf(fmaxf(p[0][0][c], p[0][1][c]), fmaxf(p[1][0][c], p[1][1][c]));
    // a maximum may lag by kGrowth4: weights stay below 2^8, and the sums are
    // scaled again a few times at most
    if (__any_sync(kFull, (mx[0] - m[0]) * qs[0] > kGrowth4 || (mx[1] - m[1]) * qs[1] > kGrowth4)) {
      float f[2];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) mx[c] = fmaxf(mx[c], __shfl_xor_sync(kFull, mx[c], off));
        const float mn = fmaxf(m[c], mx[c]);
        f[c] = mn == -INFINITY ? 1.f : exp2_fast((m[c] - mn) * qs[c]);
        m[c] = mn;
        l[c] *= f[c];
      }
      // a thread's columns of O^T are the same heads
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int c = 0; c < NT; ++c)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[j][c][i] *= f[i & 1];
    }
    // Weights are kept 2^kUp4 up, at most 2^15: down to 2^-32 of the largest
    // they still count in a half's subnormals.  The maximum is subtracted
    // before the scale: it is one of the products, so the largest weight is
    // 2^kUp4 at any size of the scores.  Taken off the scaled score in one fma,
    // its own rounding, 2^-24 of it, is left over in the exponent, and from
    // scores of 2^24 on takes weights past a half's range.
    uint32_t pb[2][2][NT];  // rows 8 r + 16 u, column tile
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float p0 = exp2_fast(fmaf(p[u][r][0] - m[0], qs[0], kUp4)), p1 = exp2_fast(fmaf(p[u][r][1] - m[1], qs[1], kUp4));
        l[0] += p0;
        l[1] += p1;
        const __half2 hi = __floats2half2_rn(p0, p1);
        const float2 f = __half22float2(hi);
        const __half2 lo = __floats2half2_rn(p0 - f.x, p1 - f.y);
        if (NT == 1) {
          pb[u][r][0] = transpose8(t < 2 ? h2u(hi) : h2u(lo));
        } else {
          pb[u][r][0] = transpose8(h2u(hi));
          pb[u][r][NT - 1] = transpose8(h2u(lo));
        }
      }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const uint8_t* vs = reinterpret_cast<const uint8_t*>(st.vs) + (g >> 1);
      const uint2* vc = reinterpret_cast<const uint2*>(st.v) + g;
      const int r0 = 16 * u + vrow[0], r1 = 16 * u + vrow[1];
      const uint2 xa = vc[8 * r0], xb = vc[8 * r1], ya = vc[8 * (r0 + 8)], yb = vc[8 * (r1 + 8)];
      const __half2 S0 = u2h((uint32_t)vs[4 * r0] << 7 | (uint32_t)vs[4 * r1] << 23);
      const __half2 S1 = u2h((uint32_t)vs[4 * (r0 + 8)] << 7 | (uint32_t)vs[4 * (r1 + 8)] << 23);
      const __half2 e0 = __hmul2(S0, c_even), d0 = __hmul2(S0, c_odd), e1 = __hmul2(S1, c_even), d1 = __hmul2(S1, c_odd);
#pragma unroll
      for (int w = 0; w < 2; ++w) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // byte i of the word: channels 16 g + 8 w + 2 i and the next
          const uint32_t sel = (uint32_t)(i | (i << 4) | ((4 + i) << 8) | ((4 + i) << 12));
          uint32_t a0, a1, a2, a3;
          unpack2(__byte_perm(w ? xa.y : xa.x, w ? xb.y : xb.x, sel), magic, S0, e0, d0, a0, a1);
          unpack2(__byte_perm(w ? ya.y : ya.x, w ? yb.y : yb.x, sel), magic, S1, e1, d1, a2, a3);
#pragma unroll
          for (int c = 0; c < NT; ++c) mma_f16(o[4 * w + i][c], a0, a1, a2, a3, pb[u][0][c], pb[u][1][c]);
        }
      }
    }
    stage = stage + 1 == kDepth4 ? 0 : stage + 1;
    __syncwarp();  // the stage may be filled again
  }
  asm volatile("cp.async.wait_all;\n" ::: "memory");
#pragma unroll
  for (int c = 0; c < 2; ++c) {
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) l[c] += __shfl_xor_sync(kFull, l[c], off);
    if (g == 0 && (NT == 2 || t < 2)) {
      sh.ml[warp][hc + c][0] = m[c] * qs[c];  // qs > 0
      sh.ml[warp][hc + c][1] = l[c] * kDown4;
    }
  }
  __syncthreads();
  // every warp's result in the rings' place: [warp][head][channel]; rows g and
  // g + 8 of tile j are channels 16 g + 2 j and the next
  float* so = reinterpret_cast<float*>(ring_mem);
#pragma unroll
  for (int j = 0; j < 8; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float x = o[j][0][i], low = NT == 1 ? __shfl_xor_sync(kFull, x, 2) : o[j][NT - 1][i];
      if (NT == 2 || t < 2)
        so[(warp * kHeads4 + hc + (i & 1)) * kDim + 16 * g + 2 * j + (i >> 1)] = (x + low) * (i < 2 ? 16.f * kDown4 : kDown4);
    }
  __syncthreads();
  for (int e = tid; e < nh * kDim; e += kThreads4) {
    const int h = e / kDim, dd = e - h * kDim;
    float M = sh.ml[0][h][0];
#pragma unroll
    for (int w = 1; w < kWarps4; ++w) M = fmaxf(M, sh.ml[w][h][0]);
    float L = 0.f, O = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps4; ++w) {
      // a warp without rows has the sum 0; one whose scores are all NaN has
      // m = -inf too, and a NaN sum
      const float mw = sh.ml[w][h][0], lw = sh.ml[w][h][1], f = lw == 0.f ? 0.f : exp2_fast(mw - M);
      L += lw * f;
      O += so[(w * kHeads4 + h) * kDim + dd] * f;
    }
    float* ph = part + (int64_t)h * a.nblocks * kPartStride;
    ph[4 + dd] = O;
    if (dd == 0) {
      ph[0] = M;
      ph[1] = L;
    }
  }
}

// A warp: the maximum and the sum of one head over its splits; `first`: those
// of split `lane`, which may be anything where there is none.
__device__ __forceinline__ float2 merge_ml(const float* ph, int nsplit, int lane, float2 first) {
  auto ml_of = [&](int s) { return *reinterpret_cast<const float2*>(ph + (int64_t)s * kPartStride); };
  if (lane >= nsplit) first = make_float2(-INFINITY, 0.f);
  float M = first.x;
  for (int s = lane + 32; s < nsplit; s += 32) M = fmaxf(M, ml_of(s).x);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(kFull, M, off));
  float L = first.y != 0.f ? first.y * exp2_fast(first.x - M) : 0.f;  // the sum 0: no rows
  for (int s = lane + 32; s < nsplit; s += 32) {
    const float2 ml = ml_of(s);
    if (ml.y != 0.f) L += ml.y * exp2_fast(ml.x - M);
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) L += __shfl_xor_sync(kFull, L, off);
  return make_float2(M, L);
}

// The first blocks merge the splits of `per_block` query heads each, with
// all of a warp's loads in flight at once; the others add the weights of four
// rows a thread, head by head in ascending order.
template <int kFinishThreads>
__global__ void __launch_bounds__(kFinishThreads, kFinishThreads == 256 ? 4 : 1) k_kv4_finish(Attend4Args a, int per_block) {
  constexpr int kFinishWarps = kFinishThreads / 32, kFinishRows = 4 * kFinishThreads;
  __shared__ float2 sml[16];  // maximum, 1 / sum
  __shared__ float4 so[kFinishWarps][32];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int b = blockIdx.y / a.c.hkv, kvh = blockIdx.y - b * a.c.hkv;
  const int64_t q0 = (int64_t)b * a.hq + kvh * a.g;
  const int2 chunk = a.chunks[b];
  const int64_t len = kv4_len(a.c, b);
  const int merging = (a.g + per_block - 1) / per_block;
  const int nsplit = len > 0 ? chunk.y : 0;
  // of one sequence the first chunk is known, and its partials are loaded
  // before their number is: one round trip to memory less
  const bool one = a.c.batch == 1;
  const float* part = a.part + (int64_t)kvh * a.g * a.nblocks * kPartStride;
  if (!one) part += (int64_t)chunk.x * kPartStride;
  const int limit = one ? a.nblocks : nsplit;
  if ((int)blockIdx.x < merging) {
    const int each = kFinishWarps / per_block, sub = warp % each;
    const int h = blockIdx.x * per_block + warp / each;
    const bool live = h < a.g;
    const float* ph = part + (int64_t)h * a.nblocks * kPartStride;
    constexpr int kAhead = kFinishThreads == 256 ? 4 : 8;
    float4 x[kAhead];
    float2 ml[kAhead];
    const int most = live ? limit : 0, n = live ? nsplit : 0;
    auto load = [&](int s0) {
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int s = s0 + sub + i * each;
        if (s >= most) continue;
        ml[i] = *reinterpret_cast<const float2*>(ph + (int64_t)s * kPartStride);
        x[i] = *reinterpret_cast<const float4*>(ph + (int64_t)s * kPartStride + 4 + 4 * lane);  // not written without rows
      }
    };
    load(0);
    const float2 first = lane < most ? *reinterpret_cast<const float2*>(ph + (int64_t)lane * kPartStride) : make_float2(0.f, 0.f);
    const float2 all = merge_ml(ph, n, lane, first);
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int s0 = 0; s0 < n; s0 += kAhead * each) {
      if (s0 > 0) load(s0);
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        if (s0 + sub + i * each >= n || ml[i].y == 0.f) continue;
        const float f = exp2_fast(ml[i].x - all.x);
        o.x = fmaf(x[i].x, f, o.x);
        o.y = fmaf(x[i].y, f, o.y);
        o.z = fmaf(x[i].z, f, o.z);
        o.w = fmaf(x[i].w, f, o.w);
      }
    }
    if (each > 1) {
      so[warp][lane] = o;
      __syncthreads();
      if (sub > 0 || !live) return;
      for (int w = 1; w < each; ++w) {
        const float4 y = so[warp + w][lane];
        o.x += y.x;
        o.y += y.y;
        o.z += y.z;
        o.w += y.w;
      }
    }
    if (!live) return;
    const float inv = all.y != 0.f ? 1.f / all.y : 0.f;
    *reinterpret_cast<uint2*>(a.out + (q0 + h) * kDim + 4 * lane) =
        make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
    return;
  }
  const int64_t r0 = ((int64_t)blockIdx.x - merging) * kFinishRows, r1 = min64(len, r0 + kFinishRows);
  if (r0 >= len) return;
  float* w = a.c.w + (int64_t)blockIdx.y * a.c.rmax;
  const float* sc = a.scores + q0 * a.c.rmax;
  // where heads are 16-byte aligned, four rows a thread, on their way while the
  // splits are merged; of those behind the last, which lie within the same
  // head, nothing is written
  constexpr int kHeadsAhead = 8;
  const bool vec = a.c.rmax % 4 == 0;
  const int64_t rv = r0 + 4 * tid;
  float4 x[kHeadsAhead], old = make_float4(0.f, 0.f, 0.f, 0.f);
  if (vec && rv < len) {
    old = *reinterpret_cast<const float4*>(w + rv);
#pragma unroll
    for (int h = 0; h < kHeadsAhead; ++h)
      if (h < a.g) x[h] = *reinterpret_cast<const float4*>(sc + h * a.c.rmax + rv);
  }
  for (int h = warp; h < a.g; h += kFinishWarps) {
    const float* ph = part + (int64_t)h * a.nblocks * kPartStride;
    const float2 first = lane < limit ? *reinterpret_cast<const float2*>(ph + (int64_t)lane * kPartStride) : make_float2(0.f, 0.f);
    const float2 all = merge_ml(ph, nsplit, lane, first);
    if (lane == 0) sml[h] = make_float2(all.x, all.y != 0.f ? 1.f / all.y : 0.f);
  }
  __syncthreads();
  if (vec) {
    if (rv >= len) return;
    float4 p = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](const float4& v, int h) {
      const float2 ml = sml[h];
      p.x += exp2_fast(v.x - ml.x) * ml.y;
      p.y += exp2_fast(v.y - ml.x) * ml.y;
      p.z += exp2_fast(v.z - ml.x) * ml.y;
      p.w += exp2_fast(v.w - ml.x) * ml.y;
    };
#pragma unroll
    for (int h = 0; h < kHeadsAhead; ++h)
      if (h < a.g) add(x[h], h);
    for (int h = kHeadsAhead; h < a.g; ++h) add(*reinterpret_cast<const float4*>(sc + h * a.c.rmax + rv), h);
    p = make_float4(old.x + p.x, old.y + p.y, old.z + p.z, old.w + p.w);
    if (rv + 4 <= len) {
      *reinterpret_cast<float4*>(w + rv) = p;
      return;
    }
    w[rv] = p.x;
    if (rv + 1 < len) w[rv + 1] = p.y;
    if (rv + 2 < len) w[rv + 2] = p.z;
    return;
  }
  for (int64_t r = r0 + tid; r < r1; r += kFinishThreads) {
    float p = 0.f;
#pragma unroll 4
    for (int h = 0; h < a.g; ++h) p += exp2_fast(sc[h * a.c.rmax + r] - sml[h].x) * sml[h].y;
    w[r] += p;
  }
}

}  // namespace

int kv4_blocks(int batch, int hkv, int g, int64_t rmax, int sm_count) {
  // one wave of blocks for each KV head and head group, of one tile at least (a
  // step of 2049 rows, append and eviction with it, on the GPU alone: 14.4 us,
  // 15.8 with two); a batch that is cut by its
  // lengths needs more blocks than sequences, and one that is cut evenly a
  // multiple of its sequences
  const int64_t wave = std::max<int64_t>(1, (g <= 4 ? 4 : 3) * (int64_t)sm_count / ((int64_t)hkv * ((g + 7) / 8)));
  const int64_t tiles = (rmax + kTile4 - 1) / kTile4;
  if (batch > 128) return (int)(batch * std::max<int64_t>(1, std::min(wave / batch, tiles)));
  const int64_t most = batch * tiles + (batch > 1 ? batch : 0);
  return (int)std::max<int64_t>(std::min(wave, most), batch > 1 ? batch + 1 : 1);
}

namespace {

template <int NT>
cudaError_t launch_attend4(const Attend4Args& a, cudaStream_t st) {
  constexpr int smem = kWarps4 * kDepth4 * (int)sizeof(Step4);
  static std::atomic<bool> done[64];  // the limit belongs to the device; setting it twice is harmless
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess && !(dev >= 0 && dev < 64 && done[dev])) {
    e = cudaFuncSetAttribute((const void*)k_kv4_attend<NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess && dev >= 0 && dev < 64) done[dev] = true;
  }
  if (e != cudaSuccess) return e;
  const dim3 grid(a.nblocks, a.c.hkv, (a.g + 4 * NT - 1) / (4 * NT));
  return launch_pdl(k_kv4_attend<NT>, grid, dim3(kThreads4), smem, st, a, kMagic4);
}

}  // namespace

cudaError_t launch_kv4_attend(const Attend4Args& a, cudaStream_t st) {
  cudaError_t e = a.g <= 4 ? launch_attend4<1>(a, st) : launch_attend4<2>(a, st);
  if (e != cudaSuccess) return e;
  // few splits a sequence: a warp merges a head; many: a block, of 16 warps
  // where it is all that there is to do (76 splits: 5.9 -> 3.5 us)
  const int per_block = a.nblocks <= 16 * a.c.batch ? 8 : 1;
  const unsigned heads = (unsigned)(a.g + per_block - 1) / per_block, units = a.c.batch * a.c.hkv;
  if (per_block == 1 && !a.accumulate) return launch_pdl(k_kv4_finish<512>, dim3(heads, units), dim3(512), 0, st, a, 1);
  const unsigned rows = a.accumulate ? (unsigned)((a.c.rmax + 1023) / 1024) : 0u;
  return launch_pdl(k_kv4_finish<256>, dim3(heads + rows, units), dim3(256), 0, st, a, per_block);
}

}  // namespace paris
