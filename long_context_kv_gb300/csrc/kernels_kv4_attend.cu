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
//   The weights go from the one's result to the other's operand by 8x8
//   transposes in registers.
//
// A warp walks its rows 32 at a time with a running maximum and sum per
// head, its next steps' rows on the way to its own ring in shared memory; no
// warp waits for another until the end.  Partials of (split, head) are merged
// by k_kv4_finish, which also turns the scores into weights.
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
constexpr int kDepth4 = 3;                     // steps of a warp's ring
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

struct Rows4 {  // a split's rows
  const uint8_t *kc, *vc, *ks, *vs;
};

// Start the copy of rows [row0, row0 + 32); past `last` the last row again
// (its weights are set to zero).
__device__ __forceinline__ void copy_step(uint32_t dst, const Rows4& p, int row0, int last, int lane) {
  if (row0 + kRows4 - 1 <= last) {
    const uint8_t *k = p.kc + (int64_t)row0 * kCode4 + 16 * lane, *v = p.vc + (int64_t)row0 * kCode4 + 16 * lane;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      copy16(dst + 16 * lane + 512 * i, k + 512 * i);
      copy16(dst + 2048 + 16 * lane + 512 * i, v + 512 * i);
    }
  } else {
#pragma unroll 1
    for (int i = 0; i < 4; ++i) {
      const int64_t r = min(row0 + 8 * i + (lane >> 2), last);
      copy16(dst + 16 * lane + 512 * i, p.kc + r * kCode4 + 16 * (lane & 3));
      copy16(dst + 2048 + 16 * lane + 512 * i, p.vc + r * kCode4 + 16 * (lane & 3));
    }
  }
  const int64_t r = min(row0 + lane, last);
  copy4(dst + 4096 + 4 * lane, p.ks + r * kScale4);
  copy4(dst + 4224 + 4 * lane, p.vs + r * kScale4);
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
  const int split = blockIdx.x, bh = blockIdx.y, h0 = blockIdx.z * kHeads;
  const int b = bh / a.c.hkv, kvh = bh - b * a.c.hkv;
  const int nh = min(kHeads, a.g - h0);
  const int qh0 = kvh * a.g + h0;  // first query head of the block
  const int64_t len = kv4_len(a.c, b);
  const int64_t r_begin = (int64_t)split * a.rows_per_split;
  float* part = a.part + (((int64_t)b * a.hq + qh0) * a.nsplit + split) * kPartStride;
  if (r_begin >= len) {
    if (tid < nh) {
      part[(int64_t)tid * a.nsplit * kPartStride] = -INFINITY;
      part[(int64_t)tid * a.nsplit * kPartStride + 1] = 0.f;
    }
    return;
  }
  // rows of this split from its first on, and of the sequence
  const int n = (int)min64(len - r_begin, a.rows_per_split);
  const int64_t base = (int64_t)bh * a.c.rmax + r_begin;
  const Rows4 rows{a.c.kc + base * kCode4, a.c.vc + base * kCode4, a.c.ks + base * kScale4, a.c.vs + base * kScale4};
  const Step4* ring = reinterpret_cast<const Step4*>(ring_mem) + warp * kDepth4;
  const uint32_t ring_u32 = static_cast<uint32_t>(__cvta_generic_to_shared(ring));
  int row0 = warp * kRows4;
#pragma unroll
  for (int i = 0; i < kDepth4 - 1; ++i) {
    if (row0 + i * kTile4 < n) copy_step(ring_u32 + i * (int)sizeof(Step4), rows, row0 + i * kTile4, n - 1, lane);
    asm volatile("cp.async.commit_group;\n" ::: "memory");
  }

  // The query of column g's head as two half parts, scaled by a power of two
  // to at most 1 (its scores are scaled back, with log2(e) / sqrt(d)); each
  // warp makes two of the eight steps' fragments.
  {
    const int h = NT == 1 ? g & 3 : g;
    float amax = 0.f;
    const int64_t qe = ((int64_t)b * a.hq + qh0 + h) * kDim + 32 * t;
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float y[4] = {0.f, 0.f, 0.f, 0.f};
      if (h < nh) load4(a.q, a.dtype, qe + 4 * i, y);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        amax = fmaxf(amax, fabsf(y[j]));
        if (i >> 1 == warp) x[4 * (i & 1) + j] = y[j];
      }
    }
    amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 2));
    // 2^(e + 1) > amax; exponents beyond +-100 are left to overflow to the
    // infinities that such queries' scores are anyway
    const int e = min(max((int)((__float_as_uint(amax) >> 23) & 255u) - 126, -100), 100);
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
  __syncthreads();
  uint2 qf[8][NT];
#pragma unroll
  for (int s = 0; s < 8; ++s)
#pragma unroll
    for (int c = 0; c < NT; ++c) qf[s][c] = sh.q[s][c][lane];
  // a thread's columns: heads hc and hc + 1
  const int hc = NT == 1 ? 2 * (t & 1) : 2 * t;
  const float qs[2] = {sh.qscale[hc], sh.qscale[hc + 1]};
  const __half2 c_even = __float2half2_rn(-64.5f), c_odd = __float2half2_rn(-72.f);

  float o[8][NT][4];
#pragma unroll
  for (int j = 0; j < 8; ++j)
#pragma unroll
    for (int c = 0; c < NT; ++c) o[j][c][0] = o[j][c][1] = o[j][c][2] = o[j][c][3] = 0.f;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
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
      if (next < n) copy_step(ring_u32 + to * (int)sizeof(Step4), rows, next, n - 1, lane);
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
        for (int c = 0; c < NT; ++c) mma_f16(d[c], a0, a1, a2, a3, qf[2 * j][c].x, qf[2 * j][c].y);
        unpack2(w0 >> 8, magic, S[0], even[0], odd[0], a0, a2);
        unpack2(w1 >> 8, magic, S[1], even[1], odd[1], a1, a3);
#pragma unroll
        for (int c = 0; c < NT; ++c) mma_f16(d[c], a0, a1, a2, a3, qf[2 * j + 1][c].x, qf[2 * j + 1][c].y);
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
    for (int c = 0; c < 2; ++c) mx[c] = fmaxf(fmaxf(p[0][0][c], p[0][1][c]), fmaxf(p[1][0][c], p[1][1][c])) * qs[c];
    // a maximum may lag by kGrowth4: weights stay below 2^8, and the sums are
    // scaled again a few times at most
    if (__any_sync(kFull, mx[0] > m[0] + kGrowth4 || mx[1] > m[1] + kGrowth4)) {
      float f[2];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) mx[c] = fmaxf(mx[c], __shfl_xor_sync(kFull, mx[c], off));
        const float mn = fmaxf(m[c], mx[c]);
        f[c] = mn == -INFINITY ? 1.f : exp2_fast(m[c] - mn);
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
    // weights are kept 2^kUp4 up, at most 2^15: down to 2^-32 of the largest
    // they still count in a half's subnormals
    const float neg[2] = {kUp4 - m[0], kUp4 - m[1]};
    uint32_t pb[2][2][NT];  // rows 8 r + 16 u, column tile
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float p0 = exp2_fast(fmaf(p[u][r][0], qs[0], neg[0])), p1 = exp2_fast(fmaf(p[u][r][1], qs[1], neg[1]));
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
      sh.ml[warp][hc + c][0] = m[c];
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
      const float mw = sh.ml[w][h][0], lw = sh.ml[w][h][1], f = lw == 0.f ? 0.f : exp2f(mw - M);
      L += lw * f;
      O += so[(w * kHeads4 + h) * kDim + dd] * f;
    }
    float* ph = part + (int64_t)h * a.nsplit * kPartStride;
    ph[4 + dd] = O;
    if (dd == 0) {
      ph[0] = M;
      ph[1] = L;
    }
  }
}

constexpr int kFinishThreads = 512;
constexpr int kFinishWarps = kFinishThreads / 32;
constexpr int kFinishRows = 2048;  // rows whose weights a block adds up
constexpr int kMaxSplit4 = 512;

// A warp: the maximum and the sum of one head over its splits.
__device__ __forceinline__ float2 merge_ml(const float* ph, int nsplit, int lane) {
  float M = -INFINITY, L = 0.f;
#pragma unroll 4
  for (int s = lane; s < nsplit; s += 32) {
    const float2 ml = *reinterpret_cast<const float2*>(ph + (int64_t)s * kPartStride);
    if (ml.y == 0.f) continue;  // no rows
    const float mn = fmaxf(M, ml.x);
    L = (L != 0.f ? L * exp2f(M - mn) : 0.f) + ml.y * exp2f(ml.x - mn);
    M = mn;
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    const float om = __shfl_xor_sync(kFull, M, off), ol = __shfl_xor_sync(kFull, L, off);
    const float mn = fmaxf(M, om);
    L = (L != 0.f ? L * exp2f(M - mn) : 0.f) + (ol != 0.f ? ol * exp2f(om - mn) : 0.f);
    M = mn;
  }
  return make_float2(M, L);
}

// Blocks [0, G): merge the splits of one query head, a warp taking every
// 16th split with all its loads in flight at once.  Blocks from G on: add a
// range of rows' weights, head by head in ascending order.
__global__ void __launch_bounds__(kFinishThreads) k_kv4_finish(Attend4Args a) {
  __shared__ float2 sml[16];  // maximum, 1 / sum
  __shared__ float4 so[kFinishWarps][32];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int b = blockIdx.y / a.c.hkv, kvh = blockIdx.y - b * a.c.hkv;
  const int64_t q0 = (int64_t)b * a.hq + kvh * a.g;
  if ((int)blockIdx.x < a.g) {
    const float* ph = a.part + (q0 + blockIdx.x) * a.nsplit * kPartStride;
    constexpr int kAhead = 8;
    float4 x[kAhead];
    float2 ml[kAhead];
    auto load = [&](int s0) {
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int s = s0 + warp + i * kFinishWarps;
        ml[i] = make_float2(-INFINITY, 0.f);
        if (s >= a.nsplit) continue;
        ml[i] = *reinterpret_cast<const float2*>(ph + (int64_t)s * kPartStride);
        x[i] = *reinterpret_cast<const float4*>(ph + (int64_t)s * kPartStride + 4 + 4 * lane);  // not written without rows
      }
    };
    load(0);
    const float2 all = merge_ml(ph, a.nsplit, lane);
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int s0 = 0; s0 < a.nsplit; s0 += kAhead * kFinishWarps) {
      if (s0 > 0) load(s0);
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        if (ml[i].y == 0.f) continue;
        const float f = exp2f(ml[i].x - all.x);
        o.x = fmaf(x[i].x, f, o.x);
        o.y = fmaf(x[i].y, f, o.y);
        o.z = fmaf(x[i].z, f, o.z);
        o.w = fmaf(x[i].w, f, o.w);
      }
    }
    so[warp][lane] = o;
    __syncthreads();
    if (tid < kDim) {
      float r = 0.f;
#pragma unroll
      for (int w = 0; w < kFinishWarps; ++w) r += reinterpret_cast<const float*>(so[w])[tid];
      a.out[(q0 + blockIdx.x) * kDim + tid] = __float2bfloat16_rn(all.y != 0.f ? r / all.y : 0.f);
    }
    return;
  }
  const int64_t len = kv4_len(a.c, b);
  const int64_t r0 = ((int64_t)blockIdx.x - a.g) * kFinishRows, r1 = min64(len, r0 + kFinishRows);
  if (r0 >= len) return;
  if (warp < a.g) {
    const float2 all = merge_ml(a.part + (q0 + warp) * a.nsplit * kPartStride, a.nsplit, lane);
    if (lane == 0) sml[warp] = make_float2(all.x, all.y != 0.f ? 1.f / all.y : 0.f);
  }
  float* w = a.c.w + (int64_t)blockIdx.y * a.c.rmax;
  const float* sc = a.scores + q0 * a.c.rmax;
  __syncthreads();
  for (int64_t r = r0 + tid; r < r1; r += kFinishThreads) {
    float p = 0.f;
#pragma unroll 4
    for (int h = 0; h < a.g; ++h) p += exp2f(sc[h * a.c.rmax + r] - sml[h].x) * sml[h].y;
    w[r] += p;
  }
}

}  // namespace

void kv4_splits(int64_t heads, int g, int64_t rmax, int sm_count, int* nsplit, int64_t* rows_per_split) {
  // one wave of blocks over all (sequence, KV head, head group)s, at least
  // two steps of a block each
  const int64_t units = heads * ((g + 7) / 8), slots = (g <= 4 ? 4 : 3) * (int64_t)sm_count;
  const int64_t want = std::max<int64_t>(1, slots / units);
  const int64_t most = std::max<int64_t>(1, (rmax + 2 * kTile4 - 1) / (2 * kTile4));
  const int64_t n = std::min<int64_t>({want, most, kMaxSplit4});
  *rows_per_split = std::max<int64_t>(kTile4, ((rmax + n - 1) / n + kTile4 - 1) / kTile4 * kTile4);
  *nsplit = (int)std::max<int64_t>(1, (rmax + *rows_per_split - 1) / *rows_per_split);
}

namespace {

template <int NT>
cudaError_t launch_attend4(const Attend4Args& a, cudaStream_t st) {
  constexpr int smem = kWarps4 * kDepth4 * (int)sizeof(Step4);
  static bool done[64];  // the limit belongs to the device; setting it twice is harmless
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess && !(dev >= 0 && dev < 64 && done[dev])) {
    e = cudaFuncSetAttribute((const void*)k_kv4_attend<NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess && dev >= 0 && dev < 64) done[dev] = true;
  }
  if (e != cudaSuccess) return e;
  const dim3 grid(a.nsplit, a.c.batch * a.c.hkv, (a.g + 4 * NT - 1) / (4 * NT));
  return launch_pdl(k_kv4_attend<NT>, grid, dim3(kThreads4), smem, st, a, kMagic4);
}

}  // namespace

cudaError_t launch_kv4_attend(const Attend4Args& a, cudaStream_t st) {
  cudaError_t e = a.g <= 4 ? launch_attend4<1>(a, st) : launch_attend4<2>(a, st);
  if (e != cudaSuccess) return e;
  const int64_t rows = a.accumulate ? (a.c.rmax + kFinishRows - 1) / kFinishRows : 0;
  return launch_pdl(k_kv4_finish, dim3((unsigned)(a.g + rows), a.c.batch * a.c.hkv), dim3(kFinishThreads), 0, st, a);
}

}  // namespace paris
