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
// - A code word x becomes pairs of halves with one shift for two pairs, one
//   logic operation and one fma each: the nibble lands in the mantissa of 256 (bits
//   2-5) or 16 (bits 6-9), giving 256 + u or 16 + u, and the fma with S and
//   -264 S or -24 S gives S (u - 8) exactly (S has four significant bits, so
//   every term fits a half's eleven).
// - The M side of the mma has 16 rows for at most 8 query heads, so rows
//   0-7 hold the upper and rows 8-15 the lower half-precision part of the
//   queries, and then of the softmax weights: 22 bits for the cost of 11.
// - The score fragments are already the weight fragments of the second
//   product (rows: heads; columns: tokens), as in any m16n8k16 chain.
//
// A warp walks its rows 32 at a time with a running maximum and sum per
// head; the next 32 rows' loads are in flight meanwhile.  Partials of (split, head)
// are merged by k_kv4_finish, which also turns the scores into weights.
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

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
               "{%0,%1,%2,%3};\n"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t h2u(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }
__device__ __forceinline__ __half2 u2h(uint32_t u) { return *reinterpret_cast<__half2*>(&u); }

// The four nibbles of each half of x (two words' or one word's) as four
// pairs of halves, times their scales: v[i] = S (nibble i - 8).
__device__ __forceinline__ void unpack4(uint32_t x, __half2 S, __half2 m264, __half2 m24, uint32_t (&v)[4]) {
  const uint32_t z = x << 2, y = x >> 6;
  v[0] = h2u(__hfma2(u2h((z & 0x003C003Cu) | 0x5C005C00u), S, m264));
  v[1] = h2u(__hfma2(u2h((z & 0x03C003C0u) | 0x4C004C00u), S, m24));
  v[2] = h2u(__hfma2(u2h((y & 0x003C003Cu) | 0x5C005C00u), S, m264));
  v[3] = h2u(__hfma2(u2h((y & 0x03C003C0u) | 0x4C004C00u), S, m24));
}

struct Step4 {  // one 32-row step of a warp as loaded
  uint4 k[4];        // rows 8 i + lane / 4, bytes 16 (lane % 4) ...
  uint32_t ks[4];    // their scale byte
  uint2 v[4][2];     // rows 8 i + 2 (lane % 4) + {0, 1}, bytes 8 (lane / 4) ...
  uint32_t vs[4][2];
};

__device__ __forceinline__ void load_step(Step4& s, const uint8_t* kc, const uint8_t* ks, const uint8_t* vc,
                                          const uint8_t* vs, int64_t row0, int64_t last, int g, int t) {
  // rows past the end read the last row again; their weights become zero
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t r = min64(row0 + 8 * i + g, last);
    s.k[i] = __ldg(reinterpret_cast<const uint4*>(kc + r * kCode4 + 16 * t));
    s.ks[i] = __ldg(ks + r * kScale4 + t);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int64_t rv = min64(row0 + 8 * i + 2 * t + j, last);
      s.v[i][j] = __ldg(reinterpret_cast<const uint2*>(vc + rv * kCode4 + 8 * g));
      s.vs[i][j] = __ldg(vs + rv * kScale4 + (g >> 1));
    }
  }
}

__global__ void __launch_bounds__(kThreads4) k_kv4_attend(Attend4Args a) {
  __shared__ float so[kWarps4][kHeads4][kDim];
  __shared__ float sml[kWarps4][kHeads4][2];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int split = blockIdx.x, bh = blockIdx.y, h0 = blockIdx.z * kHeads4;
  const int b = bh / a.c.hkv, kvh = bh - b * a.c.hkv;
  const int nh = min(kHeads4, a.g - h0);
  const int qh0 = kvh * a.g + h0;  // first query head of the block
  const int64_t len = kv4_len(a.c, b);
  const int64_t r_begin = (int64_t)split * a.rows_per_split, r_end = min64(len, r_begin + a.rows_per_split);
  float* part = a.part + (((int64_t)b * a.hq + qh0) * a.nsplit + split) * kPartStride;
  if (r_begin >= r_end) {
    if (tid < nh) {
      part[(int64_t)tid * a.nsplit * kPartStride] = -INFINITY;
      part[(int64_t)tid * a.nsplit * kPartStride + 1] = 0.f;
    }
    return;
  }
  const int64_t base = (int64_t)bh * a.c.rmax;
  const uint8_t *kc = a.c.kc + base * kCode4, *ks = a.c.ks + base * kScale4;
  const uint8_t *vc = a.c.vc + base * kCode4, *vs = a.c.vs + base * kScale4;

  // the query of head g as two half parts, scaled by a power of two to at
  // most 1 (its scores are scaled back, with log2(e) / sqrt(d))
  uint32_t qa[8][4];
  float qscale;
  {
    float x[32];
    float amax = 0.f;
    const int64_t qe = ((int64_t)b * a.hq + qh0 + g) * kDim + 32 * t;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float y[4] = {0.f, 0.f, 0.f, 0.f};
      if (g < nh) load4(a.q, a.dtype, qe + 4 * i, y);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x[4 * i + j] = y[j];
        amax = fmaxf(amax, fabsf(y[j]));
      }
    }
    amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 2));
    // 2^(e + 1) > amax; exponents beyond +-100 are left to overflow to the
    // infinities that such queries' scores are anyway
    const int e = min(max((int)((__float_as_uint(amax) >> 23) & 255u) - 126, -100), 100);
    const float down = __uint_as_float((uint32_t)(127 - e) << 23);
    qscale = __uint_as_float((uint32_t)(127 + e) << 23) * (1.4426950408889634f * 0.08838834764831845f);
#pragma unroll
    for (int s = 0; s < 8; ++s) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        // fragment slots of step s: channels c and c + 4, c = 8 (s / 2) + 2 (s % 2) + j
        const int c = 8 * (s >> 1) + 2 * (s & 1) + j;
        const float y0 = x[c] * down, y1 = x[c + 4] * down;
        const __half2 hi = __floats2half2_rn(y0, y1);
        const float2 f = __half22float2(hi);
        qa[s][2 * j] = h2u(hi);
        qa[s][2 * j + 1] = h2u(__floats2half2_rn(y0 - f.x, y1 - f.y));
      }
    }
  }
  const __half2 c264 = __float2half2_rn(-264.f), c24 = __float2half2_rn(-24.f);

  float o[16][4];
#pragma unroll
  for (int j = 0; j < 16; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
  float m = -INFINITY, l = 0.f;
  float* sc = a.accumulate ? a.scores + ((int64_t)b * a.hq + qh0 + g) * a.c.rmax : nullptr;

  Step4 cur;
  int64_t row0 = r_begin + warp * kRows4;
  if (row0 < r_end) load_step(cur, kc, ks, vc, vs, row0, len - 1, g, t);
  for (; row0 < r_end; row0 += kTile4) {
    Step4 s = cur;
    if (row0 + kTile4 < r_end) load_step(cur, kc, ks, vc, vs, row0 + kTile4, len - 1, g, t);
    float p[4][2];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float d[4] = {0.f, 0.f, 0.f, 0.f};
      const __half2 S = u2h((s.ks[i] << 7) * 0x10001u);
      const __half2 m264 = __hmul2(S, c264), m24 = __hmul2(S, c24);
      const uint32_t w[4] = {s.k[i].x, s.k[i].y, s.k[i].z, s.k[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t v[4];
        unpack4(w[j], S, m264, m24, v);
        mma_f16(d, qa[2 * j][0], qa[2 * j][1], qa[2 * j][2], qa[2 * j][3], v[0], v[1]);
        mma_f16(d, qa[2 * j + 1][0], qa[2 * j + 1][1], qa[2 * j + 1][2], qa[2 * j + 1][3], v[2], v[3]);
      }
      const int64_t r = row0 + 8 * i + 2 * t;
      p[i][0] = r < r_end ? (d[0] + d[2]) * qscale : -INFINITY;
      p[i][1] = r + 1 < r_end ? (d[1] + d[3]) * qscale : -INFINITY;
      if (sc != nullptr && g < nh) {
        if (r < r_end) sc[r] = p[i][0];
        if (r + 1 < r_end) sc[r + 1] = p[i][1];
      }
    }
    float mx = p[0][0];
#pragma unroll
    for (int i = 0; i < 4; ++i) mx = fmaxf(mx, fmaxf(p[i][0], p[i][1]));
    mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 1));
    mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 2));
    if (__any_sync(kFull, mx > m)) {
      const float mn = fmaxf(m, mx);
      const float f = mn == -INFINITY ? 1.f : exp2f(m - mn);
      m = mn;
      l *= f;
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        o[j][0] *= f;
        o[j][1] *= f;
        o[j][2] *= f;
        o[j][3] *= f;
      }
    }
    uint32_t ph[4], pl[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float p0 = exp2f(p[i][0] - m), p1 = exp2f(p[i][1] - m);
      l += p0 + p1;
      const __half2 hi = __floats2half2_rn(p0, p1);
      const float2 f = __half22float2(hi);
      ph[i] = h2u(hi);
      pl[i] = h2u(__floats2half2_rn(p0 - f.x, p1 - f.y));
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {  // 16 rows: row pairs of 8-row groups 2u and 2u + 1
      const __half2 S0 = u2h((s.vs[2 * u][0] << 7) | (s.vs[2 * u][1] << 23));
      const __half2 S1 = u2h((s.vs[2 * u + 1][0] << 7) | (s.vs[2 * u + 1][1] << 23));
      const __half2 a0 = __hmul2(S0, c264), b0 = __hmul2(S0, c24), a1 = __hmul2(S1, c264), b1 = __hmul2(S1, c24);
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const uint32_t x0 = w ? s.v[2 * u][0].y : s.v[2 * u][0].x, x1 = w ? s.v[2 * u][1].y : s.v[2 * u][1].x;
        const uint32_t y0 = w ? s.v[2 * u + 1][0].y : s.v[2 * u + 1][0].x,
                       y1 = w ? s.v[2 * u + 1][1].y : s.v[2 * u + 1][1].x;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t v0[4], v1[4];
          unpack4(__byte_perm(x0, x1, half ? 0x7632 : 0x5410), S0, a0, b0, v0);
          unpack4(__byte_perm(y0, y1, half ? 0x7632 : 0x5410), S1, a1, b1, v1);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            mma_f16(o[8 * w + 4 * half + j], ph[2 * u], pl[2 * u], ph[2 * u + 1], pl[2 * u + 1], v0[j], v1[j]);
        }
      }
    }
  }
  l += __shfl_xor_sync(kFull, l, 1);
  l += __shfl_xor_sync(kFull, l, 2);
#pragma unroll
  for (int j = 0; j < 16; ++j) {  // columns 2t, 2t + 1 of tile j are channels 16 (2t) + j and 16 (2t + 1) + j
    so[warp][g][32 * t + j] = o[j][0] + o[j][2];
    so[warp][g][32 * t + 16 + j] = o[j][1] + o[j][3];
  }
  if (t == 0) {
    sml[warp][g][0] = m;
    sml[warp][g][1] = l;
  }
  __syncthreads();
  for (int e = tid; e < nh * kDim; e += kThreads4) {
    const int h = e / kDim, d = e - h * kDim;
    float M = sml[0][h][0];
#pragma unroll
    for (int w = 1; w < kWarps4; ++w) M = fmaxf(M, sml[w][h][0]);
    float L = 0.f, O = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps4; ++w) {
      const float mw = sml[w][h][0], f = mw == -INFINITY ? 0.f : exp2f(mw - M);
      L += sml[w][h][1] * f;
      O += so[w][h][d] * f;
    }
    float* ph = part + (int64_t)h * a.nsplit * kPartStride;
    ph[4 + d] = O;
    if (d == 0) {
      ph[0] = M;
      ph[1] = L;
    }
  }
}

constexpr int kFinishThreads = 256;
constexpr int kFinishRows = 2048;  // rows whose weights a block adds up

// Blocks [0, G): merge the splits of one query head.  Blocks from G on: add
// a range of rows' weights, head by head in ascending order.
__global__ void __launch_bounds__(kFinishThreads) k_kv4_finish(Attend4Args a) {
  __shared__ float sM[16], sI[16];
  __shared__ float half_o[kDim];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int b = blockIdx.y / a.c.hkv, kvh = blockIdx.y - b * a.c.hkv;
  const int64_t len = kv4_len(a.c, b);
  const int64_t q0 = (int64_t)b * a.hq + kvh * a.g;
  const bool merge = (int)blockIdx.x < a.g;
  const int64_t r0 = ((int64_t)blockIdx.x - a.g) * kFinishRows;
  if (!merge && r0 >= len) return;
  for (int h = warp; h < a.g; h += kFinishThreads / 32) {
    if (merge && h != (int)blockIdx.x) continue;
    const float* ph = a.part + (q0 + h) * a.nsplit * kPartStride;
    float M = -INFINITY;
    for (int s = lane; s < a.nsplit; s += 32) {
      const float2 ml = *reinterpret_cast<const float2*>(ph + (int64_t)s * kPartStride);
      M = fmaxf(M, ml.x);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(kFull, M, off));
    float L = 0.f;
    for (int s = lane; s < a.nsplit; s += 32) {
      const float2 ml = *reinterpret_cast<const float2*>(ph + (int64_t)s * kPartStride);
      if (ml.y != 0.f) L += ml.y * exp2f(ml.x - M);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) L += __shfl_xor_sync(kFull, L, off);
    if (lane == 0) {
      sM[h] = M;
      sI[h] = L != 0.f ? 1.f / L : 0.f;
    }
  }
  __syncthreads();
  if (merge) {
    const int h = blockIdx.x, d = tid & (kDim - 1), part = tid >> 7;
    const float* ph = a.part + (q0 + h) * a.nsplit * kPartStride;
    const float M = sM[h];
    float o = 0.f;
#pragma unroll 8
    for (int s = part; s < a.nsplit; s += 2) {
      const float2 ml = *reinterpret_cast<const float2*>(ph + (int64_t)s * kPartStride);
      const float x = ph[(int64_t)s * kPartStride + 4 + d];  // not written by a split without rows
      if (ml.y != 0.f) o += x * exp2f(ml.x - M);
    }
    if (part == 1) half_o[d] = o;
    __syncthreads();
    if (part == 0) a.out[(q0 + h) * kDim + d] = __float2bfloat16_rn((o + half_o[d]) * sI[h]);
    return;
  }
  const int64_t r1 = min64(len, r0 + kFinishRows);
  float* w = a.c.w + (int64_t)blockIdx.y * a.c.rmax;
  const float* sc = a.scores + q0 * a.c.rmax;
  for (int64_t r = r0 + tid; r < r1; r += kFinishThreads) {
    float p = 0.f;
    for (int h = 0; h < a.g; ++h) p += exp2f(sc[h * a.c.rmax + r] - sM[h]) * sI[h];
    w[r] += p;
  }
}

}  // namespace

void kv4_splits(int64_t units, int64_t rmax, int sm_count, int* nsplit, int64_t* rows_per_split) {
  // about three blocks per SM over all (sequence, KV head, head group)s, at
  // least two steps of a block each
  const int64_t want = std::max<int64_t>(1, (3 * sm_count + units - 1) / units);
  const int64_t most = std::max<int64_t>(1, (rmax + 2 * kTile4 - 1) / (2 * kTile4));
  const int64_t n = std::min<int64_t>({want, most, 512});
  *rows_per_split = std::max<int64_t>(kTile4, ((rmax + n - 1) / n + kTile4 - 1) / kTile4 * kTile4);
  *nsplit = (int)std::max<int64_t>(1, (rmax + *rows_per_split - 1) / *rows_per_split);
}

cudaError_t launch_kv4_attend(const Attend4Args& a, cudaStream_t st) {
  const dim3 grid(a.nsplit, a.c.batch * a.c.hkv, (a.g + kHeads4 - 1) / kHeads4);
  cudaError_t e = launch_pdl(k_kv4_attend, grid, dim3(kThreads4), 0, st, a);
  if (e != cudaSuccess) return e;
  const int64_t rows = a.accumulate ? (a.c.rmax + kFinishRows - 1) / kFinishRows : 0;
  return launch_pdl(k_kv4_finish, dim3((unsigned)(a.g + rows), a.c.batch * a.c.hkv), dim3(kFinishThreads), 0, st, a);
}

}  // namespace paris
