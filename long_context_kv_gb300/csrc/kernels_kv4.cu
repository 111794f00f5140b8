// The cache in 4 bits: store and read.
//
// A row is 128 values in four groups of 32; S = max|x| / 7 rounded up to
// four significant bits and c = rint(x / S).  Both are defined so that they
// come out the same in any precision that holds the inputs: S has 4 bits and
// (c + 1/2) S at most 8, so which code a value gets is decided by an exact
// comparison except within float32's last bit.
#include <cuda_fp16.h>

#include "kv4_internal.cuh"

namespace paris {
namespace {

constexpr int kStoreThreads = 256;

__device__ __forceinline__ float clean4(float x) {
  return x == x ? fminf(fmaxf(x, -kLimit4), kLimit4) : 0.f;
}

// S of a group from its largest magnitude, and its stored byte.
__device__ __forceinline__ float group_scale(float amax, uint32_t& byte) {
  const float t = __fdiv_rn(amax, 7.f);
  if (t >= 6.103515625e-05f) {  // 2^-14: four bits are a half's top mantissa bits
    const uint32_t up = (__float_as_uint(t) + 0xFFFFFu) & ~0xFFFFFu;
    byte = (up >> 20) - 896u;
    return __uint_as_float(up);
  }
  const float n = ceilf(t * 131072.f);  // multiples of 2^-17
  byte = (uint32_t)n;
  return n * 7.62939453125e-06f;
}

// A thread's 16 channels of a row; a group is two threads.
struct RowF32 {
  float x[16];
};
struct RowBf16 {
  uint32_t w[8];
};

__device__ __forceinline__ void load_row(const void* p, int64_t e, RowF32& r) {
  const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + e);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 v = __ldg(q + i);
    r.x[4 * i] = v.x; r.x[4 * i + 1] = v.y; r.x[4 * i + 2] = v.z; r.x[4 * i + 3] = v.w;
  }
}
__device__ __forceinline__ void load_row(const void* p, int64_t e, RowBf16& r) {
  const uint4* q = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + e);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint4 v = __ldg(q + i);
    r.w[4 * i] = v.x; r.w[4 * i + 1] = v.y; r.w[4 * i + 2] = v.z; r.w[4 * i + 3] = v.w;
  }
}

// Codes and scale byte, any values.
__device__ __forceinline__ uint2 quantise(RowF32& r, uint32_t& byte) {
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    r.x[i] = clean4(r.x[i]);
    amax = fmaxf(amax, fabsf(r.x[i]));
  }
  amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 1));
  const float S = group_scale(amax, byte);
  uint32_t word[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float c = S > 0.f ? fminf(fmaxf(rintf(__fdiv_rn(r.x[i], S)), -7.f), 7.f) : 0.f;
    word[i >> 3] |= (uint32_t)((int)c + 8) << (4 * (i & 7));
  }
  return make_uint2(word[0], word[1]);
}

// The same of bf16 values, without divisions and in five operations a value.
//
// With A the largest value's 8-bit integer, A 2^e / 7 is on the grid of
// four-bit scales or at least 2^-11 of itself from it, so its product with an
// approximate 1 / 7, taken down by 2^-17, rounds up to the same scale.
//
// With X a value's 8-bit and s the scale's 4-bit integer, x / S = X 2^e / s is
// a tie or at least 2^-10 from one where it could round to 1..7; so x times an
// approximate 1 / S (off by 2^-20 at most), rounded to multiples of 2^-13 by
// an addition of 1536, is the tie exactly where x / S is, and on its side of it
// elsewhere.  The second addition rounds it to the integer c + 8 (8 is even:
// ties still go to even c) in the low bits of 1.5 2^23 + 8 + c; the shifted sum
// of eight of these, less the sum of what is above those bits, is a code word.
__device__ __forceinline__ uint2 quantise(RowBf16& r, uint32_t& byte) {
  uint32_t top = r.w[0] & 0x7fff7fffu;
#pragma unroll
  for (int i = 1; i < 8; ++i) top = __vmaxu2(top, r.w[i] & 0x7fff7fffu);
  uint32_t amax = max(top & 0xffffu, top >> 16);
  amax = max(amax, __shfl_xor_sync(kFull, amax, 1));
  if (__any_sync(kFull, amax > 0x44D2u)) {  // past 1680, infinities, NaN
    RowF32 f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      f.x[2 * i] = bf16_bits_to_float(r.w[i] & 0xffffu);
      f.x[2 * i + 1] = __uint_as_float(r.w[i] & 0xffff0000u);
    }
    return quantise(f, byte);
  }
  const float t = bf16_bits_to_float(amax) * (1.f / 7.f);
  const uint32_t up = (__float_as_uint(t) - 64u + 0xFFFFFu) & ~0xFFFFFu;
  const float small = ceilf(t * (131072.f * (1.f - 7.62939453125e-06f)));  // multiples of 2^-17
  const bool is_small = t < 6.1e-05f;  // below 2^-14, whose neighbours the 64 steps leave on its side
  byte = is_small ? (uint32_t)small : (up >> 20) - 896u;
  const float S = is_small ? small * 7.62939453125e-06f : __uint_as_float(up);
  float inv;
  asm("rcp.approx.ftz.f32 %0, %1;\n" : "=f"(inv) : "f"(S));
  if (S == 0.f) inv = 0.f;
  uint32_t word[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t x = 0;
#pragma unroll
    for (int i = 4 * h + 3; i >= 4 * h; --i) {
      // both values of the word at once
      uint32_t lo, hi;
      asm("{\n .reg .b64 v, f, m, a;\n mov.b64 v, {%2, %3};\n mov.b64 f, {%4, %4};\n mov.b64 m, {%5, %5};\n mov.b64 a, {%6, %6};\n"
          " fma.rn.f32x2 v, v, f, m;\n add.rn.f32x2 v, v, a;\n mov.b64 {%0, %1}, v;\n}\n"
          : "=r"(lo), "=r"(hi)
          : "r"(r.w[i] << 16), "r"(r.w[i] & 0xffff0000u), "f"(inv), "f"(1536.f), "f"(12582920.f - 1536.f));
      x = (x << 4) + hi;
      x = (x << 4) + lo;
    }
    word[h] = x - (0x4B400000u + 0xB4000000u + 0x40000000u);
  }
  return make_uint2(word[0], word[1]);
}

// Block: up to `tokens` tokens of one sequence.  Eight threads take the key
// and the value row of a (token, KV head), 16 channels each.  Bound by the
// read of k and v: the arithmetic (35 operations of a warp a row) stays below
// the memory's time.  32768 tokens of 8 KV heads in bf16 (134 MB read, 38
// written): 36.8 us from cold caches, 4.7 TB/s.
template <typename Row>
__global__ void __launch_bounds__(kStoreThreads, 5) k_kv4_store(StoreArgs a, int nblk, int tokens, uint32_t hkv_inv) {
  pdl_wait();
  pdl_trigger();
  const int b = blockIdx.x / nblk, blk = blockIdx.x - b * nblk;
  const int tid = threadIdx.x, l8 = tid & 7;
  const int hkv = a.c.hkv;
  int64_t start, len;
  seq_rows(a.cu, b, a.rows, start, len);
  len = min64(len, a.max_new);
  const int64_t old_len = kv4_len(a.c, b);
  const int64_t stored = min64(len, a.c.rmax - old_len);
  const int64_t t0 = (int64_t)blk * tokens;
  const int n = (int)max64(0, min64(tokens, stored - t0));
  const int32_t pos0 = a.c.next[b];
  const uint32_t items = n * hkv;
  const int64_t k0 = (a.cu ? 0 : b * a.ks.seq) + (start + t0) * a.ks.token + 16 * l8;
  const int64_t v0 = (a.cu ? 0 : b * a.vs.seq) + (start + t0) * a.vs.token + 16 * l8;
  const int64_t row0 = (int64_t)b * hkv * a.c.rmax + old_len + t0;
  // strides and max_rows fit 32 bits: offsets are one wide product each
  const uint32_t kt = (uint32_t)a.ks.token, kh = (uint32_t)a.ks.head, vt = (uint32_t)a.vs.token, vh = (uint32_t)a.vs.head;
  const uint32_t rmax = (uint32_t)a.c.rmax;
  for (uint32_t it0 = (tid >> 5) * 4; it0 < items; it0 += kStoreThreads / 8) {
    const uint32_t it = min(it0 + ((tid >> 3) & 3), items - 1);  // past the end the last again: the same is written twice
    const uint32_t tok = hkv == 1 ? it : __umulhi(it, hkv_inv), h = it - tok * hkv;
    Row k, v;
    load_row(a.k, k0 + (uint64_t)tok * kt + (uint64_t)h * kh, k);
    load_row(a.v, v0 + (uint64_t)tok * vt + (uint64_t)h * vh, v);
    float wt = 0.f;
    if (a.weights != nullptr && l8 == 2) wt = a.weights[(a.cu ? (int64_t)h * a.rows + start : ((int64_t)b * hkv + h) * a.rows) + t0 + tok];
    const int64_t row = row0 + (uint64_t)h * rmax + tok;
    uint32_t kb, vb;
    const uint2 kw = quantise(k, kb), vw = quantise(v, vb);
    reinterpret_cast<uint2*>(a.c.kc + row * kCode4)[l8] = kw;
    reinterpret_cast<uint2*>(a.c.vc + row * kCode4)[l8] = vw;
    // a row's four scale bytes: the even threads hold one of each
    uint32_t sw = (kb | vb << 16) << (l8 & 2 ? 8 : 0);
    sw |= __shfl_xor_sync(kFull, sw, 2);                    // k 0, 1 and v 0, 1; k 2, 3 and v 2, 3
    const uint32_t other = __shfl_xor_sync(kFull, sw, 4);
    if (l8 == 0) *reinterpret_cast<uint32_t*>(a.c.ks + row * kScale4) = (sw & 0xffffu) | other << 16;
    if (l8 == 4) *reinterpret_cast<uint32_t*>(a.c.vs + row * kScale4) = other >> 16 | (sw & 0xffff0000u);
    if (l8 == 6) a.c.pos[row] = pos0 + (int32_t)(t0 + tok);
    if (l8 == 2) a.c.w[row] = wt;
  }
  // the last block of the sequence to finish moves its length on: every
  // block has read the old one (and the counter wraps back to zero)
  __syncthreads();
  if (tid == 0) {
    __threadfence();
    if (atomicInc(&a.c.counters[b], (uint32_t)(nblk - 1)) == (uint32_t)(nblk - 1)) {
      a.c.lens[b] = (int32_t)(old_len + stored);
      a.c.next[b] = pos0 + (int32_t)stored;
      if (stored < len) atomicOr(a.c.status, kStatusNoRoom);
    }
  }
}

// Eight values of a code word as bf16, c S having at most 7 significant bits.
// A byte's two nibbles go into the mantissas of two halves 64 (64 + u / 16 and
// 64 + u), which a subtraction and a product with 16 S and S make exact.
__device__ __forceinline__ uint4 word_values(uint32_t w, uint32_t byte) {
  const __half S = __ushort_as_half((unsigned short)(byte << 7));
  const __half2 scale = __halves2half2(__hmul(S, __float2half(16.f)), S), off = __floats2half2_rn(64.5f, 72.f);
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t x = (__byte_perm(w, 0, 0x4040 | i | i << 8) & 0x00F0000Fu) | 0x54005400u;
    const float2 f = __half22float2(__hmul2(__hsub2(*reinterpret_cast<const __half2*>(&x), off), scale));
    o[i] = pack_bf16x2(f.x, f.y);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// 16 threads per row, 8 channels each, four rows at a time; blocks (rows,
// sequence x KV head).  Bound by the write of the values: 32768 rows of 8 KV
// heads (134 MB written, 36 read) take 28 us, 6.1 TB/s.
constexpr int kReadRows = 64;
__global__ void __launch_bounds__(256) k_kv4_read(Kv4 c, __nv_bfloat16* k_out, __nv_bfloat16* v_out, int64_t rows) {
  pdl_wait();
  pdl_trigger();
  const int l16 = threadIdx.x & 15;
  const int64_t bh = blockIdx.y, i0 = (int64_t)blockIdx.x * kReadRows + (threadIdx.x >> 4);
  const int64_t n = min64(rows, kv4_len(c, (int)(bh / c.hkv)));
  uint32_t kw[4], vw[4], ks[4], vs[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int64_t i = i0 + 16 * u, src = bh * c.rmax + i;
    if (i >= n) continue;
    kw[u] = *reinterpret_cast<const uint32_t*>(c.kc + src * kCode4 + 4 * l16);
    vw[u] = *reinterpret_cast<const uint32_t*>(c.vc + src * kCode4 + 4 * l16);
    ks[u] = c.ks[src * kScale4 + (l16 >> 2)];
    vs[u] = c.vs[src * kScale4 + (l16 >> 2)];
  }
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int64_t i = i0 + 16 * u, dst = (bh * rows + i) * kDim + 8 * l16;
    if (i >= n) continue;
    __stcs(reinterpret_cast<uint4*>(k_out + dst), word_values(kw[u], ks[u]));
    __stcs(reinterpret_cast<uint4*>(v_out + dst), word_values(vw[u], vs[u]));
  }
}

}  // namespace

cudaError_t launch_kv4_store(const StoreArgs& a, cudaStream_t st) {
  // 16 tokens a block, fewer where that leaves SMs without two blocks
  int tokens = 16;
  while (tokens > 1 && a.c.batch * ((a.max_new + tokens - 1) / tokens) < 2 * 152) tokens /= 2;
  // the division by hkv is a product: exact below 2^32 / hkv items
  while (tokens > 1 && (int64_t)tokens * a.c.hkv * a.c.hkv >= (int64_t)1 << 32) tokens /= 2;
  const int64_t nblk = max64(1, (a.max_new + tokens - 1) / tokens);
  if (nblk * a.c.batch > 0x7fffffff) return cudaErrorInvalidValue;
  const uint32_t inv = (uint32_t)(((uint64_t)1 << 32) / a.c.hkv + 1);
  const dim3 grid((unsigned)(nblk * a.c.batch));
  if (a.dtype == 1) return launch_pdl(k_kv4_store<RowBf16>, grid, dim3(kStoreThreads), 0, st, a, (int)nblk, tokens, inv);
  return launch_pdl(k_kv4_store<RowF32>, grid, dim3(kStoreThreads), 0, st, a, (int)nblk, tokens, inv);
}

cudaError_t launch_kv4_read(const Kv4& c, __nv_bfloat16* k_out, __nv_bfloat16* v_out, int64_t rows, cudaStream_t st) {
  const dim3 grid((unsigned)((rows + kReadRows - 1) / kReadRows), c.batch * c.hkv);
  return launch_pdl(k_kv4_read, grid, dim3(256), 0, st, c, k_out, v_out, rows);
}

}  // namespace paris
