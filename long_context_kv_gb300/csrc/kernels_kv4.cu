// The cache in 4 bits: store and read.
//
// A row is 128 values in four groups of 32; S = max|x| / 7 rounded up to
// four significant bits and c = rint(x / S).  Both are defined so that they
// come out the same in any precision that holds the inputs: S has 4 bits and
// (c + 1/2) S at most 8, so which code a value gets is decided by an exact
// comparison except within float32's last bit.
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

// Codes and scale byte of a thread's 8 channels (a group is 4 threads), any
// values.
__device__ __forceinline__ uint32_t quantise8(float (&x)[8], uint32_t& byte) {
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[i] = clean4(x[i]);
    amax = fmaxf(amax, fabsf(x[i]));
  }
  amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 1));
  amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 2));
  const float S = group_scale(amax, byte);
  uint32_t word = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float c = S > 0.f ? fminf(fmaxf(rintf(__fdiv_rn(x[i], S)), -7.f), 7.f) : 0.f;
    word |= (uint32_t)((int)c + 8) << (4 * i);
  }
  return word;
}

// The same of 8 bf16 values, five operations each.  With X the value's 8-bit
// and s the scale's 4-bit integer, x / S = X 2^e / s is a tie or at least
// 2^-10 from one where it could round to 1..7; so x times an approximate 1 / S
// (off by 2^-20 at most), rounded to multiples of 2^-13 by an addition of
// 1536, is the tie exactly where x / S is, and on its side of it elsewhere.
// The second addition rounds it to the integer c + 8 (8 is even: ties still
// go to even c) in the low bits of 1.5 2^23 + 8 + c; the shifted sum of the
// eight words, less the sum of what is above those bits, is the code word.
__device__ __forceinline__ uint32_t quantise8(uint4 v, uint32_t& byte) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t top = w[0] & 0x7fff7fffu;
#pragma unroll
  for (int i = 1; i < 4; ++i) top = __vmaxu2(top, w[i] & 0x7fff7fffu);
  uint32_t amax = max(top & 0xffffu, top >> 16);
  amax = max(amax, __shfl_xor_sync(kFull, amax, 1));
  amax = max(amax, __shfl_xor_sync(kFull, amax, 2));
  if (__any_sync(kFull, amax > 0x44D2u)) {  // past 1680, infinities, NaN
    float x[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = bf16_bits_to_float(w[i] & 0xffffu);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
    return quantise8(x, byte);
  }
  const float S = group_scale(bf16_bits_to_float(amax), byte);
  float inv;
  asm("rcp.approx.ftz.f32 %0, %1;\n" : "=f"(inv) : "f"(S));
  if (S == 0.f) inv = 0.f;
  uint32_t word = 0;
#pragma unroll
  for (int i = 3; i >= 0; --i) {
    const float hi = fmaf(__uint_as_float(w[i] & 0xffff0000u), inv, 1536.f) + (12582920.f - 1536.f);
    const float lo = fmaf(__uint_as_float(w[i] << 16), inv, 1536.f) + (12582920.f - 1536.f);
    word = (word << 4) + __float_as_uint(hi);
    word = (word << 4) + __float_as_uint(lo);
  }
  return word - (0x4B400000u + 0xB4000000u + 0x40000000u);
}

__device__ __forceinline__ void load8(const void* p, int64_t e, uint4& v) {
  v = __ldcs(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + e));
}
struct Eight {
  float x[8];
};
__device__ __forceinline__ void load8(const void* p, int64_t e, Eight& v) {
  const float4 a = __ldcs(reinterpret_cast<const float4*>(static_cast<const float*>(p) + e));
  const float4 b = __ldcs(reinterpret_cast<const float4*>(static_cast<const float*>(p) + e + 4));
  v.x[0] = a.x; v.x[1] = a.y; v.x[2] = a.z; v.x[3] = a.w;
  v.x[4] = b.x; v.x[5] = b.y; v.x[6] = b.z; v.x[7] = b.w;
}
__device__ __forceinline__ uint32_t quantise8(Eight& v, uint32_t& byte) { return quantise8(v.x, byte); }

// Block: up to `tokens` tokens of one sequence.  16 threads take the key and
// the value row of a (token, KV head), 8 channels each, two such pairs at a
// time.  Bound by the read of k and v: four 16-byte loads a thread are in
// flight, and the arithmetic is kept below the memory's time.
template <typename V>
__global__ void __launch_bounds__(kStoreThreads) k_kv4_store(StoreArgs a, int nblk, int tokens, uint32_t hkv_inv) {
  pdl_wait();
  pdl_trigger();
  const int b = blockIdx.x / nblk, blk = blockIdx.x - b * nblk;
  const int tid = threadIdx.x, lane = tid & 31, l16 = tid & 15;
  const int hkv = a.c.hkv;
  int64_t start, len;
  seq_rows(a.cu, b, a.rows, start, len);
  len = min64(len, a.max_new);
  const int64_t old_len = kv4_len(a.c, b);
  const int64_t stored = min64(len, a.c.rmax - old_len);
  const int64_t t0 = (int64_t)blk * tokens;
  const int n = (int)max64(0, min64(tokens, stored - t0));
  const int32_t pos0 = a.c.next[b];
  const int items = n * hkv;
  const int64_t seq_k = a.cu ? 0 : b * a.ks.seq, seq_v = a.cu ? 0 : b * a.vs.seq;
  for (int it0 = (tid >> 5) * 2; it0 < items; it0 += 2 * (kStoreThreads / 16)) {
    V x[2][2];
    int tok[2], h[2];
    bool active[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int it = it0 + u * (kStoreThreads / 16) + (lane >> 4);
      active[u] = it < items;
      tok[u] = hkv == 1 ? it : (int)__umulhi((uint32_t)it, hkv_inv);
      h[u] = it - tok[u] * hkv;
      if (!active[u]) tok[u] = h[u] = 0;  // read again, and dropped
      const int64_t r = start + t0 + tok[u];
      load8(a.k, seq_k + r * a.ks.token + h[u] * a.ks.head + 8 * l16, x[u][0]);
      load8(a.v, seq_v + r * a.vs.token + h[u] * a.vs.head + 8 * l16, x[u][1]);
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int64_t row = ((int64_t)b * hkv + h[u]) * a.c.rmax + old_len + t0 + tok[u];
      uint32_t sw[2];
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        uint32_t byte;
        const uint32_t word = quantise8(x[u][kv], byte);
        sw[kv] = byte << (8 * (l16 >> 2));
        sw[kv] |= __shfl_xor_sync(kFull, sw[kv], 4);
        sw[kv] |= __shfl_xor_sync(kFull, sw[kv], 8);
        if (active[u]) *reinterpret_cast<uint32_t*>((kv ? a.c.vc : a.c.kc) + row * kCode4 + 4 * l16) = word;
      }
      if (!active[u]) continue;
      if (l16 == 0) *reinterpret_cast<uint32_t*>(a.c.ks + row * kScale4) = sw[0];
      if (l16 == 4) *reinterpret_cast<uint32_t*>(a.c.vs + row * kScale4) = sw[1];
      if (l16 == 8) a.c.pos[row] = pos0 + (int32_t)(t0 + tok[u]);
      if (l16 == 12) {
        const int64_t wrow = (a.cu ? (int64_t)h[u] * a.rows + start : ((int64_t)b * hkv + h[u]) * a.rows) + t0 + tok[u];
        a.c.w[row] = a.weights ? a.weights[wrow] : 0.f;
      }
    }
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

// Eight values of a code word as bf16: c S has at most 7 significant bits.
__device__ __forceinline__ uint4 word_values(uint32_t w, float S) {
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float lo = (float)((int)((w >> (8 * i)) & 15u) - 8) * S;
    const float hi = (float)((int)((w >> (8 * i + 4)) & 15u) - 8) * S;
    o[i] = pack_bf16x2(lo, hi);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

__device__ __forceinline__ float scale_value(uint32_t byte) {
  return __half2float(__ushort_as_half((unsigned short)(byte << 7)));
}

// 16 threads per row, 8 channels each; row index over [batch * Hkv][rows].
__global__ void __launch_bounds__(256) k_kv4_read(Kv4 c, __nv_bfloat16* k_out, __nv_bfloat16* v_out, int64_t rows,
                                                  int64_t total) {
  pdl_wait();
  pdl_trigger();
  const int l16 = threadIdx.x & 15;
  const int64_t step = (int64_t)gridDim.x * (blockDim.x / 16);
  for (int64_t r = (int64_t)blockIdx.x * (blockDim.x / 16) + (threadIdx.x >> 4); r < total; r += step) {
    const int64_t bh = r / rows, i = r - bh * rows;
    if (i >= kv4_len(c, (int)(bh / c.hkv))) continue;
    const int64_t src = bh * c.rmax + i;
    const uint32_t kw = *reinterpret_cast<const uint32_t*>(c.kc + src * kCode4 + 4 * l16);
    const uint32_t vw = *reinterpret_cast<const uint32_t*>(c.vc + src * kCode4 + 4 * l16);
    const float sk = scale_value(c.ks[src * kScale4 + (l16 >> 2)]), sv = scale_value(c.vs[src * kScale4 + (l16 >> 2)]);
    __stcs(reinterpret_cast<uint4*>(k_out + r * kDim + 8 * l16), word_values(kw, sk));
    __stcs(reinterpret_cast<uint4*>(v_out + r * kDim + 8 * l16), word_values(vw, sv));
  }
}

}  // namespace

cudaError_t launch_kv4_store(const StoreArgs& a, cudaStream_t st) {
  // 16 tokens a block, fewer where that leaves SMs without four blocks
  int tokens = 16;
  while (tokens > 1 && a.c.batch * ((a.max_new + tokens - 1) / tokens) < 4 * 152) tokens /= 2;
  const int64_t nblk = max64(1, (a.max_new + tokens - 1) / tokens);
  if (nblk * a.c.batch > 0x7fffffff) return cudaErrorInvalidValue;
  // exact for the at most 16 hkv items of a block
  const uint32_t inv = (uint32_t)(((uint64_t)1 << 32) / a.c.hkv + 1);
  const dim3 grid((unsigned)(nblk * a.c.batch));
  if (a.dtype == 1) return launch_pdl(k_kv4_store<uint4>, grid, dim3(kStoreThreads), 0, st, a, (int)nblk, tokens, inv);
  return launch_pdl(k_kv4_store<Eight>, grid, dim3(kStoreThreads), 0, st, a, (int)nblk, tokens, inv);
}

cudaError_t launch_kv4_read(const Kv4& c, __nv_bfloat16* k_out, __nv_bfloat16* v_out, int64_t rows, cudaStream_t st) {
  const int64_t total = (int64_t)c.batch * c.hkv * rows;
  const int64_t blocks = min64((total + 15) / 16, 152 * 16);
  return launch_pdl(k_kv4_read, dim3((unsigned)max64(1, blocks)), dim3(256), 0, st, c, k_out, v_out, rows, total);
}

}  // namespace paris
