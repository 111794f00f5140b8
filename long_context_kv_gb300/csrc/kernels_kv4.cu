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
constexpr int kStoreTokens = 16;  // tokens of one sequence per block

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

// Block: kStoreTokens tokens of one sequence, keys then values.  16 threads
// take a row, 8 channels (16 bytes of bf16) each; a group is 4 threads.
__global__ void __launch_bounds__(kStoreThreads) k_kv4_store(StoreArgs a, int nblk) {
  pdl_wait();
  pdl_trigger();
  const int b = blockIdx.x / nblk, blk = blockIdx.x - b * nblk;
  const int tid = threadIdx.x, lane = tid & 31, l16 = tid & 15;
  const int hkv = a.c.hkv;
  int64_t start, len;
  seq_rows(a.cu, b, a.rows, start, len);
  len = min64(len, a.max_new);
  const int64_t old_len = kv4_len(a.c, b);
  const int64_t room = a.c.rmax - old_len;
  const int64_t stored = min64(len, room);
  const int64_t t0 = (int64_t)blk * kStoreTokens;
  const int n = (int)max64(0, min64(kStoreTokens, stored - t0));
  const int32_t pos0 = a.c.next[b];
  const int items = n * hkv * 2;
  for (int it0 = (tid >> 5) * 2; it0 < items; it0 += kStoreThreads / 16) {
    const int it = it0 + (lane >> 4);
    const bool active = it < items;
    const bool is_v = it >= n * hkv;
    const int r = is_v ? it - n * hkv : it;
    const int tok = r / hkv, h = r - tok * hkv;
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = 0.f;
    if (active) {
      const Strides& s = is_v ? a.vs : a.ks;
      const int64_t e = (a.cu ? 0 : b * s.seq) + (start + t0 + tok) * s.token + h * s.head + 8 * l16;
      const void* p = is_v ? a.v : a.k;
      if (a.dtype == 1) {
        const uint4 u = __ldcs(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + e));
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[2 * i] = bf16_bits_to_float(w[i] & 0xffffu);
          x[2 * i + 1] = bf16_bits_to_float(w[i] >> 16);
        }
      } else {
        const float4 u = __ldcs(reinterpret_cast<const float4*>(static_cast<const float*>(p) + e));
        const float4 w = __ldcs(reinterpret_cast<const float4*>(static_cast<const float*>(p) + e + 4));
        x[0] = u.x; x[1] = u.y; x[2] = u.z; x[3] = u.w;
        x[4] = w.x; x[5] = w.y; x[6] = w.z; x[7] = w.w;
      }
    }
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[i] = clean4(x[i]);
      amax = fmaxf(amax, fabsf(x[i]));
    }
    amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 2));
    uint32_t byte;
    const float S = group_scale(amax, byte);
    uint32_t word = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float c = S > 0.f ? fminf(fmaxf(rintf(__fdiv_rn(x[i], S)), -7.f), 7.f) : 0.f;
      word |= (uint32_t)((int)c + 8) << (4 * i);
    }
    uint32_t sw = byte << (8 * (l16 >> 2));
    sw |= __shfl_xor_sync(kFull, sw, 4);
    sw |= __shfl_xor_sync(kFull, sw, 8);
    if (active) {
      const int64_t row = ((int64_t)b * hkv + h) * a.c.rmax + old_len + t0 + tok;
      *reinterpret_cast<uint32_t*>((is_v ? a.c.vc : a.c.kc) + row * kCode4 + 4 * l16) = word;
      if (l16 == 0) *reinterpret_cast<uint32_t*>((is_v ? a.c.vs : a.c.ks) + row * kScale4) = sw;
      if (!is_v && l16 == 1) a.c.pos[row] = pos0 + (int32_t)(t0 + tok);
      if (!is_v && l16 == 2) {
        const int64_t wrow = a.cu ? (int64_t)h * a.rows + start + t0 + tok : ((int64_t)b * hkv + h) * a.rows + t0 + tok;
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
  const int64_t nblk = max64(1, (a.max_new + kStoreTokens - 1) / kStoreTokens);
  if (nblk * a.c.batch > 0x7fffffff) return cudaErrorInvalidValue;
  return launch_pdl(k_kv4_store, dim3((unsigned)(nblk * a.c.batch)), dim3(kStoreThreads), 0, st, a, (int)nblk);
}

cudaError_t launch_kv4_read(const Kv4& c, __nv_bfloat16* k_out, __nv_bfloat16* v_out, int64_t rows, cudaStream_t st) {
  const int64_t total = (int64_t)c.batch * c.hkv * rows;
  const int64_t blocks = min64((total + 15) / 16, 152 * 16);
  return launch_pdl(k_kv4_read, dim3((unsigned)max64(1, blocks)), dim3(256), 0, st, c, k_out, v_out, rows, total);
}

}  // namespace paris
