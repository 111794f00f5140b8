// The paged cache: growing sequences, storing rows and reading them back.
#include <cuda_fp16.h>

#include "paged_device.cuh"

namespace paris {
namespace {

// One block: what every sequence needs, where its pages begin among the free
// ones (a scan), and then the free pages in ascending order, each of which
// finds its sequence in the scanned numbers.  Bound by latency: the lengths,
// a scan, and only when pages are needed the bits, 32768 pages at a time.
__global__ void __launch_bounds__(kPlanThreads) k_paged_grow(Paged c, const int32_t* tokens) {
  __shared__ uint32_t first[kMaxPagedSeqs + 1];  // number of a sequence's first new page
  __shared__ uint32_t tmp[33];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, cap = paged_cap(c);
  const uint32_t n_free = (uint32_t)max(c.n_pages - max(c.n_used[0], 0), 0);
  uint32_t taken = 0;
  bool short_of = false;
  for (int s0 = 0; s0 < c.n_seqs; s0 += kPlanThreads) {
    const int s = s0 + tid;
    int len = 0, want = 0, have = 0;
    uint32_t need = 0, total;
    if (s < c.n_seqs) {
      len = paged_len(c, s);
      want = max(tokens[s], 0);
      const int fits = min(want, cap - len);
      short_of |= fits < want;
      want = fits;
      have = pages_of(c, len);
      need = min((uint32_t)(pages_of(c, len + want) - have), n_free);
    }
    // needs are at most 2^21 each: their sum fits, and more than is free counts as that
    const uint32_t at = min(block_excl_scan(need, tmp, &total) + taken, n_free);
    if (s < c.n_seqs) {
      const uint32_t got = min(need, n_free - at);
      first[s] = at;
      const int room = (int)min64(((int64_t)have + got) << c.shift, cap) - len;
      short_of |= room < want;
      c.starts[s] = len;
      c.lens[s] = len + min(want, room);
    }
    taken = min(taken + total, n_free);
  }
  if (tid == 0) first[c.n_seqs] = taken;
  if (short_of) atomicOr(c.status, kStatusNoRoom);
  if (taken == 0) return;
  __syncthreads();
  int s = -1;
  take_free(c, taken, tmp, [&](uint32_t r, int page) {
    if (s < 0) {  // the last sequence that begins at or before r, of those with a page
      int lo = 0, hi = c.n_seqs - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (first[mid] <= r) lo = mid;
        else hi = mid - 1;
      }
      s = lo;
    }
    while (first[s + 1] <= r) ++s;
    c.table[(int64_t)s * c.width + pages_of(c, c.starts[s]) + (r - first[s])] = page;
    c.refs[page] = 1;
  });
  if (tid == 0) c.n_used[0] = max(c.n_used[0], 0) + (int)taken;
}

constexpr int kRowThreads = 256;

__device__ __forceinline__ float clean8(float x) {
  constexpr float lim = 1152921504606846976.f;  // 2^60
  return x == x ? fminf(fmaxf(x, -lim), lim) : 0.f;
}

// Eight channels of a row, as they are in memory.
template <bool kF32>
struct Raw8 {
  uint4 w[kF32 ? 2 : 1];
};

template <bool kF32>
__device__ __forceinline__ Raw8<kF32> load_raw(const uint8_t* p, int64_t e) {
  Raw8<kF32> r;
  const uint4* q = reinterpret_cast<const uint4*>(p + e * (kF32 ? 4 : 2));
  r.w[0] = __ldg(q);
  if constexpr (kF32) r.w[1] = __ldg(q + 1);
  return r;
}

__device__ __forceinline__ void unpack_bf16(const uint4& w, float (&x)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = bf16_bits_to_float(u[i] & 0xffffu);
    x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}

template <bool kF32>
__device__ __forceinline__ void floats(const Raw8<kF32>& r, float (&x)[8]) {
  if constexpr (kF32) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      x[4 * i] = __uint_as_float(r.w[i].x);
      x[4 * i + 1] = __uint_as_float(r.w[i].y);
      x[4 * i + 2] = __uint_as_float(r.w[i].z);
      x[4 * i + 3] = __uint_as_float(r.w[i].w);
    }
  } else {
    unpack_bf16(r.w[0], x);
  }
}

// A row's eight channels into its page; 16 lanes hold a row.
template <bool kF32, bool kE4m3>
__device__ __forceinline__ void store_row(const Raw8<kF32>& r, uint8_t* dst, uint8_t* scale, int l16) {
  if constexpr (!kE4m3) {
    if constexpr (!kF32) {
      reinterpret_cast<uint4*>(dst)[l16] = r.w[0];
    } else {
      float x[8];
      floats(r, x);
      reinterpret_cast<uint4*>(dst)[l16] = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                                                      pack_bf16x2(x[6], x[7]));
    }
  } else {
    float x[8], amax = 0.f;
    floats(r, x);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[i] = clean8(x[i]);
      amax = fmaxf(amax, fabsf(x[i]));
    }
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, o));
    // the smallest e with amax <= 1.75 2^(8 + e): from its exponent, one more past the mantissa of 1.75
    const uint32_t u = __float_as_uint(amax);
    const int e = min(max((int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0), -60), 52);
    const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint16_t lo, hi;
      asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(lo) : "f"(x[4 * i + 1] * inv), "f"(x[4 * i] * inv));
      asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(hi) : "f"(x[4 * i + 3] * inv), "f"(x[4 * i + 2] * inv));
      w[i] = (uint32_t)lo | (uint32_t)hi << 16;
    }
    reinterpret_cast<uint2*>(dst)[l16] = make_uint2(w[0], w[1]);
    if (l16 == 0) *scale = (uint8_t)(e + 127);
  }
}

// A block: up to `tokens` tokens of one sequence, 16 lanes a row of 128
// channels, two (token, KV head) a warp.  Rows of heads are contiguous on the
// side of the prompt, rows of tokens on that of the pages: full lines on both.
// Bound by the bytes.
template <bool kF32, bool kE4m3>
__global__ void __launch_bounds__(kRowThreads) k_paged_store(PagedRows a, int nblk, int tokens) {
  pdl_wait();
  pdl_trigger();
  const int b = blockIdx.x / nblk, blk = blockIdx.x - b * nblk;
  const int l16 = threadIdx.x & 15, hkv = a.c.hkv;
  int64_t start, len;
  seq_rows(a.cu, b, a.rows, start, len);
  const int row0 = min(max(a.c.starts[b], 0), paged_cap(a.c));
  len = min64(min64(len, a.max_rows), max(paged_len(a.c, b) - row0, 0));
  const int64_t t0 = (int64_t)blk * tokens;
  const int n = (int)max64(0, min64(tokens, len - t0));
  const int items = n * hkv;
  const int64_t k0 = (a.cu ? 0 : b * a.ks.seq) + (start + t0) * a.ks.token + 8 * l16;
  const int64_t v0 = (a.cu ? 0 : b * a.vs.seq) + (start + t0) * a.vs.token + 8 * l16;
  uint8_t* kp = a.c.k + a.layer * a.c.sk.layer;
  uint8_t* vp = a.c.v + a.layer * a.c.sv.layer;
  const int mask = (1 << a.c.shift) - 1;
  // a warp's two items together, as its lanes exchange; past the end the last one again (the same is written twice)
  for (int it0 = (threadIdx.x >> 5) * 2; it0 < items; it0 += kRowThreads / 16) {
    const int it = min(it0 + ((threadIdx.x >> 4) & 1), items - 1);
    const int tok = it / hkv, h = it - tok * hkv;
    const Raw8<kF32> k = load_raw<kF32>(a.k, k0 + tok * a.ks.token + h * a.ks.head);
    const Raw8<kF32> v = load_raw<kF32>(a.v, v0 + tok * a.vs.token + h * a.vs.head);
    const int r = row0 + (int)t0 + tok, page = page_at(a.c, b, r >> a.c.shift), pr = r & mask;
    const int64_t s = kE4m3 ? scale_at(a.c, a.layer, page, h, pr) : 0;
    store_row<kF32, kE4m3>(k, kp + page * a.c.sk.page + h * a.c.sk.head + pr * a.c.sk.row, a.c.ks + s, l16);
    store_row<kF32, kE4m3>(v, vp + page * a.c.sv.page + h * a.c.sv.head + pr * a.c.sv.row, a.c.vs + s, l16);
  }
}

__device__ __forceinline__ uint4 values8(uint2 codes, uint32_t byte) {
  const float S = __uint_as_float(byte << 23);
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t w = i < 2 ? codes.x : codes.y, h = i & 1 ? e4m3_hi(w) : e4m3_lo(w);
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    o[i] = pack_bf16x2(f.x * S, f.y * S);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// The way back, laid out as k_paged_store.
template <bool kE4m3>
__global__ void __launch_bounds__(kRowThreads) k_paged_read(PagedRows a, int nblk, int tokens) {
  pdl_wait();
  pdl_trigger();
  const int b = blockIdx.x / nblk, blk = blockIdx.x - b * nblk;
  const int l16 = threadIdx.x & 15, hkv = a.c.hkv;
  int64_t start, len;
  seq_rows(a.cu, b, a.rows, start, len);
  len = min64(min64(len, a.max_rows), paged_len(a.c, b));
  const int64_t t0 = (int64_t)blk * tokens;
  const int n = (int)max64(0, min64(tokens, len - t0));
  const int64_t k0 = (a.cu ? 0 : b * a.ks.seq) + (start + t0) * a.ks.token + 8 * l16;
  const int64_t v0 = (a.cu ? 0 : b * a.vs.seq) + (start + t0) * a.vs.token + 8 * l16;
  const uint8_t* kp = a.c.k + a.layer * a.c.sk.layer;
  const uint8_t* vp = a.c.v + a.layer * a.c.sv.layer;
  const int mask = (1 << a.c.shift) - 1;
  for (int it = threadIdx.x >> 4; it < n * hkv; it += kRowThreads / 16) {
    const int tok = it / hkv, h = it - tok * hkv;
    const int r = (int)t0 + tok, page = page_at(a.c, b, r >> a.c.shift), pr = r & mask;
    const uint8_t* k = kp + page * a.c.sk.page + h * a.c.sk.head + pr * a.c.sk.row;
    const uint8_t* v = vp + page * a.c.sv.page + h * a.c.sv.head + pr * a.c.sv.row;
    uint4 x, y;
    if constexpr (kE4m3) {
      const int64_t s = scale_at(a.c, a.layer, page, h, pr);
      const uint2 kc = reinterpret_cast<const uint2*>(k)[l16], vc = reinterpret_cast<const uint2*>(v)[l16];
      const uint32_t kb = a.c.ks[s], vb = a.c.vs[s];
      x = values8(kc, kb);
      y = values8(vc, vb);
    } else {
      x = reinterpret_cast<const uint4*>(k)[l16];
      y = reinterpret_cast<const uint4*>(v)[l16];
    }
    __stcs(reinterpret_cast<uint4*>(a.k + 2 * (k0 + tok * a.ks.token + h * a.ks.head)), x);
    __stcs(reinterpret_cast<uint4*>(a.v + 2 * (v0 + tok * a.vs.token + h * a.vs.head)), y);
  }
}

// Tokens a block: 16, fewer where that leaves SMs without two blocks.
int block_tokens(const PagedRows& a) {
  int tokens = 16;
  while (tokens > 1 && a.c.n_seqs * ((a.max_rows + tokens - 1) / tokens) < 2 * 152) tokens /= 2;
  return tokens;
}

}  // namespace

cudaError_t launch_paged_grow(const Paged& c, const int32_t* tokens, cudaStream_t st) {
  return launch_pdl(k_paged_grow, dim3(1), dim3(kPlanThreads), 0, st, c, tokens);
}

cudaError_t launch_paged_store(const PagedRows& a, cudaStream_t st) {
  const int tokens = block_tokens(a);
  const int64_t nblk = (a.max_rows + tokens - 1) / tokens, blocks = nblk * a.c.n_seqs;
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  const dim3 grid((unsigned)blocks), block(kRowThreads);
  if (a.dtype == 1)
    return a.c.e4m3 ? launch_pdl(k_paged_store<false, true>, grid, block, 0, st, a, (int)nblk, tokens)
                    : launch_pdl(k_paged_store<false, false>, grid, block, 0, st, a, (int)nblk, tokens);
  return a.c.e4m3 ? launch_pdl(k_paged_store<true, true>, grid, block, 0, st, a, (int)nblk, tokens)
                  : launch_pdl(k_paged_store<true, false>, grid, block, 0, st, a, (int)nblk, tokens);
}

cudaError_t launch_paged_read(const PagedRows& a, cudaStream_t st) {
  const int tokens = block_tokens(a);
  const int64_t nblk = (a.max_rows + tokens - 1) / tokens, blocks = nblk * a.c.n_seqs;
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  const dim3 grid((unsigned)blocks), block(kRowThreads);
  return a.c.e4m3 ? launch_pdl(k_paged_read<true>, grid, block, 0, st, a, (int)nblk, tokens)
                  : launch_pdl(k_paged_read<false>, grid, block, 0, st, a, (int)nblk, tokens);
}

}  // namespace paris
