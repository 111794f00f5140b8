// The paged cache: growing sequences, storing rows and reading them back.
#include <cuda_fp16.h>

#include <type_traits>

#include "paged_device.cuh"

namespace paris {
namespace {

// One block: what every sequence needs, where its pages begin among the free
// ones (a scan), and then the free pages in ascending order, each of which
// finds its sequence in the scanned numbers.  Bound by latency: the lengths,
// a scan, and only when pages are needed the bits, 32768 pages at a time: 3 to
// 4.5 us in a replayed graph, 10 from cold caches.
__global__ void __launch_bounds__(kPlanThreads) k_paged_grow(Paged c, const int32_t* tokens) {
  __shared__ uint32_t first[kMaxPagedSeqs + 1];  // number of a sequence's first new page
  __shared__ int pages[kMaxPagedSeqs];           // that it had
  __shared__ uint32_t tmp[33];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, cap = paged_cap(c);
  const uint32_t n_free = (uint32_t)max(c.n_pages - max(c.n_used[0], 0), 0);
  const uint32_t bits = first_bits(c);
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
      pages[s] = have;
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
  const uint32_t found = take_free(c, taken, bits, tmp, [&](uint32_t r, int page) {
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
    c.table[(int64_t)s * c.width + pages[s] + (r - first[s])] = page;
    c.refs[page] = 1;
  });
  if (found < taken) {  // n_used and free_bits do not agree: rows without a page are not there
    for (int i = tid; i < c.n_seqs; i += kPlanThreads) {
      const int most = (int)min64((int64_t)(pages[i] + (int)(min(first[i + 1], found) - min(first[i], found))) << c.shift, cap);
      if (c.lens[i] > most) c.lens[i] = most;
    }
    if (tid == 0) atomicOr(c.status, kStatusNoRoom);
  }
  if (tid == 0) c.n_used[0] = c.n_pages - (int)(n_free - found);
}

constexpr int kRowThreads = 256;
// Eight threads take a row, 16 channels each: eight from 8 l on and the same of
// the row's other half, so that a load or store of theirs is contiguous (16 in a
// row each: reading 7422 tokens of 8 heads 14.0 -> 17.2 us).
constexpr int kRowItems = kRowThreads / 8;

__device__ __forceinline__ float clean8(float x) {
  constexpr float lim = 1152921504606846976.f;  // 2^60
  return x == x ? fminf(fmaxf(x, -lim), lim) : 0.f;
}

// 16 channels of a row, as they are in memory.
template <bool kF32>
struct Raw16 {
  uint4 w[kF32 ? 4 : 2];
};

template <bool kF32>
__device__ __forceinline__ Raw16<kF32> load_raw(const uint8_t* p, int64_t e) {
  Raw16<kF32> r;
  const uint4* q = reinterpret_cast<const uint4*>(p + e * (kF32 ? 4 : 2));
#pragma unroll
  for (int i = 0; i < (kF32 ? 4 : 2); ++i) r.w[i] = __ldg(q + (kF32 ? i / 2 * 16 + i % 2 : 8 * i));
  return r;
}

template <bool kF32>
__device__ __forceinline__ void floats(const Raw16<kF32>& r, float (&x)[16]) {
#pragma unroll
  for (int i = 0; i < (kF32 ? 4 : 2); ++i) {
    const uint32_t u[4] = {r.w[i].x, r.w[i].y, r.w[i].z, r.w[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (kF32) {
        x[4 * i + j] = __uint_as_float(u[j]);
      } else {
        x[8 * i + 2 * j] = bf16_bits_to_float(u[j] & 0xffffu);
        x[8 * i + 2 * j + 1] = __uint_as_float(u[j] & 0xffff0000u);
      }
    }
  }
}

// A row's 16 channels into its page; its eight threads are neighbours.
template <bool kF32, bool kE4m3>
__device__ __forceinline__ void store_row(const Raw16<kF32>& r, uint8_t* dst, uint8_t* scale, int l8) {
  float x[16];
  if constexpr (!kE4m3) {
    uint4* to = reinterpret_cast<uint4*>(dst) + l8;
    if constexpr (!kF32) {
      to[0] = r.w[0];
      to[8] = r.w[1];
    } else {
      floats(r, x);
#pragma unroll
      for (int i = 0; i < 2; ++i)
        to[8 * i] = make_uint4(pack_bf16x2(x[8 * i], x[8 * i + 1]), pack_bf16x2(x[8 * i + 2], x[8 * i + 3]),
                           pack_bf16x2(x[8 * i + 4], x[8 * i + 5]), pack_bf16x2(x[8 * i + 6], x[8 * i + 7]));
    }
  } else {
    // the largest magnitude's bits; of bf16 values two at a time
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < (kF32 ? 4 : 2); ++i) {
      const uint32_t u[4] = {r.w[i].x, r.w[i].y, r.w[i].z, r.w[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) top = kF32 ? max(top, u[j] & 0x7fffffffu) : __vmaxu2(top, u[j] & 0x7fff7fffu);
    }
    if (!kF32) top = max(top << 16, top & 0xffff0000u);
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) top = max(top, __shfl_xor_sync(kFull, top, o));
    floats(r, x);
    if (__any_sync(kFull, top > 0x5D800000u)) {  // past 2^60, infinities, NaN
      float amax = 0.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        x[i] = clean8(x[i]);
        amax = fmaxf(amax, fabsf(x[i]));
      }
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, o));
      top = __float_as_uint(amax);
    }
    // the smallest e with amax <= 1.75 2^(8 + e): from its exponent, one more past the mantissa of 1.75
    const int e = min(max((int)((top + 0x1fffffu) >> 23) - 127 - 8, -60), 52);
    const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint16_t lo, hi;
      asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(lo) : "f"(x[4 * i + 1] * inv), "f"(x[4 * i] * inv));
      asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(hi) : "f"(x[4 * i + 3] * inv), "f"(x[4 * i + 2] * inv));
      w[i] = (uint32_t)lo | (uint32_t)hi << 16;
    }
    reinterpret_cast<uint2*>(dst)[l8] = make_uint2(w[0], w[1]);
    reinterpret_cast<uint2*>(dst)[l8 + 8] = make_uint2(w[2], w[3]);
    if (l8 == 0) *scale = (uint8_t)(e + 127);
  }
}

// What the threads of a store or read call go through: `tokens` tokens of one
// sequence a block, eight threads a row.
struct RowWalk {
  int b, l8, items;
  int row0;          // the block's first row in the sequence
  int64_t k0, v0;    // its elements next to the cache
  __device__ __forceinline__ RowWalk(const PagedRows& a, int nblk, int tokens, int first, int rows_left) {
    b = blockIdx.x / nblk;
    l8 = threadIdx.x & 7;
    int64_t start, len;
    seq_rows(a.cu, b, a.rows, start, len);
    len = min64(min64(len, a.max_rows), rows_left);
    const int64_t t0 = (int64_t)(blockIdx.x - b * nblk) * tokens;
    items = (int)max64(0, min64(tokens, len - t0)) * a.c.hkv;
    row0 = first + (int)t0;
    k0 = (a.cu ? 0 : b * a.ks.seq) + (start + t0) * a.ks.token + 8 * l8;
    v0 = (a.cu ? 0 : b * a.vs.seq) + (start + t0) * a.vs.token + 8 * l8;
  }
};

// A block: up to `tokens` tokens of one sequence.  Rows of heads are contiguous
// on the side of the prompt, rows of tokens on that of the pages: full lines
// on both.  Bound by the bytes: 32768 tokens of 8 KV heads into 8 bits (134 MB
// read, 68 written) 33 us, 6.1 TB/s; two maxima at a time instead of one by one
// and eight threads a row instead of 16 took it there from 50.
template <bool kF32, bool kE4m3>
__global__ void __launch_bounds__(kRowThreads) k_paged_store(PagedRows a, int nblk, int tokens, uint32_t hkv_inv) {
  pdl_wait();
  pdl_trigger();
  const int first = min(max(a.c.starts[blockIdx.x / nblk], 0), paged_cap(a.c));
  const RowWalk w(a, nblk, tokens, first, max(paged_len(a.c, blockIdx.x / nblk) - first, 0));
  uint8_t* kp = a.c.k + a.layer * a.c.sk.layer;
  uint8_t* vp = a.c.v + a.layer * a.c.sv.layer;
  const int mask = (1 << a.c.shift) - 1;
  // a warp's four items together, as its lanes exchange; past the end the last one again (the same is written twice)
  for (int it0 = (threadIdx.x >> 5) * 4; it0 < w.items; it0 += kRowItems) {
    const uint32_t it = min(it0 + (int)((threadIdx.x >> 3) & 3), w.items - 1);
    const uint32_t tok = a.c.hkv == 1 ? it : __umulhi(it, hkv_inv), h = it - tok * a.c.hkv;
    const Raw16<kF32> k = load_raw<kF32>(a.k, w.k0 + (int64_t)tok * a.ks.token + (int64_t)h * a.ks.head);
    const Raw16<kF32> v = load_raw<kF32>(a.v, w.v0 + (int64_t)tok * a.vs.token + (int64_t)h * a.vs.head);
    const int r = w.row0 + (int)tok, page = page_at(a.c, w.b, r >> a.c.shift), pr = r & mask;
    const int64_t s = kE4m3 ? scale_at(a.c, a.layer, page, h, pr) : 0;
    store_row<kF32, kE4m3>(k, kp + page * a.c.sk.page + h * a.c.sk.head + pr * a.c.sk.row, a.c.ks + s, w.l8);
    store_row<kF32, kE4m3>(v, vp + page * a.c.sv.page + h * a.c.sv.head + pr * a.c.sv.row, a.c.vs + s, w.l8);
  }
}

// 16 codes as bf16 values, exact.
__device__ __forceinline__ void values16(const uint2 (&codes)[2], uint32_t byte, uint4* to) {
  const float S = __uint_as_float(byte << 23);
  const uint32_t u[4] = {codes[0].x, codes[0].y, codes[1].x, codes[1].y};
  uint32_t o[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t h = i & 1 ? e4m3_hi(u[i >> 1]) : e4m3_lo(u[i >> 1]);
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    o[i] = pack_bf16x2(f.x * S, f.y * S);
  }
  __stcs(to, make_uint4(o[0], o[1], o[2], o[3]));
  __stcs(to + 8, make_uint4(o[4], o[5], o[6], o[7]));
}

// The way back, laid out as k_paged_store; two items under way at a time.  The
// same rows: 30 us, 6.7 TB/s.
template <bool kE4m3>
__global__ void __launch_bounds__(kRowThreads) k_paged_read(PagedRows a, int nblk, int tokens, uint32_t hkv_inv) {
  pdl_wait();
  pdl_trigger();
  const RowWalk w(a, nblk, tokens, 0, paged_len(a.c, blockIdx.x / nblk));
  const uint8_t* kp = a.c.k + a.layer * a.c.sk.layer;
  const uint8_t* vp = a.c.v + a.layer * a.c.sv.layer;
  const int mask = (1 << a.c.shift) - 1;
  using Piece = std::conditional_t<kE4m3, uint2, uint4>;
  for (int it0 = threadIdx.x >> 3; it0 < w.items; it0 += 2 * kRowItems) {
    Piece x[2][2], y[2][2];
    uint32_t kb[2], vb[2], tok[2], h[2];
    int page[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const uint32_t it = it0 + u * kRowItems;
      tok[u] = a.c.hkv == 1 ? it : __umulhi(it, hkv_inv);
      h[u] = it - tok[u] * a.c.hkv;
      if ((int)it < w.items) page[u] = page_at(a.c, w.b, (w.row0 + (int)tok[u]) >> a.c.shift);
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      if (it0 + u * kRowItems >= w.items) continue;
      const int pr = (w.row0 + (int)tok[u]) & mask;
      const Piece* k = reinterpret_cast<const Piece*>(kp + page[u] * a.c.sk.page + h[u] * a.c.sk.head + pr * a.c.sk.row) + w.l8;
      const Piece* v = reinterpret_cast<const Piece*>(vp + page[u] * a.c.sv.page + h[u] * a.c.sv.head + pr * a.c.sv.row) + w.l8;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        x[u][i] = k[8 * i];
        y[u][i] = v[8 * i];
      }
      if constexpr (kE4m3) {
        const int64_t s = scale_at(a.c, a.layer, page[u], h[u], pr);
        kb[u] = a.c.ks[s];
        vb[u] = a.c.vs[s];
      }
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      if (it0 + u * kRowItems >= w.items) continue;
      uint4* k = reinterpret_cast<uint4*>(a.k + 2 * (w.k0 + (int64_t)tok[u] * a.ks.token + (int64_t)h[u] * a.ks.head));
      uint4* v = reinterpret_cast<uint4*>(a.v + 2 * (w.v0 + (int64_t)tok[u] * a.vs.token + (int64_t)h[u] * a.vs.head));
      if constexpr (kE4m3) {
        values16(x[u], kb[u], k);
        values16(y[u], vb[u], v);
      } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          __stcs(k + 8 * i, x[u][i]);
          __stcs(v + 8 * i, y[u][i]);
        }
      }
    }
  }
}

// The grid of a store or read call: 16 tokens a block, fewer where that leaves
// SMs without two blocks, and more past 2^18 blocks: packed rows of many
// sequences and no better limit than all of them, so that nearly all blocks are
// empty, which takes 1.1 ns each (a million rows of 4096 sequences: 289 -> 0.99
// ms, with their own limit 0.94; where no block is empty, 8 million rows of one
// sequence, 923 -> 917 us).
constexpr int64_t kRowBlocks = 1 << 18;
struct RowGrid {
  int tokens = 16, nblk;
  uint32_t hkv_inv;  // the division by hkv is a product: exact below 2^32 / hkv items
  dim3 grid;
  bool fits;
  RowGrid(const PagedRows& a, int sm_count) {
    while (tokens > 1 && a.c.n_seqs * ((a.max_rows + tokens - 1) / tokens) < 2 * sm_count) tokens /= 2;
    while (tokens > 1 && (int64_t)tokens * a.c.hkv * a.c.hkv >= (int64_t)1 << 32) tokens /= 2;
    while ((a.max_rows + tokens - 1) / tokens * a.c.n_seqs > kRowBlocks && (int64_t)2 * tokens * a.c.hkv * a.c.hkv < (int64_t)1 << 32) tokens *= 2;
    const int64_t n = (a.max_rows + tokens - 1) / tokens;
    fits = n * a.c.n_seqs <= 0x7fffffff;
    nblk = (int)n;
    grid = dim3((unsigned)(n * a.c.n_seqs));
    hkv_inv = (uint32_t)(((uint64_t)1 << 32) / a.c.hkv + 1);
  }
};

}  // namespace

cudaError_t launch_paged_grow(const Paged& c, const int32_t* tokens, cudaStream_t st) {
  return launch_pdl(k_paged_grow, dim3(1), dim3(kPlanThreads), 0, st, c, tokens);
}

cudaError_t launch_paged_store(const PagedRows& a, int sm_count, cudaStream_t st) {
  const RowGrid g(a, sm_count);
  if (!g.fits) return cudaErrorInvalidValue;
  const dim3 block(kRowThreads);
  if (a.dtype == 1)
    return a.c.e4m3 ? launch_pdl(k_paged_store<false, true>, g.grid, block, 0, st, a, g.nblk, g.tokens, g.hkv_inv)
                    : launch_pdl(k_paged_store<false, false>, g.grid, block, 0, st, a, g.nblk, g.tokens, g.hkv_inv);
  return a.c.e4m3 ? launch_pdl(k_paged_store<true, true>, g.grid, block, 0, st, a, g.nblk, g.tokens, g.hkv_inv)
                  : launch_pdl(k_paged_store<true, false>, g.grid, block, 0, st, a, g.nblk, g.tokens, g.hkv_inv);
}

cudaError_t launch_paged_read(const PagedRows& a, int sm_count, cudaStream_t st) {
  const RowGrid g(a, sm_count);
  if (!g.fits) return cudaErrorInvalidValue;
  const dim3 block(kRowThreads);
  return a.c.e4m3 ? launch_pdl(k_paged_read<true>, g.grid, block, 0, st, a, g.nblk, g.tokens, g.hkv_inv)
                  : launch_pdl(k_paged_read<false>, g.grid, block, 0, st, a, g.nblk, g.tokens, g.hkv_inv);
}

}  // namespace paris
