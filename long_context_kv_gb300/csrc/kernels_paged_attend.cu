// Attention of one new token over a paged cache.
//
// Bound by the read of the rows in use: 512 bytes for each row and KV head
// in bf16, 258 in 8 bits.  What that asks for:
//
// - All SMs read to the end.  The tiles of all sequences form one line, which
//   is cut into units within sequences: long ones in front, short ones in its
//   last quarter or third.  Blocks take (unit, KV head, head group) jobs from a queue,
//   since SMs differ by a third in what the memory gives them (equal parts of
//   131072 rows ended 72 to 104 us after the start).  A sequence of one unit
//   is done with its job; the units of others leave partial sums (maximum,
//   sum, unnormalised result), which a second kernel joins in their order
//   (k_paged_join, k_paged_join_many).  Which block has which job changes no
//   result.
// - Copies are always under way.  A warp takes steps of 8 KB of its own (16
//   bf16 rows of keys and values, or 32 in 8 bits) through a ring in shared
//   memory that TMA fills, two steps ahead and across the ends of sequences;
//   no warp waits for another but at those.  (Twelve warps an SM with two
//   steps each took 111.9 instead of 110.9 us for a ragged batch and 43.9
//   instead of 41.5 in 8 bits, a warp that copies for four others 113.7 and
//   70.)  The tensor maps' swizzle makes the reads below free of bank
//   conflicts, and their strides take any order of the pages' dimensions.
// - The arithmetic stays out of the way.  Both products have the cache's rows
//   on their M side, S^T = K Q^T and O^T = V^T P^T (m16n8k16, float32 sums), so
//   that the eight columns are what there are few of.  For up to four query
//   heads the columns hold each head twice, and P's upper and lower part; for
//   more, bf16 weights take a second product for their lower parts.  Values
//   of 8-bit rows are converted to halves, in which they are exact, and their
//   scales stay outside the products: a key row's multiplies its scores, a
//   value row's joins the exponent.  (The tensor pipe is 8 to 11 % busy: what
//   tcgen05 is faster at is not what is missing here, and it takes weights
//   through memory.)
//
// Weights are p = 2^(s - m) of base-2 scores, m a maximum so far that may lag
// by 2^8.  With a value row's scale 2^e, what enters the product with V is
// 2^(s + e - m), m the maximum of s + e, and the sum takes 2^-e of it.  m is kept
// as a row's own product and e, and both are subtracted before the scale, so
// that weights are right at any size of the scores.
//
// Measured: 131072 rows of 8 KV heads in bf16 82.8 us, 6.5 TB/s; 24 ragged
// sequences, 167K rows of 4 KV heads in 8 bits, 38.9 us, 4.4 TB/s.  Of those 39
// the rows take 24 at the memory's rate; the first of them are there after 3 to
// 5.5 us (lengths, pages, rows: one round trip after another), blocks end up to
// 3 us apart (a unit of four tiles takes 4), joining takes 5 with its launch, and
// the next call starts 2.5 later.
// A step of 32 8-bit rows is 0.9 us of a warp's time, hidden behind the copies
// but for the last one.  (Four more warps a block that do the copying, with
// registers moved from them to the others: 8-bit batch 38.2, long sequence 88.)
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
constexpr int kPgEntries = 512;  // of the line's table
constexpr uint32_t kPgMinUnit = 4;  // tiles (8-bit batch of 24: 44.1 us, with 3 46.0; one sequence of 128K rows the same)
// Where sequences can have no more tiles than this, each is one unit, and there
// is nothing to join (four of up to 300 rows: 8.0 -> 7.2 us; one of six tiles: 6.4 -> 6.6).
constexpr uint32_t kPgWhole = 6;
constexpr int kPgUnknown = -1;
constexpr int kPgSmem = 1024 + kPgWarps * kPgDepth * (kPgStage + kPgScale) + kPgOut + 16 * 16 * kPgWarps;

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
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
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
// Rows are read once, by one block of the call: they go first when the L2 makes
// room, so that tables, queries and partial sums stay.  Caches in turn, as the
// layers of a model come: 2 to 7% at every size (30 MB of rows 10.5 -> 9.8 us, in
// 8 bits 16.2 -> 15.4, 230 MB 45.6 -> 43.6).  Only one small cache that is read
// again and again loses (30 MB: 18.1 -> 19.1 us), since its rows would have stayed.
// With several head groups, which read the same rows, they have no such mark.
__device__ __forceinline__ uint64_t rows_policy(bool once) {
  uint64_t p;
  if (once) asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;\n" : "=l"(p));
  else asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;\n" : "=l"(p));
  return p;
}
__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2, int c3, uint32_t bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, {%2, %3, %4, %5}], [%6], "
      "%7;\n" ::"r"(dst),
      "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar), "l"(policy)
      : "memory");
}
__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2, int c3, int c4, uint32_t bar,
                                         uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, {%2, %3, %4, %5, %6}], "
      "[%7], %8;\n" ::"r"(dst),
      "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4), "r"(bar), "l"(policy)
      : "memory");
}

// A maximum: a row's product d and exponent e, for scores d qs + e.
struct PgMax {
  float d, e;
};
// How far x lies above y.
__device__ __forceinline__ float above(PgMax x, PgMax y, float qs) { return fmaf(x.d - y.d, qs, x.e - y.e); }

// Sums of bf16 rows that are not finite though the weights are: a value is not
// finite, also where the lower part of its weight is 0 and their product NaN, or
// the sum of large values passes float32's range before it is divided by the
// weights' sum.  (8-bit rows are at most 2^60.)
__device__ __forceinline__ bool not_finite(const float4& o, float sum) {
  return fmaf(o.x, 0.f, fmaf(o.y, 0.f, fmaf(o.z, 0.f, o.w * 0.f))) != 0.f && fabsf(sum) < INFINITY;
}
// Such a query head again by one warp, channels [c0, c1) of its result: 32 rows at
// a time, a lane a row for the scores, four channels a lane for the mean, to which
// every row adds its own weight of the whole: nothing passes the range that the
// mean does not.  A row whose weight is below 2^-118 of the largest adds nothing,
// whatever it holds: as where units and warps are joined, whose weights of up to
// 2^8 meet factors that are 0 below 2^-126.  Bound by latency: 4096 rows take 1.5
// ms, 131072 87.
__device__ __forceinline__ void paged_row(const PagedAttendArgs& a, int s, int h, int c0, int c1) {
  const int lane = threadIdx.x & 31, kvh = h / a.g, mask = (1 << a.c.shift) - 1, channel = 4 * lane;
  const int len = paged_len(a.c, s), first = a.window > 0 ? max(len - a.window, 0) : 0;
  const uint4* q = reinterpret_cast<const uint4*>(a.q + ((int64_t)s * a.hq + h) * kDim);
  const uint8_t* kp = a.c.k + a.layer * a.c.sk.layer + kvh * a.c.sk.head;
  const uint8_t* vp = a.c.v + a.layer * a.c.sv.layer + kvh * a.c.sv.head;
  auto score = [&](int r) {
    const uint4* row = reinterpret_cast<const uint4*>(kp + page_at(a.c, s, r >> a.c.shift) * a.c.sk.page + (r & mask) * a.c.sk.row);
    float d = 0.f;
#pragma unroll 2
    for (int i = 0; i < kDim / 8; ++i) {
      const uint4 x = row[i], y = __ldg(q + i);
      const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        d = fmaf(bf16_bits_to_float(xs[j] & 0xffffu), bf16_bits_to_float(ys[j] & 0xffffu), d);
        d = fmaf(__uint_as_float(xs[j] & 0xffff0000u), __uint_as_float(ys[j] & 0xffff0000u), d);
      }
    }
    return d;
  };
  float m = -INFINITY, l = 0.f;
  for (int r = first + lane; r < len; r += 32) {
    const float d = score(r), top = fmaxf(m, d);
    if (top == -INFINITY) continue;
    l = l * ex2((m - top) * kScaleLog2) + ex2((d - top) * kScaleLog2);
    m = top;
  }
  float top = m;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, off));
  l = m > -INFINITY ? l * ex2((m - top) * kScaleLog2) : 0.f;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) l += __shfl_xor_sync(kFull, l, off);
  const float inv = 1.f / l;
  float o[4] = {0.f, 0.f, 0.f, 0.f};
  for (int r0 = first; r0 < len; r0 += 32) {
    const float w = r0 + lane < len ? ex2((score(r0 + lane) - top) * kScaleLog2) : 0.f;
    for (uint32_t some = __ballot_sync(kFull, !(w < 0x1p-118f)); some != 0; some &= some - 1) {
      const int j = __ffs(some) - 1, r = r0 + j;
      const float p = __shfl_sync(kFull, w, j) * inv;
      float v[4];
      load4(vp + page_at(a.c, s, r >> a.c.shift) * a.c.sv.page + (r & mask) * a.c.sv.row, 1, channel, v);
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = fmaf(p, v[i], o[i]);
    }
  }
  if (channel >= c0 && channel < c1)
    *reinterpret_cast<uint2*>(a.out + ((int64_t)s * a.hq + h) * kDim + channel) = make_uint2(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]));
}

// The same if what is there, in those channels, is not finite.  A whole warp.
__device__ __forceinline__ void row_again(const PagedAttendArgs& a, int s, int h, int c0, int c1) {
  const int channel = 4 * (threadIdx.x & 31);
  const uint2 y = *reinterpret_cast<const uint2*>(a.out + ((int64_t)s * a.hq + h) * kDim + channel);
  auto special = [](uint32_t x) { return (x & 0x7f80u) == 0x7f80u || (x & 0x7f800000u) == 0x7f800000u; };
  if (__any_sync(kFull, channel >= c0 && channel < c1 && (special(y.x) || special(y.y)))) paged_row(a, s, h, c0, c1);
}
// At the end of a joining kernel, whose blocks each had every gridDim.x-th of the
// (split sequence, head, part of the channels): its own results that are not
// finite, and (once the kernel in front has left word in counts[2], which the last
// block that is done takes back) those of sequences of one unit, spread over the
// blocks.
__device__ __forceinline__ void rows_again(const PagedAttendArgs& a, int parts, bool mine, bool others) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5, splits = (int)min(a.counts[1], (uint32_t)a.max_splits);
  if (mine) {
    __syncthreads();
    for (int64_t b = blockIdx.x + (int64_t)warp * gridDim.x; b < (int64_t)splits * a.hq * parts; b += (int64_t)warps * gridDim.x) {
      const int64_t it = b / parts;
      const int u = (int)(it / a.hq), c0 = (int)(b - it * parts) * (kDim / parts);
      row_again(a, a.splits[u].s, (int)(it - (int64_t)u * a.hq), c0, c0 + kDim / parts);
    }
  }
  if (!others) return;
  for (int64_t it = (int64_t)blockIdx.x * warps + warp; it < (int64_t)a.c.n_seqs * a.hq; it += (int64_t)gridDim.x * warps) {
    const int s = (int)(it / a.hq);
    bool split = false;  // not those: their blocks have written them, or will
    for (int i = lane; i < splits; i += 32) split |= a.splits[i].s == s;
    if (!__any_sync(kFull, split)) row_again(a, s, (int)(it - (int64_t)s * a.hq), 0, kDim);
  }
  __syncthreads();
  if (threadIdx.x == 0 && atomicAdd(&a.counts[3], 1u) == gridDim.x - 1) a.counts[2] = a.counts[3] = 0;
}

// What a joining block has to look at again, in shared memory: a register more in
// its loop, or a call there, cost 2 to 3% of the whole attention (64 sequences of
// 2000 rows 85.3 -> 87.0 us, 256 of 700 122.5 -> 126; so 84.7 and 122.1).
struct AgainFlags {
  uint32_t mine, others;
  template <bool kE4m3>
  static __device__ __forceinline__ void start(AgainFlags& f, const PagedAttendArgs& a) {
    if (kE4m3 || threadIdx.x != 0) return;
    f.mine = 0;
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;\n" ::"r"(smem_u32(&f.others)), "l"(a.counts + 2) : "memory");
  }
  __device__ __forceinline__ void finish(const PagedAttendArgs& a, int parts) {
    asm volatile("cp.async.wait_all;\n" ::: "memory");
    __syncthreads();
    if ((mine | others) != 0) rows_again(a, parts, mine != 0, others != 0);
  }
};

// How the line of all tiles is cut: units of at most `large` tiles in front of
// `border`, of at most `small` behind it; sequences of at most `small` whole.
struct PgCut {
  uint32_t border, large, small;
};
// total tiles of seqs sequences, heads jobs a unit, for so many blocks.  Where
// units of a few tiles give no more jobs than blocks, all are of that size.
// Otherwise two large units a block, and four small ones to even out what they
// took.  (Two or three small ones end later: a ragged batch of 24 104 -> 111
// us.)  Where the memory alone bounds the call, SMs differ most in what they
// get, and the large units leave a third to the small ones instead of a quarter:
// the same batch 109.5 -> 106.7 us, twice its rows 220 -> 210, a decode step of
// 30 sequences 59.7 -> 57.8; but with 16 heads 41.0 -> 43.9 and in 8 bits 39.4
// -> 41.1, where small units cost a warp's time.  Of few sequences one large
// unit: they are cut into as many as there are blocks (one sequence of 128K rows
// 89.4 -> 88.0 us, in 8 bits 60.9 -> 57.5; a ragged batch would have blocks with
// two of them, 112 -> 131).
__device__ __forceinline__ PgCut pg_cut(uint32_t total, uint32_t seqs, uint32_t heads, uint32_t blocks, bool whole, bool memory) {
  PgCut c;
  c.border = total - total / 4;
  c.small = c.large = kPgWhole;
  if (whole) return c;
  const uint32_t each = blocks / heads;
  if (each > seqs) {  // a sequence's last unit may not be full
    c.small = c.large = max(1u, (total + each - seqs - 1) / (each - seqs));
    if (c.small <= kPgMinUnit) return c;
  }
  const float share = (float)total * (float)heads / (float)blocks;
  const bool few = 16 * seqs <= each;
  memory &= !few;
  if (memory) c.border = (uint32_t)((float)total * 0.66f);
  c.small = max(kPgMinUnit, (uint32_t)ceilf(share * (memory ? 0.085f : 0.0625f)));
  c.large = max(c.small, (uint32_t)ceilf(share * (few ? 0.75f : memory ? 0.33f : 0.375f)));
  return c;
}
// A sequence's units: in front of the border and behind it.
struct PgUnits {
  uint32_t front, nf, nb;  // tiles in front, units in front and behind
};
__device__ __forceinline__ PgUnits pg_units(const PgCut& c, uint32_t at, uint32_t tiles) {
  PgUnits u = {tiles, tiles > 0 ? 1u : 0u, 0};
  if (tiles > c.small) {
    u.front = at < c.border ? min(c.border - at, tiles) : 0u;
    u.nf = (u.front + c.large - 1) / c.large;
    u.nb = (tiles - u.front + c.small - 1) / c.small;
  }
  return u;
}
// Units, and units of sequences with several of them in the upper half.
__device__ __forceinline__ uint32_t pg_count(const PgUnits& u) {
  const uint32_t n = u.nf + u.nb;
  return n > 1 ? n | n << 16 : n;
}

// A unit of one KV head and head group.
struct PgJob {
  int s, len, first, base;
  uint32_t t0, t1;  // tiles of the sequence
  int slot;         // of its partial sums, or -1: it is the whole sequence
  int kvh, h0;
};

struct PgShared {
  uint64_t bar[kPgWarps][kPgDepth];
  float4 ml[kPgWarps][16];   // maximum (product, exponent), sum, scale of a head's scores
  uint2 line[kPgEntries];    // tiles and units (pg_count) in front of every `group`-th sequence
  uint32_t tmp[33];
  int used[kPgWarps];        // sequences with rows
  int next[2];               // the job after the present one, or kPgUnknown
  uint32_t gave_up;
};

// kWhole: no sequence can have several units, the jobs are gridDim.x apart and no
// kernel follows (of its own, four sequences of up to 300 rows 7.4 -> 7.0 us).
template <bool kE4m3, int kHeads, bool kWhole>
__global__ void __launch_bounds__(kPgThreads, 2)
    k_paged_attend(const __grid_constant__ PagedAttendArgs a, const __grid_constant__ CUtensorMap km, const __grid_constant__ CUtensorMap vm) {
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
    for (int i = 0; i < kPgDepth; ++i) bar_init(bar0 + 8 * i, kE4m3 ? 33 : 1);
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  if (tid == 0) {
    sh.gave_up = 0;
    sh.next[0] = sh.next[1] = kPgUnknown;
    asm volatile("prefetch.tensormap [%0];\n" ::"l"(&km) : "memory");
    asm volatile("prefetch.tensormap [%0];\n" ::"l"(&vm) : "memory");
  }
  volatile uint32_t* gave_up = &sh.gave_up;
  const uint32_t heads = (uint32_t)(a.c.hkv * a.groups), blocks = gridDim.x;
  pdl_wait();
  pdl_trigger();

  // The line: up to 32 sequences are a lane each of every warp; more of them are
  // in a table, of whose entries a thread has up to four in a row.
  const bool few = a.c.n_seqs <= 32;
  const int group = (a.c.n_seqs + kPgEntries - 1) / kPgEntries, entries = (a.c.n_seqs + group - 1) / group;
  PgCut cut;
  uint32_t jobs, my_at = 0, my_begin = 0;
  PgSeq my_q = {0, 0, 0, 0};
  if (few) {
    if (lane < a.c.n_seqs) my_q = pg_seq<kE4m3>(a, lane);
    __syncthreads();  // the barriers are there
    const uint32_t seqs = __popc(__ballot_sync(kFull, my_q.tiles > 0)), end = warp_incl_scan(my_q.tiles, lane);
    cut = pg_cut(__shfl_sync(kFull, end, 31), seqs, heads, blocks, kWhole, !kE4m3 && kHeads < 16);
    my_at = end - my_q.tiles;
    const uint32_t c = pg_count(pg_units(cut, my_at, my_q.tiles)), units = warp_incl_scan(c, lane);
    my_begin = units - c;
    jobs = (__shfl_sync(kFull, units, 31) & 0xffffu) * heads;
    if (!kWhole && blockIdx.x == 0 && warp == 0) {
      const uint32_t several = __ballot_sync(kFull, c >> 16 != 0);
      if (c >> 16 != 0) a.splits[__popc(several & ((1u << lane) - 1u))] = PgSplit{lane, (int)(my_begin >> 16), (int)(c >> 16), 0};
      if (lane == 0) a.counts[1] = __popc(several);
    }
  } else {
    const int per = (entries + kPgThreads - 1) / kPgThreads * group;
    const int s0 = min(tid * per, a.c.n_seqs), s1 = min(s0 + per, a.c.n_seqs);
    const uint32_t only = s0 < s1 ? pg_seq<kE4m3>(a, s0).tiles : 0u;  // of a thread's first sequence
    auto tiles_of = [&](int s) { return s == s0 ? only : pg_seq<kE4m3>(a, s).tiles; };
    uint32_t mine = 0, total;
    int used = 0;
    for (int s = s0; s < s1; ++s) {
      const uint32_t n = tiles_of(s);
      mine += n;
      used += n > 0 ? 1 : 0;
    }
    used = __reduce_add_sync(kFull, used);
    if (lane == 0) sh.used[warp] = used;
    const uint32_t at0 = block_excl_scan(mine, sh.tmp, &total);
    cut = pg_cut(total, sh.used[0] + sh.used[1] + sh.used[2] + sh.used[3], heads, blocks, kWhole, !kE4m3 && kHeads < 16);
    uint32_t at = at0, count = 0, several = 0;
    for (int s = s0; s < s1; ++s) {
      const uint32_t n = tiles_of(s), c = pg_count(pg_units(cut, at, n));
      count += c;
      several += c >> 16 != 0 ? 1u : 0u;
      at += n;
    }
    uint32_t units, splits = 0, split = 0;
    uint32_t unit = block_excl_scan(count, sh.tmp, &units);
    jobs = (units & 0xffffu) * heads;
    if (!kWhole && blockIdx.x == 0) {
      split = block_excl_scan(several, sh.tmp, &splits);
      if (tid == 0) a.counts[1] = splits;
    }
    at = at0;
    for (int s = s0; s < s1; ++s) {
      if (s % group == 0) sh.line[s / group] = make_uint2(at, unit);
      if (per == 1 && blockIdx.x != 0) break;
      const uint32_t n = tiles_of(s), c = pg_count(pg_units(cut, at, n));
      if (!kWhole && blockIdx.x == 0 && c >> 16 != 0) a.splits[split++] = PgSplit{s, (int)(unit >> 16), (int)(c >> 16), 0};
      unit += c;
      at += n;
    }
    __syncthreads();
  }

  // a job's unit and sequence
  auto find = [&](uint32_t job) {
    const uint32_t unit = job / heads, head = job - unit * heads;
    PgJob r;
    r.kvh = (int)head / a.groups;
    r.h0 = ((int)head - r.kvh * a.groups) * kHeads;
    PgSeq q;
    uint32_t at, begin;
    if (few) {  // the last lane that begins at or before the unit
      r.s = __popc(__ballot_sync(kFull, lane < a.c.n_seqs && (my_begin & 0xffffu) <= unit)) - 1;
      q.len = __shfl_sync(kFull, my_q.len, r.s);
      q.first = __shfl_sync(kFull, my_q.first, r.s);
      q.base = __shfl_sync(kFull, my_q.base, r.s);
      q.tiles = __shfl_sync(kFull, my_q.tiles, r.s);
      at = __shfl_sync(kFull, my_at, r.s);
      begin = __shfl_sync(kFull, my_begin, r.s);
    } else {  // likewise the entry, and a sequence of its `group`
      int e = -1;
      for (int e0 = 0; e0 < entries; e0 += 32) {
        const int n = __popc(__ballot_sync(kFull, e0 + lane < entries && (sh.line[e0 + lane].y & 0xffffu) <= unit));
        e += n;
        if (n < 32) break;
      }
      at = sh.line[e].x;
      begin = sh.line[e].y;
      r.s = e * group;
      q = pg_seq<kE4m3>(a, r.s);
      while (r.s + 1 < a.c.n_seqs) {
        const uint32_t count = pg_count(pg_units(cut, at, q.tiles));
        if (unit - (begin & 0xffffu) < (count & 0xffffu)) break;
        at += q.tiles;
        begin += count;
        q = pg_seq<kE4m3>(a, ++r.s);
      }
    }
    const PgUnits u = pg_units(cut, at, q.tiles);
    const uint32_t i = unit - (begin & 0xffffu), n = u.nf + u.nb;  // the sequence's i-th unit
    const bool back = i >= u.nf;
    const uint32_t size = back ? cut.small : cut.large, from = back ? u.front : 0u, to = back || n == 1 ? q.tiles : u.front;
    r.len = q.len;
    r.first = q.first;
    r.base = q.base;
    r.t0 = from + (back ? i - u.nf : i) * size;
    r.t1 = n == 1 ? to : min(r.t0 + size, to);
    r.slot = n > 1 ? (int)min((begin >> 16) + i, (uint32_t)a.slots - 1u) : -1;
    return r;
  };

  // What the warp copies next: a step of the present job, or of the next one
  // once that is known.
  const bool busy = blockIdx.x < jobs;
  uint32_t job = blockIdx.x;
  PgJob cur = find(busy ? job : 0u), nxt = cur;
  int k = 0;  // jobs that the block has had
  bool in_next = false, stop = false;  // stop: a wait gave up, nothing more is copied
  // The steps left of the job that is copied, and the place of the next one
  // among 32 that were looked up, a lane each: its page, its first row there in
  // 16s, whether it has rows (and, in 8 bits and pages of 16 rows, its second
  // page if that has rows).  As little as possible is left for a step's own
  // copy, which all of the warp waits for.
  constexpr uint32_t kPageMask = (1u << kMaxPagesLog) - 1u, kHas = 1u << 31;
  int p_left = 0, p_i = 0, p_row = 0;
  uint32_t step0 = 0, step1 = 0;
  const uint8_t* p_scales = nullptr;  // of the job's layer and head: a lane's keys' or values', four rows
  const uint32_t p_pitch = (uint32_t)a.c.hkv << a.c.shift;
  auto look_up = [&](const PgJob& p) {
    const int row = p_row + lane * G::kTile, j = row >> a.c.shift;
    const int32_t* t = a.c.table + (int64_t)p.s * a.c.width;
    p_i = 0;
    p_row += 32 * G::kTile;
    step0 = step1 = 0;
    if (lane < p_left && row < p.len) {
      step0 = kHas | (uint32_t)(row & ((1 << a.c.shift) - 1)) >> 4 << kMaxPagesLog | (uint32_t)clamp_page(a.c, t[j]);
      if (kE4m3 && a.c.shift == 4 && row + 16 < p.len) step1 = kHas | (uint32_t)clamp_page(a.c, t[j + 1]);
    }
  };
  auto enter = [&](const PgJob& j) {
    p_row = j.base + (int)j.t0 * G::kTile + warp * kRows;
    p_left = (int)(j.t1 - j.t0);
    if (kE4m3) p_scales = (lane < 8 ? a.c.ks : a.c.vs) + scale_at(a.c, a.layer, 0, j.kvh, 4 * (lane & 7));
    look_up(j);
  };
  uint32_t ahead = 0, p_stage = 0, c_stage = 0, c_parity = 0;  // steps that are copied and not yet taken
  const uint64_t policy = rows_policy(a.groups == 1);
  auto copy_next = [&]() {
    if (ahead >= kPgDepth) return;
    if (p_left == 0) {
      if (in_next) return;
      const int j = __shfl_sync(kFull, *(volatile int*)&sh.next[(k + 1) & 1], 0);
      if (j == kPgUnknown || (uint32_t)j >= jobs) return;
      nxt = find(j);
      in_next = true;
      enter(nxt);
    }
    if (p_i == 32) look_up(in_next ? nxt : cur);
    const uint32_t w0 = __shfl_sync(kFull, step0, p_i), w1 = kE4m3 ? __shfl_sync(kFull, step1, p_i) : 0u;
    const int kvh = in_next ? nxt.kvh : cur.kvh;
    ++p_i;
    --p_left;
    if ((w0 & kHas) == 0 || stop) return;
    const int page = (int)(w0 & kPageMask), r = (int)(w0 >> kMaxPagesLog & 15u) << 4;
    const uint32_t dst = ring + p_stage * kPgStage, bar = bar0 + 8 * p_stage;
    if constexpr (!kE4m3) {
      if (elect()) {
        bar_expect(bar, kPgStage);
        load_box(dst, &km, 0, r, 0, kvh, page, bar, policy);
        load_box(dst + kPgStage / 2, &vm, 0, r, 0, kvh, page, bar, policy);
      }
    } else {
      // Pages of 16 rows: two, the second one if it has rows.  The scale bytes
      // go by the lanes, four rows each: as copies of their own they took as
      // much of the copy engine's time as the rows.
      const bool one = a.c.shift > 4, two = (w1 & kHas) != 0, upper = !one && (lane & 4) != 0;
      const int next = (int)(w1 & kPageMask);
      if (lane < 16 && (!upper || two)) {
        const uint8_t* e = p_scales + (uint64_t)(uint32_t)(upper ? next : page) * p_pitch + (upper ? -16 : r);
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;\n" ::"r"(smem_u32(scales) + p_stage * kPgScale + 4 * lane), "l"(e) : "memory");
      }
      asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];\n" ::"r"(bar) : "memory");
      if (elect()) {
        bar_expect(bar, one || two ? kPgStage : kPgStage / 2);
        load_box(dst, &km, 0, r, kvh, page, bar, policy);
        load_box(dst + kPgStage / 2, &vm, 0, r, kvh, page, bar, policy);
        if (two) {
          load_box(dst + 2048, &km, 0, 0, kvh, next, bar, policy);
          load_box(dst + kPgStage / 2 + 2048, &vm, 0, 0, kvh, next, bar, policy);
        }
      }
    }
    __syncwarp();
    p_stage = p_stage + 1 == kPgDepth ? 0 : p_stage + 1;
    ++ahead;
  };

  // a lane's places in a step's boxes (128 bytes a row, 16-byte pieces swizzled by the row)
  const uint32_t lrow = lane & 15, lhi = lane >> 4, lsw = lane & 7;

  // the queries' words: column g's head (of four: twice)
  uint32_t qw[kQ][8][2];
  auto load_queries = [&](const PgJob& j) {
    const int nh = min(kHeads, a.g - j.h0);
#pragma unroll
    for (int c = 0; c < kQ; ++c) {
      const int h = 8 * c + (kHeads == 4 ? g & 3 : g);
      const uint32_t* q = reinterpret_cast<const uint32_t*>(a.q + ((int64_t)j.s * a.hq + j.kvh * a.g + j.h0 + h) * kDim);
#pragma unroll
      for (int s = 0; s < 8; ++s) {
        if constexpr (!kE4m3) {
          qw[c][s][0] = h < nh ? __ldg(q + 8 * s + t) : 0u;
          qw[c][s][1] = h < nh ? __ldg(q + 8 * s + 4 + t) : 0u;
        } else {
          const uint2 u = h < nh ? __ldg(reinterpret_cast<const uint2*>(q + 8 * s) + t) : make_uint2(0, 0);
          qw[c][s][0] = u.x;
          qw[c][s][1] = u.y;
        }
      }
    }
  };
  if (busy) {
    enter(cur);
    load_queries(cur);
  }
  bool again = false;  // a sequence's result is not finite
  while (busy) {
#pragma unroll 1
    for (int i = 0; i < kPgDepth - 1 && !in_next && ahead < kPgDepth - 1; ++i) copy_next();
    // the job after this one: on its way while the first steps are computed
    int fetched = 0;
    bool pending = tid == 0;
    if (pending) fetched = (int)(kWhole ? job + blocks : blocks + atomicAdd(a.counts, 1u));
    const int kvh = cur.kvh, h0 = cur.h0, nh = min(kHeads, a.g - h0), qh0 = kvh * a.g + h0;

    uint32_t qf[kQ][8][2];
    float qs[kQ][2];  // of a thread's columns 2 t and 2 t + 1
#pragma unroll
    for (int c = 0; c < kQ; ++c) {
      if constexpr (!kE4m3) {
#pragma unroll
        for (int s = 0; s < 8; ++s) {
          qf[c][s][0] = qw[c][s][0];
          qf[c][s][1] = qw[c][s][1];
        }
        qs[c][0] = qs[c][1] = kScoreScale;
      } else {
        // as halves, scaled by a power of two to below 1; eight bits fit their eleven
        float amax = 0.f;
#pragma unroll
        for (int s = 0; s < 8; ++s)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            amax = fmaxf(amax, fmaxf(fabsf(bf16_bits_to_float(qw[c][s][i] & 0xffffu)), fabsf(__uint_as_float(qw[c][s][i] & 0xffff0000u))));
        amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 2));
        const int e = min(max((int)((__float_as_uint(amax) >> 23) & 255u) - 126, -100), 126);
        const float down = __uint_as_float((uint32_t)(127 - e) << 23), up = __uint_as_float((uint32_t)(127 + e) << 23) * kScoreScale;
#pragma unroll
        for (int s = 0; s < 8; ++s)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            qf[c][s][i] = pack_weights<true>(bf16_bits_to_float(qw[c][s][i] & 0xffffu) * down, __uint_as_float(qw[c][s][i] & 0xffff0000u) * down);
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
    for (uint32_t tile = cur.t0; tile < cur.t1; ++tile) {
      if (pending && tile != cur.t0) {
        *(volatile int*)&sh.next[(k + 1) & 1] = fetched;
        pending = false;
      }
      __syncwarp();
      copy_next();
      const int row0 = cur.base + (int)tile * G::kTile + warp * kRows;
      if (row0 >= cur.len || ahead == 0) continue;  // (nothing is copied any more after a wait that gave up)
      const uint32_t kst = ring + c_stage * kPgStage, vst = kst + kPgStage / 2;
      if (__any_sync(kFull, !bar_wait(bar0 + 8 * c_stage, c_parity, gave_up))) {
        stop = true;
        WaitLimit limit(now_ns());  // the copy ends before the block does
        while (!bar_try(bar0 + 8 * c_stage, c_parity) && !limit.over(now_ns())) {}
      }
      --ahead;
      const bool edge = row0 < cur.first || row0 + kRows > cur.len;
      if (edge) {
        // rows that do not count may hold anything, and 0 times NaN is NaN
        for (int r = lane >> 3; r < kRows; r += 4) {
          if (row0 + r >= cur.first && row0 + r < cur.len) continue;
          const uint32_t z = vst + r * 128 + 16 * (lane & 7);
          asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};\n" ::"r"(z), "r"(0) : "memory");
          if (!kE4m3) asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};\n" ::"r"(z + 2048), "r"(0) : "memory");
        }
        asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");  // before the next copy into the step's place
        __syncwarp();
      }

      // S^T: p[u][c][2 r + i] of row 16 u + 8 r + g, column 2 t + i
      float p[kU][kQ][4], p2[kU][kQ][4], ev[kU][2], inv[kU][2];  // p2: every second product, as they wait for one another
#pragma unroll
      for (int u = 0; u < kU; ++u) {
#pragma unroll
        for (int c = 0; c < kQ; ++c)
#pragma unroll
          for (int x = 0; x < 4; ++x) p[u][c][x] = p2[u][c][x] = 0.f;
        if constexpr (!kE4m3) {
#pragma unroll
          for (int s = 0; s < 8; ++s) {
            uint32_t f[4];
            ldsm4(f, kst + (s >> 2) * 2048 + lrow * 128 + (((2 * (s & 3) + lhi) ^ lsw) << 4));
#pragma unroll
            for (int c = 0; c < kQ; ++c) mma16<false>(s & 1 ? p2[u][c] : p[u][c], f[0], f[1], f[2], f[3], qf[c][s][0], qf[c][s][1]);
          }
#pragma unroll
          for (int c = 0; c < kQ; ++c)
#pragma unroll
            for (int x = 0; x < 4; ++x) p[u][c][x] += p2[u][c][x];
        } else {
#pragma unroll
          for (int s = 0; s < 4; ++s) {
            // four neighbouring channels of a row: two at places 2 t of the product's inner axis, two at 2 t + 8
            uint32_t f[4];
            ldsm4(f, kst + (16 * u + lrow) * 128 + (((2 * s + lhi) ^ lsw) << 4));
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const uint32_t a0 = e4m3_lo(f[2 * i]), a1 = e4m3_lo(f[2 * i + 1]), a2 = e4m3_hi(f[2 * i]), a3 = e4m3_hi(f[2 * i + 1]);
#pragma unroll
              for (int c = 0; c < kQ; ++c) mma16<true>(i ? p2[u][c] : p[u][c], a0, a1, a2, a3, qf[c][2 * s + i][0], qf[c][2 * s + i][1]);
            }
          }
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const uint8_t* sc = scales + c_stage * kPgScale + 16 * u + 8 * r + g;
            const int kb = sc[0], vb = sc[32];
            const float S = __uint_as_float((uint32_t)kb << 23);
            ev[u][r] = (float)vb - (127.f - kUp);
            inv[u][r] = __uint_as_float((uint32_t)(254 - vb) << 23);
#pragma unroll
            for (int c = 0; c < kQ; ++c) {
              p[u][c][2 * r] = (p[u][c][2 * r] + p2[u][c][2 * r]) * S;
              p[u][c][2 * r + 1] = (p[u][c][2 * r + 1] + p2[u][c][2 * r + 1]) * S;
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
            if (row >= cur.first && row < cur.len) continue;
            ev[u][r] = kUp;
            inv[u][r] = 1.f;
#pragma unroll
            for (int c = 0; c < kQ; ++c) p[u][c][2 * r] = p[u][c][2 * r + 1] = -INFINITY;
          }
      }
      // the values' fragments are on their way while the weights are computed, where registers allow it
      constexpr bool kEarly = kHeads < 16;
      uint32_t vf[8][4];
      const uint32_t vrow = (lane & 7) + ((lane >> 4) << 3), vhi = (lane >> 3) & 1;  // rows 0-7 and 8-15 by channels 16 j and 16 j + 8
      auto load_values = [&](int j) {
        if constexpr (kE4m3) ldsm4_t(vf[j], vst + lane * 128 + ((j ^ lsw) << 4));
        else ldsm4_t(vf[j], vst + (j >> 2) * 2048 + vrow * 128 + (((2 * (j & 3) + vhi) ^ lsw) << 4));
      };
      if constexpr (kEarly)
#pragma unroll
        for (int j = 0; j < 8; ++j) load_values(j);
      // exponents of the weights, kUp up (NaN counts as no growth)
      float sc[kU][kQ][4];
      auto exponents = [&]() {
#pragma unroll
        for (int c = 0; c < kQ; ++c)
#pragma unroll
          for (int u = 0; u < kU; ++u)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const float d = p[u][c][x] - m[c][x & 1].d;
              sc[u][c][x] = kE4m3 ? fmaf(d, qs[c][x & 1], ev[u][x >> 1] - m[c][x & 1].e) : d * qs[c][x & 1];
            }
      };
      exponents();
      bool grows = false;
#pragma unroll
      for (int u = 0; u < kU; ++u)
#pragma unroll
        for (int c = 0; c < kQ; ++c)
#pragma unroll
          for (int x = 0; x < 4; ++x)
            grows |= sc[u][c][x] > kPgGrowth + kUp || (!live[c][x & 1] && p[u][c][x] > -INFINITY);
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
            PgMax best = {-INFINITY, 0.f};
#pragma unroll
            for (int u = 0; u < kU; ++u)
#pragma unroll
              for (int r = 0; r < 2; ++r) {
                const float d = p[u][c][2 * r + i], k2 = kE4m3 ? sc[u][c][2 * r + i] : d;
                const bool more = k2 > k;
                k = more ? k2 : k;
                best.d = more ? d : best.d;
                if (kE4m3) best.e = more ? ev[u][r] - kUp : best.e;
              }
            float top = k;
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, off));
            if (kE4m3) {  // that of the first of the eight lanes that have it
              const int src = __ffs(__ballot_sync(kFull, k == top) & (0x11111111u << t)) - 1;
              best = {__shfl_sync(kFull, best.d, src), __shfl_sync(kFull, best.e, src)};
            } else {
              best.d = top;
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
          }
        exponents();
#pragma unroll
        for (int u = 0; u < kU; ++u)
#pragma unroll
          for (int c = 0; c < kQ; ++c)
#pragma unroll
            for (int x = 0; x < 4; ++x) grows |= sc[u][c][x] > kPgGrowth + kUp;
      }

      // P^T as the second operand: rows 16 u + 8 r, a column tile's upper and lower parts
      uint32_t pb[kU][kQ][kParts][2];
#pragma unroll
      for (int u = 0; u < kU; ++u)
#pragma unroll
        for (int c = 0; c < kQ; ++c)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float w0 = ex2(sc[u][c][2 * r]), w1 = ex2(sc[u][c][2 * r + 1]);
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
        if constexpr (!kEarly) load_values(j);
        const uint32_t (&f)[4] = vf[j];
        if constexpr (!kE4m3) {
#pragma unroll
          for (int c = 0; c < kQ; ++c)
#pragma unroll
            for (int s = 0; s < kParts; ++s) mma16<false>(o[j][c], f[0], f[1], f[2], f[3], pb[0][c][s][0], pb[0][c][s][1]);
        } else {
#pragma unroll
          for (int u = 0; u < kU; ++u) {
            // two rows by two channels a word: even channels are the product's first eight rows, odd ones the others
            const uint32_t w0 = __byte_perm(f[2 * u], 0, 0x3120), w1 = __byte_perm(f[2 * u + 1], 0, 0x3120);
            const uint32_t a0 = e4m3_lo(w0), a1 = e4m3_hi(w0), a2 = e4m3_lo(w1), a3 = e4m3_hi(w1);
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

    if (pending) sh.next[(k + 1) & 1] = fetched;
    // the next job's queries, on their way through what follows
    if (in_next) load_queries(nxt);
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
    if (tid == kPgThreads - 1) sh.next[k & 1] = kPgUnknown;  // this job's own: read by all before
    // their results, kCh channels at a time: [warp][head][channel]
    constexpr int kCh = kPgOut / 4 / kPgWarps / kHeads, kTiles = kCh / 16, kStride = kCh + 4;
    const int h = tid * 4 / kCh, ch = tid * 4 % kCh;  // a thread's share of the joined result
    PgMax best = {0.f, 0.f};
    const float scale = sh.ml[0][h].w;
    float share[kPgWarps], sum = 0.f;
    {
      bool any = false;
#pragma unroll
      for (int w = 0; w < kPgWarps; ++w) {
        const float4 v = sh.ml[w][h];
        if (v.z != 0.f && (!any || above({v.x, v.y}, best, scale) > 0.f)) {
          best = {v.x, v.y};
          any = true;
        }
      }
#pragma unroll
      for (int w = 0; w < kPgWarps; ++w) {
        const float4 v = sh.ml[w][h];
        share[w] = v.z != 0.f ? ex2(above({v.x, v.y}, best, scale)) : 0.f;
        sum += v.z != 0.f ? v.z * share[w] : 0.f;
        share[w] *= kDown;
      }
    }
    bool bad = false;
#pragma unroll
    for (int pass = 0; pass < kDim / kCh; ++pass) {
      if (pass > 0) __syncthreads();
#pragma unroll
      for (int jj = 0; jj < kTiles; ++jj) {
        const int j = pass * kTiles + jj;
#pragma unroll
        for (int c = 0; c < kQ; ++c)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float v0 = o[j][c][i], v1 = o[j][c][i + 2];
            if constexpr (kHeads == 4) {
              v0 += __shfl_xor_sync(kFull, v0, 2);
              v1 += __shfl_xor_sync(kFull, v1, 2);
            }
            float* to = so + (warp * kHeads + 8 * c + 2 * t + i) * kStride + 16 * jj;
            if (kHeads > 4 || t < 2) {
              if constexpr (kE4m3) {
                *reinterpret_cast<float2*>(to + 2 * g) = make_float2(v0, v1);
              } else {
                to[g] = v0;
                to[g + 8] = v1;
              }
            }
          }
      }
      __syncthreads();
      if (h < nh) {
        float4 r = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kPgWarps; ++w) {
          const float f = share[w];
          const float4 v = *reinterpret_cast<const float4*>(so + (w * kHeads + h) * kStride + ch);
          if (f == 0.f) continue;  // no rows of weight
          r.x = fmaf(v.x, f, r.x);
          r.y = fmaf(v.y, f, r.y);
          r.z = fmaf(v.z, f, r.z);
          r.w = fmaf(v.w, f, r.w);
        }
        const float4 all = make_float4(best.d, best.e, sum, scale);
        const int channel = pass * kCh + ch;
        if (kWhole || cur.slot < 0) {
          if constexpr (!kE4m3) bad |= not_finite(r, sum);
          const float inv = all.z != 0.f ? 1.f / all.z : 0.f;
          const int64_t q = (int64_t)cur.s * a.hq + qh0 + h;
          *reinterpret_cast<uint2*>(a.out + q * kDim + channel) =
              make_uint2(pack_bf16x2(r.x * inv, r.y * inv), pack_bf16x2(r.z * inv, r.w * inv));
          if (a.lse != nullptr && channel == 0)
            a.lse[q] = all.z != 0.f ? kLn2 * (fmaf(all.x, all.w, all.y) + log2f(all.z)) : -INFINITY;
        } else {
          float* part = a.part + ((int64_t)cur.slot * a.hq + qh0 + h) * kPartStride;
          *reinterpret_cast<float4*>(part + 4 + channel) = r;
          if (channel == 0) *reinterpret_cast<float4*>(part) = all;
        }
      }
    }
    // what the sums went through may be used again
    if constexpr (kE4m3) {
      __syncthreads();
    } else if (__syncthreads_or(bad)) {
      again = true;
      if (tid == 0 && !kWhole) a.counts[2] = 1;  // the joining kernel looks for it
    }
    job = (uint32_t)sh.next[(k + 1) & 1];
    if (job >= jobs) break;
    if (!in_next) {
      nxt = find(job);
      enter(nxt);
      load_queries(nxt);
    }
    cur = nxt;
    in_next = false;
    ++k;
  }

  // sequences without rows: spread over the blocks
  for (int s = blockIdx.x; s < a.c.n_seqs; s += blocks) {
    if (paged_len(a.c, s) > 0) continue;
    const int64_t q = (int64_t)s * a.hq;
    for (int i = tid; i < a.hq * (kDim / 8); i += kPgThreads) reinterpret_cast<uint4*>(a.out + q * kDim)[i] = make_uint4(0, 0, 0, 0);
    if (a.lse != nullptr)
      for (int i = tid; i < a.hq; i += kPgThreads) a.lse[q + i] = -INFINITY;
  }

  // Where no other kernel follows, a block's results that are not finite wait for
  // the end of its jobs, blockIdx.x + k blocks (in the loop above, reached or not,
  // they cost 0.7 us of a call's 7.2; here 0.2).
  if (kE4m3 || !kWhole || !again) return;
  for (uint32_t j = blockIdx.x; j < jobs; j += blocks) {
    const PgJob w = find(j);
    for (int i = warp; i < min(kHeads, a.g - w.h0); i += kPgWarps) row_again(a, w.s, w.kvh * a.g + w.h0 + i, 0, kDim);
  }
}

// The units' partial sums of a sequence and query head, joined: a block an
// item, each of its warps every fourth result, eight of them under way
// while the maxima are looked at, which every warp does for itself.  Bound by
// latency: three loads that need one another.
constexpr int kPgJoin = 4;
template <bool kE4m3>
__global__ void __launch_bounds__(32 * kPgJoin, 8) k_paged_join(const __grid_constant__ PagedAttendArgs a) {
  constexpr int kWarps = kPgJoin, kAhead = 8;
  constexpr int kHeld = kWarps * kAhead / 32;  // maxima and sums a lane has of as many units as the results under way
  __shared__ float4 so[kWarps][32];
  __shared__ AgainFlags again;
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (blockIdx.x == 0 && tid == 0) a.counts[0] = 0;  // the queue, for the next call
  AgainFlags::start<kE4m3>(again, a);
  for (int64_t it = blockIdx.x; it < (int64_t)a.max_splits * a.hq; it += gridDim.x) {
    const PgSplit sp = a.splits[it / a.hq];
    if (it / a.hq >= a.counts[1]) break;
    const int h = (int)(it - it / a.hq * a.hq), n = min(sp.units, a.slots - sp.slot);
    const float* part = a.part + ((int64_t)sp.slot * a.hq + h) * kPartStride;
    const int64_t step = (int64_t)a.hq * kPartStride;
    float4 v[kHeld], x[kAhead];
    auto load = [&](int u0) {
#pragma unroll
      for (int k = 0; k < kHeld; ++k) {
        v[k] = make_float4(0.f, 0.f, 0.f, 0.f);  // the sum 0: no rows of weight
        if (u0 + 32 * k + lane < n) v[k] = *reinterpret_cast<const float4*>(part + (u0 + 32 * k + lane) * step);
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (u0 + warp + i * kWarps < n) x[i] = *(reinterpret_cast<const float4*>(part + (u0 + warp + i * kWarps) * step + 4) + lane);
    };
    load(0);
    const float qs = __shfl_sync(kFull, v[0].w, 0);
    PgMax m = {0.f, 0.f};
#pragma unroll 1
    for (int round = 0; round < 2; ++round) {  // the second finds the largest by exact distances from about the largest
      float far = -INFINITY;
      PgMax best = {-INFINITY, -INFINITY};
      auto look = [&](const float4& w) {
        const float d = w.z != 0.f ? above({w.x, w.y}, m, qs) : -INFINITY;
        const bool more = d > far;
        far = more ? d : far;
        best.d = more ? w.x : best.d;
        best.e = more ? w.y : best.e;
      };
#pragma unroll
      for (int k = 0; k < kHeld; ++k) look(v[k]);
      for (int i = 32 * kHeld + lane; i < n; i += 32) look(*reinterpret_cast<const float4*>(part + i * step));
      float top = far;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, off));
      const int src = __ffs(__ballot_sync(kFull, far == top)) - 1;
      if (top > -INFINITY) m = {__shfl_sync(kFull, best.d, src), __shfl_sync(kFull, best.e, src)};
    }
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    float sum = 0.f;
    for (int u0 = 0; u0 < n; u0 += 32 * kHeld) {
      if (u0 > 0) load(u0);
      float f[kHeld];
#pragma unroll
      for (int k = 0; k < kHeld; ++k) {
        f[k] = v[k].z != 0.f ? ex2(above({v[k].x, v[k].y}, m, qs)) : 0.f;
        if (v[k].z != 0.f) sum = fmaf(v[k].z, f[k], sum);
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int u = warp + i * kWarps;
        const float fi = __shfl_sync(kFull, f[i * kWarps / 32], u & 31);
        if (u0 + u >= n || fi == 0.f) continue;
        o.x = fmaf(x[i].x, fi, o.x);
        o.y = fmaf(x[i].y, fi, o.y);
        o.z = fmaf(x[i].z, fi, o.z);
        o.w = fmaf(x[i].w, fi, o.w);
      }
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(kFull, sum, off);
    so[warp][lane] = o;
    __syncthreads();
    if (warp == 0) {
#pragma unroll
      for (int w = 1; w < kWarps; ++w) {
        const float4 y = so[w][lane];
        o.x += y.x;
        o.y += y.y;
        o.z += y.z;
        o.w += y.w;
      }
      const float inv = sum != 0.f ? 1.f / sum : 0.f;
      const int64_t q = (int64_t)sp.s * a.hq + h;
      reinterpret_cast<uint2*>(a.out + q * kDim)[lane] = make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
      if (a.lse != nullptr && lane == 0) a.lse[q] = sum != 0.f ? kLn2 * (fmaf(m.d, qs, m.e) + log2f(sum)) : -INFINITY;
      if (!kE4m3 && not_finite(o, sum)) again.mine = 1;
    }
    __syncthreads();
  }
  if constexpr (!kE4m3) again.finish(a, 1);
}

// The same for sequences of many units (few KV heads or sequences), with more
// threads an item: kParts blocks, each for its part of the channels, whose
// threads share the maxima and leave the units' weights in shared memory.  In
// place of 16 of the other's warps: 131072 rows of one KV head and 8 query heads
// 32.6 -> 24.3 us, 400000 69.1 -> 48.8, 30000 of 8 KV heads 28.6 -> 27.9.
constexpr int kPgManyUnits = 2048;
template <bool kE4m3, int kWarps, int kParts>
__global__ void __launch_bounds__(32 * kWarps) k_paged_join_many(const __grid_constant__ PagedAttendArgs a) {
  constexpr int kThreads = 32 * kWarps, kLanes = 32 / kParts, kEach = kThreads / kLanes, kAhead = 4;  // lanes of a result, results at once
  __shared__ float2 top[kPgManyUnits];      // a unit's maximum
  __shared__ float weight[kPgManyUnits];    // its sum, then its share
  __shared__ float4 far[2][kWarps], so[kWarps][kLanes];
  __shared__ float sums[kWarps];
  __shared__ AgainFlags again;
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, mine = tid / kLanes;
  if (blockIdx.x == 0 && tid == 0) a.counts[0] = 0;  // the queue, for the next call
  AgainFlags::start<kE4m3>(again, a);
  for (int64_t b = blockIdx.x; b < (int64_t)a.max_splits * a.hq * kParts; b += gridDim.x) {
    const int64_t it = b / kParts;
    const int channel = ((int)(b - it * kParts) * kLanes + lane % kLanes) * 4;
    const PgSplit sp = a.splits[it / a.hq];
    if (it / a.hq >= a.counts[1]) break;
    const int h = (int)(it - it / a.hq * a.hq), n = min(min(sp.units, a.slots - sp.slot), kPgManyUnits);
    const float* part = a.part + ((int64_t)sp.slot * a.hq + h) * kPartStride;
    const int64_t step = (int64_t)a.hq * kPartStride;
    float4 x[kAhead];
    PgMax m = {0.f, 0.f};
    float qs = 0.f, d0 = -INFINITY;
    PgMax best = {-INFINITY, -INFINITY};
    auto look = [&](float d, float e, float z) {
      const float up = z != 0.f ? above({d, e}, m, qs) : -INFINITY;
      const bool more = up > d0;
      d0 = more ? up : d0;
      best.d = more ? d : best.d;
      best.e = more ? e : best.e;
    };
    auto meet = [&](int round) {  // the block's largest, the first one of several
      float t = d0;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) t = fmaxf(t, __shfl_xor_sync(kFull, t, off));
      const int src = __ffs(__ballot_sync(kFull, d0 == t)) - 1;
      const float d = __shfl_sync(kFull, best.d, src), e = __shfl_sync(kFull, best.e, src);
      if (lane == 0) far[round][warp] = make_float4(t, d, e, qs);
      __syncthreads();
      qs = far[round][0].w;
      t = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float4 v = far[round][w];
        if (v.x > t) {
          t = v.x;
          m = {v.y, v.z};
        }
      }
    };
#pragma unroll 4
    for (int u = tid; u < n; u += kThreads) {
      const float4 v = *reinterpret_cast<const float4*>(part + u * step);
      top[u] = make_float2(v.x, v.y);
      weight[u] = v.z;
      qs = v.w;
      look(v.x, v.y, v.z);
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (mine + i * kEach < n) x[i] = *reinterpret_cast<const float4*>(part + (mine + i * kEach) * step + 4 + channel);
    meet(0);
    d0 = -INFINITY;  // by exact distances from about the largest
    best = {-INFINITY, -INFINITY};
    for (int u = tid; u < n; u += kThreads) look(top[u].x, top[u].y, weight[u]);
    meet(1);
    float sum = 0.f;
    for (int u = tid; u < n; u += kThreads) {
      const float z = weight[u], f = z != 0.f ? ex2(above({top[u].x, top[u].y}, m, qs)) : 0.f;
      if (z != 0.f) sum = fmaf(z, f, sum);
      weight[u] = f;
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(kFull, sum, off);
    if (lane == 0) sums[warp] = sum;
    __syncthreads();
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int u0 = mine; u0 < n; u0 += kAhead * kEach) {
      float f[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int u = u0 + i * kEach;
        f[i] = u < n ? weight[u] : 0.f;
        if (u0 != mine && u < n) x[i] = *reinterpret_cast<const float4*>(part + u * step + 4 + channel);
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        if (f[i] == 0.f) continue;
        o.x = fmaf(x[i].x, f[i], o.x);
        o.y = fmaf(x[i].y, f[i], o.y);
        o.z = fmaf(x[i].z, f[i], o.z);
        o.w = fmaf(x[i].w, f[i], o.w);
      }
    }
#pragma unroll
    for (int off = 16; off >= kLanes; off >>= 1) {
      o.x += __shfl_xor_sync(kFull, o.x, off);
      o.y += __shfl_xor_sync(kFull, o.y, off);
      o.z += __shfl_xor_sync(kFull, o.z, off);
      o.w += __shfl_xor_sync(kFull, o.w, off);
    }
    if (lane < kLanes) so[warp][lane] = o;
    __syncthreads();
    if (tid < kLanes) {
      sum = sums[0];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) {
        const float4 y = so[w][lane];
        o.x += y.x;
        o.y += y.y;
        o.z += y.z;
        o.w += y.w;
        sum += sums[w];
      }
      const float inv = sum != 0.f ? 1.f / sum : 0.f;
      const int64_t q = (int64_t)sp.s * a.hq + h;
      *reinterpret_cast<uint2*>(a.out + q * kDim + channel) = make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
      if (a.lse != nullptr && channel == 0) a.lse[q] = sum != 0.f ? kLn2 * (fmaf(m.d, qs, m.e) + log2f(sum)) : -INFINITY;
      if (!kE4m3 && not_finite(o, sum)) again.mine = 1;
    }
    __syncthreads();  // what was shared may be used again
  }
  if constexpr (!kE4m3) again.finish(a, kParts);
}

// Rows of one head and page: 128 codes each, or two halves of 64 bf16 values,
// one behind the other in shared memory; 128 bytes a row of either.
bool encode_pages(CUtensorMap* m, const Paged& c, const uint8_t* base, const PageStrides& s, int layer) {
  EncodeTiled fn = encode_tiled();
  if (fn == nullptr) return false;
  const cuuint32_t rows = 1u << c.shift, hkv = c.hkv, pages = c.n_pages, one[5] = {1, 1, 1, 1, 1};
  const cuuint64_t row = s.row, head = s.head, page = s.page;
  void* p = const_cast<uint8_t*>(base + layer * s.layer);
  if (c.e4m3) {
    const cuuint64_t dims[4] = {kDim, rows, hkv, pages}, strides[3] = {row, head, page};
    const cuuint32_t box[4] = {kDim, std::min(rows, 32u), 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, p, dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  }
  const cuuint64_t dims[5] = {kDim / 2, rows, 2, hkv, pages}, strides[4] = {row, kDim, head, page};
  const cuuint32_t box[5] = {kDim / 2, 16, 2, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, p, dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int heads_of(int g) { return g <= 4 ? 4 : g <= 8 ? 8 : 16; }

template <bool kE4m3, int kHeads, bool kWhole>
cudaError_t launch_heads(const PagedAttendArgs& a, const CUtensorMap& km, const CUtensorMap& vm, cudaStream_t st) {
  static std::atomic<bool> done[64];  // the limit belongs to the device; setting it twice is harmless
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess && !(dev >= 0 && dev < 64 && done[dev])) {
    e = cudaFuncSetAttribute((const void*)k_paged_attend<kE4m3, kHeads, kWhole>, cudaFuncAttributeMaxDynamicSharedMemorySize, kPgSmem);
    if (e == cudaSuccess && dev >= 0 && dev < 64) done[dev] = true;
  }
  if (e != cudaSuccess) return e;
  return launch_pdl(k_paged_attend<kE4m3, kHeads, kWhole>, dim3(a.nblocks), dim3(kPgThreads), kPgSmem, st, a, km, vm);
}

template <bool kE4m3, bool kWhole>
cudaError_t launch_attend(const PagedAttendArgs& a, const CUtensorMap& km, const CUtensorMap& vm, cudaStream_t st) {
  const int heads = heads_of(a.g);
  return heads == 4   ? launch_heads<kE4m3, 4, kWhole>(a, km, vm, st)
         : heads == 8 ? launch_heads<kE4m3, 8, kWhole>(a, km, vm, st)
                      : launch_heads<kE4m3, 16, kWhole>(a, km, vm, st);
}

// Few items have many units each, and many have few; eight parts of the
// channels where that leaves no block without an SM (one sequence 48.8 us, four
// parts 50.6; 128 items 41.7, four 39.0).
template <bool kE4m3>
cudaError_t launch_join(const PagedAttendArgs& a, int64_t items, cudaStream_t st) {
  if (items <= a.nblocks / 2 && 6 * a.nblocks / (a.c.hkv * a.groups) + 2 <= kPgManyUnits) {
    constexpr int kWarps = 8;
    if (8 * items <= 2 * a.nblocks)
      return launch_pdl(k_paged_join_many<kE4m3, kWarps, 8>, dim3((unsigned)(8 * items)), dim3(32 * kWarps), 0, st, a);
    return launch_pdl(k_paged_join_many<kE4m3, kWarps, 4>, dim3((unsigned)std::min<int64_t>(4 * items, 4 * a.nblocks)), dim3(32 * kWarps), 0, st, a);
  }
  return launch_pdl(k_paged_join<kE4m3>, dim3((unsigned)std::min<int64_t>(items, 4 * a.nblocks)), dim3(32 * kPgJoin), 0, st, a);
}

}  // namespace

// What a call needs for its cache, heads and GPU.
PagedAttendPlan paged_attend_plan(const Paged& c, int hq, int sm_count) {
  PagedAttendPlan p;
  const int g = hq / c.hkv, heads = heads_of(g);
  p.groups = (g + heads - 1) / heads;
  const int64_t jobs = (int64_t)c.hkv * p.groups, tile = c.e4m3 ? Pg<true>::kTile : Pg<false>::kTile;
  const int64_t tiles = (((int64_t)c.width << c.shift) + tile - 1) / tile * c.n_seqs;
  p.blocks = (int)std::min<int64_t>(2 * (int64_t)sm_count, tiles * jobs);  // two an SM
  // Units of sequences that have several: with T tiles, `large` is at least
  // 3/8 and `small` 1/16 of T jobs / blocks, so 3/4 T makes two and 1/4 T four
  // units a block and head (as 0.66 T and 0.34 T of 0.33 and 0.085 do), at most
  // one more each for a sequence, of which fewer than T / small have several.
  p.max_splits = tiles <= kPgWhole * (int64_t)c.n_seqs ? 0 : (int)std::min<int64_t>(c.n_seqs, 16 * p.blocks / jobs + 1);
  p.slots = (int)(6 * p.blocks / jobs + 2 * p.max_splits + 4);
  p.part_bytes = (size_t)p.slots * hq * kPartStride * sizeof(float);
  p.bytes = p.part_bytes + (size_t)p.max_splits * sizeof(PgSplit);
  return p;
}

cudaError_t paged_attend_error(uint32_t* bits) { return take_gave_up(bits); }

cudaError_t launch_paged_attend(const PagedAttendArgs& a, cudaStream_t st) {
  CUtensorMap km, vm;
  if (!encode_pages(&km, a.c, a.c.k, a.c.sk, a.layer) || !encode_pages(&vm, a.c, a.c.v, a.c.sv, a.layer)) return cudaErrorInvalidValue;
  const bool whole = a.max_splits == 0;  // no sequence can have several units
  const cudaError_t e = a.c.e4m3 ? whole ? launch_attend<true, true>(a, km, vm, st) : launch_attend<true, false>(a, km, vm, st)
                        : whole  ? launch_attend<false, true>(a, km, vm, st)
                                 : launch_attend<false, false>(a, km, vm, st);
  if (e != cudaSuccess || whole) return e;
  const int64_t items = (int64_t)a.max_splits * a.hq;
  return a.c.e4m3 ? launch_join<true>(a, items, st) : launch_join<false>(a, items, st);
}

}  // namespace paris
