// Attention of one new token over a paged cache.
#include <cuda_fp16.h>

#include "paged_internal.cuh"

namespace paris {
namespace {

// A warp for each (sequence, query head), four channels a lane, row by row
// with a running maximum and sum.
__global__ void __launch_bounds__(128) k_paged_attend_rows(PagedAttendArgs a) {
  pdl_wait();
  pdl_trigger();
  const int64_t w = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31, b = (int)(w / a.hq), h = (int)(w - (int64_t)b * a.hq);
  if (b >= a.c.n_seqs) return;
  const int kvh = h / a.g, len = paged_len(a.c, b), first = a.window > 0 ? max(0, len - a.window) : 0;
  float q[4], o[4] = {0.f, 0.f, 0.f, 0.f}, m = -INFINITY, l = 0.f;
  load4(a.q, 1, w * kDim + 4 * lane, q);
  auto row = [&](const uint8_t* base, const PageStrides& st, const uint8_t* scales, int page, int r, float (&x)[4]) {
    const uint8_t* p = base + a.layer * st.layer + page * st.page + kvh * st.head + r * st.row;
    if (!a.c.e4m3) {
      load4(p, 1, 4 * lane, x);
      return;
    }
    const uint32_t c = reinterpret_cast<const uint32_t*>(p)[lane], lo = e4m3_to_f16x2(c), hi = e4m3_to_f16x2(c >> 16);
    const float S = __uint_as_float((uint32_t)scales[scale_at(a.c, a.layer, page, kvh, r)] << 23);
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&lo)), g = __half22float2(*reinterpret_cast<const __half2*>(&hi));
    x[0] = f.x * S; x[1] = f.y * S; x[2] = g.x * S; x[3] = g.y * S;
  };
  for (int r = first; r < len; ++r) {
    const int page = page_at(a.c, b, r >> a.c.shift), pr = r & ((1 << a.c.shift) - 1);
    float k[4], v[4];
    row(a.c.k, a.c.sk, a.c.ks, page, pr, k);
    row(a.c.v, a.c.sv, a.c.vs, page, pr, v);
    float s = q[0] * k[0] + q[1] * k[1] + q[2] * k[2] + q[3] * k[3];
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(kFull, s, off);
    s *= 0.08838834764831845f;
    if (s == -INFINITY) continue;
    const float mn = fmaxf(m, s), f = l == 0.f ? 0.f : expf(m - mn), p = expf(s - mn);
    l = l * f + p;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = o[i] * f + p * v[i];
    m = mn;
  }
  const float inv = l != 0.f ? 1.f / l : 0.f;
  reinterpret_cast<uint2*>(a.out + w * kDim)[lane] = make_uint2(pack_bf16x2(o[0] * inv, o[1] * inv), pack_bf16x2(o[2] * inv, o[3] * inv));
  if (a.lse != nullptr && lane == 0) a.lse[w] = l != 0.f ? m + logf(l) : -INFINITY;
}

}  // namespace

int paged_attend_blocks(const Paged&, int, int) { return 1; }
size_t paged_attend_part_bytes(const Paged&, int, int) { return 16; }
cudaError_t paged_attend_error(uint32_t* bits) {
  *bits = 0;
  return cudaSuccess;
}

cudaError_t launch_paged_attend(const PagedAttendArgs& a, cudaStream_t st) {
  return launch_pdl(k_paged_attend_rows, dim3((unsigned)(((int64_t)a.c.n_seqs * a.hq + 3) / 4)), dim3(128), 0, st, a);
}

}  // namespace paris
