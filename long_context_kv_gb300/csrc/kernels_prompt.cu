// Causal attention over prompts, and the window weights: one warp per row.
#include "kv4_internal.cuh"

namespace paris {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kScaleLog2 = kLog2e * 0.08838834764831845f;  // log2(e) / sqrt(128)
constexpr int kRowWarps = 8;

__device__ __forceinline__ float dot8(uint4 a, const float* q, float acc) {
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    acc = fmaf(bf16_bits_to_float(w[i] & 0xffffu), q[2 * i], acc);
    acc = fmaf(bf16_bits_to_float(w[i] >> 16), q[2 * i + 1], acc);
  }
  return acc;
}

// One query row by one warp: its visible keys 32 at a time, a lane per key
// for the scores, four channels per lane for the weighted sum.  Only rows
// that the query sees are read.  qs: the warp's 128 floats of shared memory.
__device__ void prompt_row(const PromptArgs& a, int s, int h, int64_t q0, int64_t i, int64_t k0, int64_t visible,
                           float* qs) {
  const int lane = threadIdx.x & 31;
  const int kvh = h / a.g;
  const __nv_bfloat16* q = a.q + (a.cu_q ? 0 : s * a.sq.seq) + (q0 + i) * a.sq.token + h * a.sq.head;
  const __nv_bfloat16* k = a.k + (a.cu_k ? 0 : s * a.sk.seq) + k0 * a.sk.token + kvh * a.sk.head;
  const __nv_bfloat16* v = a.v + (a.cu_k ? 0 : s * a.sv.seq) + k0 * a.sv.token + kvh * a.sv.head;
  float y[4];
  load4(q, 1, 4 * lane, y);
#pragma unroll
  for (int c = 0; c < 4; ++c) qs[4 * lane + c] = y[c];
  __syncwarp();
  float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
  for (int64_t j0 = 0; j0 < visible; j0 += 32) {
    const int n = (int)min64(32, visible - j0);
    float sc = -INFINITY;
    if (lane < n) {
      const uint4* kr = reinterpret_cast<const uint4*>(k + (j0 + lane) * a.sk.token);
      float acc = 0.f;
#pragma unroll
      for (int c = 0; c < 16; ++c) acc = dot8(kr[c], qs + 8 * c, acc);
      sc = acc * kScaleLog2;
    }
    float mx = sc;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, off));
    const float mn = fmaxf(m, mx);
    const float f = m == mn ? 1.f : exp2f(m - mn);
    m = mn;
    const float p = lane < n ? exp2f(sc - m) : 0.f;
    float ps = p;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) ps += __shfl_xor_sync(kFull, ps, off);
    l = l * f + ps;
#pragma unroll
    for (int c = 0; c < 4; ++c) o[c] *= f;
    for (int j = 0; j < n; ++j) {
      const float pj = __shfl_sync(kFull, p, j);
      float vy[4];
      load4(v + (j0 + j) * a.sv.token, 1, 4 * lane, vy);
#pragma unroll
      for (int c = 0; c < 4; ++c) o[c] = fmaf(pj, vy[c], o[c]);
    }
  }
  const float inv = visible > 0 ? 1.f / l : 0.f;
  __nv_bfloat16* out = a.out + (a.cu_q ? 0 : s * a.so.seq) + (q0 + i) * a.so.token + h * a.so.head;
  *reinterpret_cast<uint2*>(out + 4 * lane) = make_uint2(pack_bf16x2(o[0] * inv, o[1] * inv), pack_bf16x2(o[2] * inv, o[3] * inv));
  if (a.lse != nullptr && lane == 0)
    a.lse[((int64_t)(a.cu_q ? 0 : s) * a.hq + h) * a.rows_q + q0 + i] = visible > 0 ? (m + log2f(l)) * kLn2 : -INFINITY;
  __syncwarp();
}

__global__ void __launch_bounds__(32 * kRowWarps) k_prompt_rows(PromptArgs a) {
  __shared__ float qs[kRowWarps][kDim];
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x >> 5;
  const int s = blockIdx.z, h = blockIdx.y;
  int64_t q0, lq, k0, lk;
  seq_rows(a.cu_q, s, a.rows_q, q0, lq);
  seq_rows(a.cu_k, s, a.rows_k, k0, lk);
  const int64_t i = (int64_t)blockIdx.x * kRowWarps + warp;
  if (i >= min64(lq, a.max_q)) return;
  prompt_row(a, s, h, q0, i, k0, max64(0, min64(lk, i + lk - lq + 1)), qs[warp]);
}

// One warp per (KV head, key): the window's queries in order.
__global__ void __launch_bounds__(32 * kRowWarps) k_prompt_weights(PromptWeightArgs w) {
  pdl_wait();
  pdl_trigger();
  const PromptArgs& a = w.p;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int s = blockIdx.z, kvh = blockIdx.y;
  int64_t q0, lq, k0, lk;
  seq_rows(a.cu_q, s, a.rows_q, q0, lq);
  seq_rows(a.cu_k, s, a.rows_k, k0, lk);
  const int64_t j = (int64_t)blockIdx.x * kRowWarps + warp;
  if (j >= min64(lk, a.max_k)) return;
  float y[4];
  load4(a.k + (a.cu_k ? 0 : s * a.sk.seq) + (k0 + j) * a.sk.token + kvh * a.sk.head, 1, 4 * lane, y);
  float sum = 0.f;
  for (int64_t i = max64(max64(0, lq - w.window), j - (lk - lq)); i < lq; ++i) {
    for (int g = 0; g < a.g; ++g) {
      const int h = kvh * a.g + g;
      float x[4];
      load4(a.q + (a.cu_q ? 0 : s * a.sq.seq) + (q0 + i) * a.sq.token + h * a.sq.head, 1, 4 * lane, x);
      float d = 0.f;
#pragma unroll
      for (int c = 0; c < 4; ++c) d = fmaf(x[c], y[c], d);
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) d += __shfl_xor_sync(kFull, d, off);
      const float lse = w.lse[((int64_t)(a.cu_q ? 0 : s) * a.hq + h) * a.rows_q + q0 + i];
      if (lse != -INFINITY) sum += exp2f(d * kScaleLog2 - lse * kLog2e);
    }
  }
  if (lane == 0) w.weights[((int64_t)(a.cu_k ? 0 : s) * a.hkv + kvh) * a.rows_k + k0 + j] = sum;
}

}  // namespace

size_t prompt_workspace_bytes(PromptArgs& a, int) {
  a.nsplit = 1;
  return 0;
}

cudaError_t launch_prompt_attend(const PromptArgs& a, cudaStream_t st) {
  const dim3 grid((unsigned)((a.max_q + kRowWarps - 1) / kRowWarps), a.hq, a.n_seqs);
  return launch_pdl(k_prompt_rows, grid, dim3(32 * kRowWarps), 0, st, a);
}

cudaError_t launch_prompt_weights(const PromptWeightArgs& w, cudaStream_t st) {
  const dim3 grid((unsigned)((w.p.max_k + kRowWarps - 1) / kRowWarps), w.p.hkv, w.p.n_seqs);
  return launch_pdl(k_prompt_weights, grid, dim3(32 * kRowWarps), 0, st, w);
}

}  // namespace paris
