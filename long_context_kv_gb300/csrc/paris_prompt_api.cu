// C ABI of the prompt calls and the 4-bit cache (include/paris.h): argument
// checks and launches.  These calls hold no state: sizes that vary live on
// the device, buffers are the caller's.
#include <algorithm>
#include <atomic>
#include <cstdarg>
#include <cstdio>

#include "../../include/paris.h"
#include "kv4_internal.cuh"

using namespace paris;

namespace {

paris_status fail(paris_status st, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  set_thread_error(buf);
  return st;
}

paris_status launched(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return PARIS_OK;
  cudaGetLastError();  // reported here, not by the caller's next call
  return fail(PARIS_ECUDA, "%s: %s", what, cudaGetErrorString(e));
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int sm_count() {
  // asked once per device: the attribute cannot change
  static std::atomic<int> cached[64];
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return 148;
  if (dev < 64 && cached[dev] > 0) return cached[dev];
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    cudaGetLastError();
    return 148;
  }
  if (dev < 64) cached[dev] = n;
  return n;
}

// Strides of an axis of more than one entry have to be positive multiples of
// 8 elements; those of an axis of one entry mean nothing and are replaced.
paris_status take_strides(const paris_strides& s, int64_t tokens, int heads, int seqs, const char* name, Strides* out) {
  const struct { int64_t stride, n; const char* axis; int64_t* to; } axes[3] = {
      {s.token, tokens, "token", &out->token}, {s.head, heads, "head", &out->head}, {s.seq, seqs, "seq", &out->seq}};
  for (const auto& x : axes) {
    if (x.n <= 1) {
      *x.to = kDim;
      continue;
    }
    // sequences may be further apart: tensor maps take 2^40 bytes
    const int64_t most = x.to == &out->seq ? (int64_t)1 << 38 : (int64_t)1 << 31;
    if (x.stride < kDim || x.stride % 8 || x.stride >= most)
      return fail(PARIS_EINVAL, "%s: the %s stride must be a multiple of 8 elements, from %d to below %lld (got %lld)", name,
                  x.axis, kDim, (long long)most, (long long)x.stride);
    *x.to = x.stride;
  }
  return PARIS_OK;
}

paris_status take_prompt(const paris_prompt* p, PromptArgs* a, bool need_v) {
  if (!p) return fail(PARIS_EINVAL, "the prompt's description must not be NULL");
  if (p->head_dim != kDim) return fail(PARIS_EINVAL, "supported geometry: head_dim = %d (got %d)", kDim, p->head_dim);
  if (p->n_seqs < 0 || p->n_seqs > 65535) return fail(PARIS_EINVAL, "n_seqs must be in [0, 65535]");
  if (p->n_kv_heads < 1 || p->n_q_heads < p->n_kv_heads || p->n_q_heads % p->n_kv_heads)
    return fail(PARIS_EINVAL, "n_q_heads must be a positive multiple of n_kv_heads");
  if (p->n_q_heads > 65535 || p->n_q_heads / p->n_kv_heads > 128)
    return fail(PARIS_EINVAL, "at most 65535 query heads, and 128 per KV head");
  if ((p->cu_q == nullptr) != (p->cu_k == nullptr))
    return fail(PARIS_EINVAL, "cu_q and cu_k must both be given or both be NULL");
  if (p->rows_q < 0 || p->rows_k < 0 || p->rows_q > 0x7fffffff || p->rows_k > 0x7fffffff)
    return fail(PARIS_EINVAL, "rows_q and rows_k must be in [0, 2^31 - 1]");
  if (p->max_q < 0 || p->max_k < 0) return fail(PARIS_EINVAL, "max_q and max_k must be >= 0");
  a->n_seqs = p->n_seqs;
  a->hq = p->n_q_heads;
  a->hkv = p->n_kv_heads;
  a->g = p->n_q_heads / p->n_kv_heads;
  a->rows_q = p->rows_q;
  a->rows_k = p->rows_k;
  a->cu_q = p->cu_q;
  a->cu_k = p->cu_k;
  a->max_q = p->cu_q ? std::min(p->max_q, p->rows_q) : p->rows_q;
  a->max_k = p->cu_k ? std::min(p->max_k, p->rows_k) : p->rows_k;
  const int seqs = p->cu_q ? 1 : p->n_seqs;
  paris_status st = take_strides(p->q, p->rows_q, a->hq, seqs, "q", &a->sq);
  if (st == PARIS_OK) st = take_strides(p->k, p->rows_k, a->hkv, seqs, "k", &a->sk);
  if (st == PARIS_OK && need_v) st = take_strides(p->v, p->rows_k, a->hkv, seqs, "v", &a->sv);
  if (st == PARIS_OK && need_v) st = take_strides(p->out, p->rows_q, a->hq, seqs, "out", &a->so);
  return st;
}

paris_status take_cache(const paris_kv4* c, Kv4* k) {
  if (!c) return fail(PARIS_EINVAL, "the cache must not be NULL");
  if (c->head_dim != kDim) return fail(PARIS_EINVAL, "supported geometry: head_dim = %d (got %d)", kDim, c->head_dim);
  if (c->batch < 1 || c->n_kv_heads < 1 || (int64_t)c->batch * c->n_kv_heads > 65535)
    return fail(PARIS_EINVAL, "batch and n_kv_heads must be positive, and their product at most 65535");
  if (c->max_rows < 1 || c->max_rows > 0x7fffffff) return fail(PARIS_EINVAL, "max_rows must be in [1, 2^31 - 1]");
  if (!c->k_codes || !c->v_codes || !c->k_scales || !c->v_scales || !c->weights || !c->positions || !c->lens ||
      !c->next_pos || !c->counters || !c->status)
    return fail(PARIS_EINVAL, "the cache's arrays must not be NULL");
  if (!aligned16(c->k_codes) || !aligned16(c->v_codes) || !aligned16(c->k_scales) || !aligned16(c->v_scales) || !aligned16(c->weights))
    return fail(PARIS_EINVAL, "the cache's codes, scales and weights must be 16-byte aligned");
  *k = Kv4{c->batch, c->n_kv_heads, c->max_rows, c->k_codes, c->v_codes, c->k_scales, c->v_scales,
           c->weights, c->positions, c->lens, c->next_pos, c->counters, c->status};
  return PARIS_OK;
}

paris_status check_dtype(paris_dtype t) {
  return t == PARIS_F32 || t == PARIS_BF16 ? PARIS_OK : fail(PARIS_EINVAL, "dtype must be PARIS_F32 or PARIS_BF16");
}

size_t attend4_workspace(const Kv4& k, int hq, bool accumulate, int* nblocks) {
  *nblocks = kv4_blocks(k.batch, k.hkv, hq / k.hkv, k.rmax, sm_count());
  return (size_t)hq * *nblocks * kPartStride * sizeof(float) + ((size_t)k.batch * sizeof(int2) + 15) / 16 * 16 + (accumulate ? (size_t)k.batch * hq * k.rmax * sizeof(float) : 0);
}

paris_status check_heads(const Kv4& k, int hq) {
  if (hq < k.hkv || hq % k.hkv || hq / k.hkv > 16)
    return fail(PARIS_EINVAL, "n_q_heads must be a positive multiple of n_kv_heads, at most 16 per KV head (got %d, %d)", hq,
                k.hkv);
  return PARIS_OK;
}

}  // namespace

extern "C" {

paris_status paris_prompt_workspace(const paris_prompt* p, size_t* bytes) {
  PromptArgs a{};
  if (!bytes) return fail(PARIS_EINVAL, "bytes must not be NULL");
  const paris_status st = take_prompt(p, &a, true);
  if (st != PARIS_OK) return st;
  *bytes = a.n_seqs == 0 || a.max_q == 0 ? 0 : prompt_workspace_bytes(a, sm_count());
  return PARIS_OK;
}

paris_status paris_prompt_attend(const paris_prompt* p, const void* q, const void* k, const void* v, paris_dtype dtype,
                                 void* out_bf16, float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  PromptArgs a{};
  paris_status st = take_prompt(p, &a, true);
  if (st != PARIS_OK) return st;
  if (dtype != PARIS_BF16) return fail(PARIS_EINVAL, "paris_prompt_attend: q, k and v must be PARIS_BF16");
  if (a.n_seqs == 0 || a.max_q == 0) return PARIS_OK;
  if (!q || !out_bf16 || (a.rows_k > 0 && (!k || !v))) return fail(PARIS_EINVAL, "q, k, v and out must not be NULL");
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out_bf16))
    return fail(PARIS_EINVAL, "q, k, v and out must be 16-byte aligned");
  const size_t need = prompt_workspace_bytes(a, sm_count());
  if (need > 0 && (!workspace || workspace_bytes < need || !aligned16(workspace)))
    return fail(PARIS_EINVAL, "paris_prompt_attend: needs %zu bytes of 16-byte aligned workspace (got %zu)", need,
                workspace ? workspace_bytes : (size_t)0);
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.k = static_cast<const __nv_bfloat16*>(k);
  a.v = static_cast<const __nv_bfloat16*>(v);
  a.out = static_cast<__nv_bfloat16*>(out_bf16);
  a.lse = lse;
  a.ws = static_cast<float*>(workspace);
  return launched(launch_prompt_attend(a, sm_count(), static_cast<cudaStream_t>(stream)), "paris_prompt_attend");
}

paris_status paris_prompt_check(void) {
  uint32_t a = 0, w = 0;
  cudaError_t e = cudaDeviceSynchronize();
  if (e == cudaSuccess) e = prompt_attend_error(&a);
  if (e == cudaSuccess) e = prompt_weights_error(&w);
  if (e != cudaSuccess) return launched(e, "paris_prompt_check");
  if (a | w) return fail(PARIS_EDEVICE, "a prompt call gave up waiting for its copies or products: its results are not valid");
  return PARIS_OK;
}

paris_status paris_prompt_weights(const paris_prompt* p, const void* q, const void* k, paris_dtype dtype,
                                  const float* lse, int window, float* weights, void* stream) {
  PromptWeightArgs w{};
  paris_status st = take_prompt(p, &w.p, false);
  if (st != PARIS_OK) return st;
  if (dtype != PARIS_BF16) return fail(PARIS_EINVAL, "paris_prompt_weights: q and k must be PARIS_BF16");
  if (window < 0 || window > 1 << 24) return fail(PARIS_EINVAL, "window must be in [0, 2^24]");
  if (w.p.n_seqs == 0 || w.p.max_k == 0) return PARIS_OK;
  if (!k || !weights || (w.p.rows_q > 0 && (!q || !lse))) return fail(PARIS_EINVAL, "q, k, lse and weights must not be NULL");
  if (!aligned16(q) || !aligned16(k)) return fail(PARIS_EINVAL, "q and k must be 16-byte aligned");
  w.p.q = static_cast<const __nv_bfloat16*>(q);
  w.p.k = static_cast<const __nv_bfloat16*>(k);
  w.lse = lse;
  w.window = window;
  w.weights = weights;
  return launched(launch_prompt_weights(w, sm_count(), static_cast<cudaStream_t>(stream)), "paris_prompt_weights");
}

paris_status paris_kv4_store(const paris_kv4* c, const void* k, const void* v, paris_dtype dtype,
                             const paris_strides* ks, const paris_strides* vs, int64_t rows, const int32_t* cu,
                             int64_t max_new, const float* weights, void* stream) {
  StoreArgs a{};
  paris_status st = take_cache(c, &a.c);
  if (st == PARIS_OK) st = check_dtype(dtype);
  if (st != PARIS_OK) return st;
  if (!ks || !vs) return fail(PARIS_EINVAL, "the strides must not be NULL");
  if (rows < 0 || rows > 0x7fffffff || max_new < 0) return fail(PARIS_EINVAL, "rows must be in [0, 2^31 - 1], max_new >= 0");
  const int seqs = cu ? 1 : a.c.batch;
  st = take_strides(*ks, rows, a.c.hkv, seqs, "k", &a.ks);
  if (st == PARIS_OK) st = take_strides(*vs, rows, a.c.hkv, seqs, "v", &a.vs);
  if (st != PARIS_OK) return st;
  a.rows = rows;
  a.max_new = cu ? std::min(max_new, rows) : rows;
  if (a.max_new == 0) return PARIS_OK;
  if (!k || !v) return fail(PARIS_EINVAL, "k and v must not be NULL");
  if (!aligned16(k) || !aligned16(v)) return fail(PARIS_EINVAL, "k and v must be 16-byte aligned");
  a.k = k;
  a.v = v;
  a.dtype = dtype;
  a.cu = cu;
  a.weights = weights;
  return launched(launch_kv4_store(a, static_cast<cudaStream_t>(stream)), "paris_kv4_store");
}

paris_status paris_kv4_append(const paris_kv4* c, const void* k, const void* v, paris_dtype dtype, void* stream) {
  if (!c) return fail(PARIS_EINVAL, "the cache must not be NULL");
  const paris_strides s{(int64_t)c->n_kv_heads * kDim, kDim, (int64_t)c->n_kv_heads * kDim};
  return paris_kv4_store(c, k, v, dtype, &s, &s, 1, nullptr, 1, nullptr, stream);
}

paris_status paris_kv4_workspace(const paris_kv4* c, int n_q_heads, int accumulate, size_t* bytes) {
  Kv4 k;
  if (!bytes) return fail(PARIS_EINVAL, "bytes must not be NULL");
  paris_status st = take_cache(c, &k);
  if (st == PARIS_OK) st = check_heads(k, n_q_heads);
  if (st != PARIS_OK) return st;
  int nblocks;
  *bytes = attend4_workspace(k, n_q_heads, accumulate != 0, &nblocks);
  return PARIS_OK;
}

paris_status paris_kv4_attend(const paris_kv4* c, const void* q, paris_dtype dtype, int n_q_heads, int accumulate,
                              void* out_bf16, void* workspace, size_t workspace_bytes, void* stream) {
  Attend4Args a{};
  paris_status st = take_cache(c, &a.c);
  if (st == PARIS_OK) st = check_dtype(dtype);
  if (st == PARIS_OK) st = check_heads(a.c, n_q_heads);
  if (st != PARIS_OK) return st;
  if (!q || !out_bf16) return fail(PARIS_EINVAL, "q and out must not be NULL");
  if (!aligned16(q) || !aligned16(out_bf16)) return fail(PARIS_EINVAL, "q and out must be 16-byte aligned");
  const size_t need = attend4_workspace(a.c, n_q_heads, accumulate != 0, &a.nblocks);
  if (!workspace || workspace_bytes < need || !aligned16(workspace))
    return fail(PARIS_EINVAL, "paris_kv4_attend: needs %zu bytes of 16-byte aligned workspace (got %zu)", need,
                workspace ? workspace_bytes : (size_t)0);
  a.q = q;
  a.dtype = dtype;
  a.hq = n_q_heads;
  a.g = n_q_heads / a.c.hkv;
  a.accumulate = accumulate != 0;
  a.part = static_cast<float*>(workspace);
  a.chunks = reinterpret_cast<int2*>(a.part + (size_t)a.hq * a.nblocks * kPartStride);
  a.scores = reinterpret_cast<float*>(a.chunks) + ((size_t)a.c.batch * 2 + 3) / 4 * 4;
  a.out = static_cast<__nv_bfloat16*>(out_bf16);
  return launched(launch_kv4_attend(a, static_cast<cudaStream_t>(stream)), "paris_kv4_attend");
}

paris_status paris_kv4_evict_workspace(const paris_kv4* c, size_t* bytes) {
  Kv4 k;
  if (!bytes) return fail(PARIS_EINVAL, "bytes must not be NULL");
  const paris_status st = take_cache(c, &k);
  if (st != PARIS_OK) return st;
  *bytes = (size_t)k.batch * k.hkv * 2 * k.rmax * sizeof(int32_t);
  return PARIS_OK;
}

paris_status paris_kv4_evict(const paris_kv4* c, int64_t keep, int64_t sink, int64_t recent, void* workspace,
                             size_t workspace_bytes, void* stream) {
  EvictArgs a{};
  paris_status st = take_cache(c, &a.c);
  if (st != PARIS_OK) return st;
  if (keep < 1 || sink < 0 || recent < 0 || sink > keep || recent > keep - sink)
    return fail(PARIS_EINVAL, "keep >= 1, sink and recent >= 0, and sink + recent <= keep required");
  const size_t need = (size_t)a.c.batch * a.c.hkv * 2 * a.c.rmax * sizeof(int32_t);
  if (!workspace || workspace_bytes < need || !aligned16(workspace))
    return fail(PARIS_EINVAL, "paris_kv4_evict: needs %zu bytes of 16-byte aligned workspace (got %zu)", need,
                workspace ? workspace_bytes : (size_t)0);
  if (keep >= a.c.rmax) return PARIS_OK;  // no sequence can have more
  a.keep = keep;
  a.sink = sink;
  a.recent = recent;
  a.list = static_cast<int32_t*>(workspace);
  return launched(launch_kv4_evict(a, static_cast<cudaStream_t>(stream)), "paris_kv4_evict");
}

paris_status paris_kv4_read(const paris_kv4* c, void* k_out, void* v_out, int64_t rows, void* stream) {
  Kv4 k;
  const paris_status st = take_cache(c, &k);
  if (st != PARIS_OK) return st;
  if (rows < 0 || rows > k.rmax) return fail(PARIS_EINVAL, "rows must be in [0, max_rows]");
  if (rows == 0) return PARIS_OK;
  if (!k_out || !v_out) return fail(PARIS_EINVAL, "k_out and v_out must not be NULL");
  if (!aligned16(k_out) || !aligned16(v_out)) return fail(PARIS_EINVAL, "k_out and v_out must be 16-byte aligned");
  return launched(launch_kv4_read(k, static_cast<__nv_bfloat16*>(k_out), static_cast<__nv_bfloat16*>(v_out), rows,
                                  static_cast<cudaStream_t>(stream)),
                  "paris_kv4_read");
}

paris_status paris_kv4_check(const paris_kv4* c) {
  Kv4 k;
  const paris_status st = take_cache(c, &k);
  if (st != PARIS_OK) return st;
  cudaError_t e = cudaDeviceSynchronize();
  uint32_t w = 0;
  if (e == cudaSuccess) e = cudaMemcpy(&w, k.status, sizeof w, cudaMemcpyDeviceToHost);
  if (e == cudaSuccess && w) e = cudaMemset(k.status, 0, sizeof w);
  if (e != cudaSuccess) return launched(e, "paris_kv4_check");
  if (w) return fail(PARIS_EDEVICE, "device status word 0x%x (bit 0: tokens dropped, the cache was full)", w);
  return PARIS_OK;
}

}  // extern "C"
