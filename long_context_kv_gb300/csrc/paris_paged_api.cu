// C ABI of the paged cache (include/paris.h): argument checks and launches.
#include <algorithm>

#include "api_checks.cuh"
#include "paged_internal.cuh"

using namespace paris;

namespace {

// Strides of an axis of more than one entry have to be positive multiples of
// 16 bytes; those of an axis of one entry mean nothing and are replaced.
paris_status take_page_strides(const paris_paged& c, const paris_page_strides& s, const char* name, PageStrides* out) {
  const int size = c.dtype == PARIS_BF16 ? 2 : 1;
  const struct { int64_t stride, n; const char* axis; int64_t* to; } axes[4] = {
      {s.layer, c.n_layers, "layer", &out->layer}, {s.page, c.n_pages, "page", &out->page},
      {s.head, c.n_kv_heads, "head", &out->head}, {s.row, c.page_rows, "row", &out->row}};
  for (const auto& x : axes) {
    if (x.n <= 1) {
      *x.to = kDim * size;
      continue;
    }
    if (x.stride < kDim || x.stride % (16 / size) || x.stride >= (int64_t)1 << 38)
      return fail(PARIS_EINVAL, "%s: the %s stride must be a multiple of %d elements, from %d to below 2^38 (got %lld)", name,
                  x.axis, 16 / size, kDim, (long long)x.stride);
    *x.to = x.stride * size;
  }
  return PARIS_OK;
}

paris_status take_paged(const paris_paged* c, Paged* k) {
  if (!c) return fail(PARIS_EINVAL, "the cache must not be NULL");
  if (c->head_dim != kDim) return fail(PARIS_EINVAL, "supported geometry: head_dim = %d (got %d)", kDim, c->head_dim);
  if (c->n_seqs < 1 || c->n_seqs > kMaxPagedSeqs || c->n_kv_heads < 1 || (int64_t)c->n_seqs * c->n_kv_heads > 65535)
    return fail(PARIS_EINVAL, "n_seqs must be in [1, %d], n_kv_heads positive, and their product at most 65535", kMaxPagedSeqs);
  if (c->n_layers < 1 || c->n_layers > 65535) return fail(PARIS_EINVAL, "n_layers must be in [1, 65535]");
  int shift = 4;
  while (shift < 8 && 1 << shift != c->page_rows) ++shift;
  if (1 << shift != c->page_rows) return fail(PARIS_EINVAL, "page_rows must be a power of two from 16 to 256 (got %d)", c->page_rows);
  if (c->dtype != PARIS_BF16 && c->dtype != PARIS_E4M3) return fail(PARIS_EINVAL, "the cache's dtype must be PARIS_BF16 or PARIS_E4M3");
  if (c->n_pages < 1 || c->n_pages > (int64_t)1 << kMaxPagesLog)
    return fail(PARIS_EINVAL, "n_pages must be in [1, 2^%d]", kMaxPagesLog);
  // rows past a sequence's end, up to 32 tiles of them, still have 32-bit numbers
  if (c->max_pages < 1 || c->max_pages > ((int64_t)1 << 30) / c->page_rows)
    return fail(PARIS_EINVAL, "max_pages must be positive, and max_pages * page_rows at most 2^30");
  if (c->n_seqs * c->max_pages * c->page_rows > (int64_t)1 << 37)
    return fail(PARIS_EINVAL, "n_seqs * max_pages * page_rows must be at most 2^37");
  const bool e4m3 = c->dtype == PARIS_E4M3;
  if (!c->k_pages || !c->v_pages || !c->table || !c->lens || !c->starts || !c->refs || !c->free_bits || !c->n_used || !c->status ||
      (e4m3 && (!c->k_scales || !c->v_scales)))
    return fail(PARIS_EINVAL, "the cache's arrays must not be NULL");
  if (!aligned16(c->k_pages) || !aligned16(c->v_pages) || (e4m3 && (!aligned16(c->k_scales) || !aligned16(c->v_scales))))
    return fail(PARIS_EINVAL, "the cache's pages and scales must be 16-byte aligned");
  *k = Paged{c->n_seqs, c->n_layers, c->n_kv_heads, e4m3 ? 1 : 0, shift, (int)c->n_pages, (int)c->max_pages,
             static_cast<uint8_t*>(c->k_pages), static_cast<uint8_t*>(c->v_pages), {}, {}, c->k_scales, c->v_scales,
             c->table, c->lens, c->starts, c->refs, c->free_bits, c->n_used, c->status};
  paris_status st = take_page_strides(*c, c->k, "k_pages", &k->sk);
  if (st == PARIS_OK) st = take_page_strides(*c, c->v, "v_pages", &k->sv);
  return st;
}

paris_status check_layer(const Paged& c, int layer) {
  return layer >= 0 && layer < c.layers ? PARIS_OK : fail(PARIS_EINVAL, "layer must be in [0, %d) (got %d)", c.layers, layer);
}

// The rows of a store or read call; nothing to do if max_rows comes out as 0.
paris_status take_rows(const paris_paged* c, int layer, const void* k, const void* v, paris_dtype dtype, const paris_strides* ks,
                       const paris_strides* vs, int64_t rows, const int32_t* cu, int64_t max_rows, PagedRows* a) {
  paris_status st = take_paged(c, &a->c);
  if (st == PARIS_OK) st = check_layer(a->c, layer);
  if (st == PARIS_OK) st = check_dtype(dtype);
  if (st != PARIS_OK) return st;
  if (!ks || !vs) return fail(PARIS_EINVAL, "the strides must not be NULL");
  if (rows < 0 || rows > 0x7fffffff || max_rows < 0) return fail(PARIS_EINVAL, "rows must be in [0, 2^31 - 1], the most rows of a sequence >= 0");
  const int seqs = cu ? 1 : a->c.n_seqs;
  st = take_strides(*ks, rows, a->c.hkv, seqs, "k", &a->ks);
  if (st == PARIS_OK) st = take_strides(*vs, rows, a->c.hkv, seqs, "v", &a->vs);
  if (st != PARIS_OK) return st;
  a->layer = layer;
  a->dtype = dtype;
  a->rows = rows;
  a->max_rows = std::min(max_rows, rows);
  a->cu = cu;
  if (a->max_rows == 0) return PARIS_OK;
  if (!k || !v) return fail(PARIS_EINVAL, "k and v must not be NULL");
  if (!aligned16(k) || !aligned16(v)) return fail(PARIS_EINVAL, "k and v must be 16-byte aligned");
  a->k = static_cast<uint8_t*>(const_cast<void*>(k));
  a->v = static_cast<uint8_t*>(const_cast<void*>(v));
  return PARIS_OK;
}

paris_status check_paged_heads(const Paged& c, int hq) {
  if (hq < c.hkv || hq % c.hkv || hq / c.hkv > 128)
    return fail(PARIS_EINVAL, "n_q_heads must be a positive multiple of n_kv_heads, at most 128 per KV head (got %d, %d)", hq, c.hkv);
  return PARIS_OK;
}

constexpr size_t kCounterBytes = 16;

size_t fork_bytes(const Paged& c, int n) { return (size_t)n * sizeof(ForkEntry) + (size_t)n * c.width * sizeof(int32_t); }
size_t compact_bytes(const Paged& c) { return 16 + 3 * (size_t)c.n_pages * sizeof(int32_t); }

paris_status fork(const paris_paged* c, const int32_t* src, const int32_t* dst, const int32_t* rows, int n, int zero,
                  void* workspace, size_t workspace_bytes, void* stream, const char* what) {
  ForkArgs a{};
  const paris_status st = take_paged(c, &a.c);
  if (st != PARIS_OK) return st;
  if (n < 0 || n > a.c.n_seqs) return fail(PARIS_EINVAL, "%s: n must be in [0, n_seqs] (got %d)", what, n);
  if (n == 0) return PARIS_OK;
  if (!src || !dst) return fail(PARIS_EINVAL, "%s: the sequences must not be NULL", what);
  const size_t need = zero && !rows ? 0 : fork_bytes(a.c, n);  // sequences that end need none
  if (need > 0 && (!workspace || workspace_bytes < need || !aligned16(workspace)))
    return fail(PARIS_EINVAL, "%s: needs %zu bytes of 16-byte aligned workspace (got %zu)", what, need, workspace ? workspace_bytes : (size_t)0);
  a.src = src;
  a.dst = dst;
  a.rows = rows;
  a.n = n;
  a.zero = zero;
  if (need > 0) {
    a.plan = static_cast<ForkEntry*>(workspace);
    a.entries = reinterpret_cast<int32_t*>(a.plan + n);
  }
  return launched(launch_paged_fork(a, static_cast<cudaStream_t>(stream)), what);
}

}  // namespace

extern "C" {

paris_status paris_paged_grow(const paris_paged* c, const int32_t* tokens, void* stream) {
  Paged k;
  const paris_status st = take_paged(c, &k);
  if (st != PARIS_OK) return st;
  if (!tokens) return fail(PARIS_EINVAL, "tokens must not be NULL");
  return launched(launch_paged_grow(k, tokens, static_cast<cudaStream_t>(stream)), "paris_paged_grow");
}

paris_status paris_paged_store(const paris_paged* c, int layer, const void* k, const void* v, paris_dtype dtype,
                               const paris_strides* ks, const paris_strides* vs, int64_t rows, const int32_t* cu,
                               int64_t max_new, void* stream) {
  PagedRows a{};
  const paris_status st = take_rows(c, layer, k, v, dtype, ks, vs, rows, cu, max_new, &a);
  if (st != PARIS_OK || a.max_rows == 0) return st;
  return launched(launch_paged_store(a, sm_count(), static_cast<cudaStream_t>(stream)), "paris_paged_store");
}

paris_status paris_paged_read(const paris_paged* c, int layer, void* k_out, void* v_out, const paris_strides* ks,
                              const paris_strides* vs, int64_t rows, const int32_t* cu, int64_t max_rows, void* stream) {
  PagedRows a{};
  const paris_status st = take_rows(c, layer, k_out, v_out, PARIS_BF16, ks, vs, rows, cu, max_rows, &a);
  if (st != PARIS_OK || a.max_rows == 0) return st;
  return launched(launch_paged_read(a, sm_count(), static_cast<cudaStream_t>(stream)), "paris_paged_read");
}

paris_status paris_paged_attend_workspace(const paris_paged* c, int n_q_heads, size_t* bytes, size_t* counter_bytes) {
  Paged k;
  if (!bytes || !counter_bytes) return fail(PARIS_EINVAL, "bytes and counter_bytes must not be NULL");
  paris_status st = take_paged(c, &k);
  if (st == PARIS_OK) st = check_paged_heads(k, n_q_heads);
  if (st != PARIS_OK) return st;
  *bytes = paged_attend_plan(k, n_q_heads, sm_count()).bytes;
  *counter_bytes = kCounterBytes;
  return PARIS_OK;
}

paris_status paris_paged_attend(const paris_paged* c, int layer, const void* q, int n_q_heads, int64_t window,
                                void* out_bf16, float* lse, void* workspace, size_t workspace_bytes, uint32_t* counters,
                                size_t counter_bytes, void* stream) {
  PagedAttendArgs a{};
  paris_status st = take_paged(c, &a.c);
  if (st == PARIS_OK) st = check_layer(a.c, layer);
  if (st == PARIS_OK) st = check_paged_heads(a.c, n_q_heads);
  if (st != PARIS_OK) return st;
  if (window < 0) return fail(PARIS_EINVAL, "window must be >= 0 (got %lld)", (long long)window);
  if (!q || !out_bf16) return fail(PARIS_EINVAL, "q and out must not be NULL");
  if (!aligned16(q) || !aligned16(out_bf16)) return fail(PARIS_EINVAL, "q and out must be 16-byte aligned");
  const PagedAttendPlan p = paged_attend_plan(a.c, n_q_heads, sm_count());
  if (!workspace || workspace_bytes < p.bytes || !aligned16(workspace) || !counters || counter_bytes < kCounterBytes || !aligned16(counters))
    return fail(PARIS_EINVAL, "paris_paged_attend: needs %zu bytes of workspace and %zu of counters, 16-byte aligned (got %zu, %zu)",
                p.bytes, kCounterBytes, workspace ? workspace_bytes : (size_t)0, counters ? counter_bytes : (size_t)0);
  a.layer = layer;
  a.hq = n_q_heads;
  a.window = window > 0x7fffffff ? 0 : (int)window;
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.out = static_cast<__nv_bfloat16*>(out_bf16);
  a.lse = lse;
  a.g = n_q_heads / a.c.hkv;
  a.groups = p.groups;
  a.nblocks = p.blocks;
  a.slots = p.slots;
  a.max_splits = p.max_splits;
  a.part = static_cast<float*>(workspace);
  a.splits = reinterpret_cast<PgSplit*>(static_cast<uint8_t*>(workspace) + p.part_bytes);
  a.counts = counters;
  return launched(launch_paged_attend(a, static_cast<cudaStream_t>(stream)), "paris_paged_attend");
}

paris_status paris_paged_fork_workspace(const paris_paged* c, int n, size_t* bytes) {
  Paged k;
  if (!bytes) return fail(PARIS_EINVAL, "bytes must not be NULL");
  const paris_status st = take_paged(c, &k);
  if (st != PARIS_OK) return st;
  if (n < 0 || n > k.n_seqs) return fail(PARIS_EINVAL, "n must be in [0, n_seqs] (got %d)", n);
  *bytes = fork_bytes(k, n);
  return PARIS_OK;
}

paris_status paris_paged_fork(const paris_paged* c, const int32_t* src, const int32_t* dst, const int32_t* rows, int n,
                              void* workspace, size_t workspace_bytes, void* stream) {
  return fork(c, src, dst, rows, n, 0, workspace, workspace_bytes, stream, "paris_paged_fork");
}

paris_status paris_paged_free(const paris_paged* c, const int32_t* seqs, const int32_t* rows, int n, void* workspace,
                              size_t workspace_bytes, void* stream) {
  return fork(c, seqs, seqs, rows, n, 1, workspace, workspace_bytes, stream, "paris_paged_free");
}

paris_status paris_paged_compact_workspace(const paris_paged* c, size_t* bytes) {
  Paged k;
  if (!bytes) return fail(PARIS_EINVAL, "bytes must not be NULL");
  const paris_status st = take_paged(c, &k);
  if (st != PARIS_OK) return st;
  *bytes = compact_bytes(k);
  return PARIS_OK;
}

paris_status paris_paged_compact(const paris_paged* c, void* workspace, size_t workspace_bytes, void* stream) {
  CompactArgs a{};
  const paris_status st = take_paged(c, &a.c);
  if (st != PARIS_OK) return st;
  const size_t need = compact_bytes(a.c);
  if (!workspace || workspace_bytes < need || !aligned16(workspace))
    return fail(PARIS_EINVAL, "paris_paged_compact: needs %zu bytes of 16-byte aligned workspace (got %zu)", need,
                workspace ? workspace_bytes : (size_t)0);
  a.moves = static_cast<int32_t*>(workspace);
  a.from = a.moves + 4;
  a.to = a.from + a.c.n_pages;
  a.rank = a.to + a.c.n_pages;
  return launched(launch_paged_compact(a, sm_count(), static_cast<cudaStream_t>(stream)), "paris_paged_compact");
}

paris_status paris_paged_check(const paris_paged* c) {
  Paged k;
  const paris_status st = take_paged(c, &k);
  if (st != PARIS_OK) return st;
  cudaError_t e = cudaDeviceSynchronize();
  uint32_t w = 0, gave_up = 0;
  if (e == cudaSuccess) e = cudaMemcpy(&w, k.status, sizeof w, cudaMemcpyDeviceToHost);
  if (e == cudaSuccess && w) e = cudaMemset(k.status, 0, sizeof w);
  if (e == cudaSuccess) e = paged_attend_error(&gave_up);
  if (e != cudaSuccess) return launched(e, "paris_paged_check");
  if (gave_up) return fail(PARIS_EDEVICE, "paris_paged_attend gave up waiting for its copies: its results are not valid");
  if (w) return fail(PARIS_EDEVICE, "device status word 0x%x (bit 0: no room for rows or pages; bit 1: a sequence out of range)", w);
  return PARIS_OK;
}

}  // extern "C"
