// Host side of the paged cache's entry points: argument validation, buffer
// sizes and dispatch.  Every check runs before any launch.
#include "hyq_paged.cuh"

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
bool int32s(const void* p) { return p && aligned(p, 4); }

hyq_status from_cuda(cudaError_t e) { return e == cudaSuccess ? HYQ_OK : HYQ_ERR_CUDA; }

// The config and the four sizes of a pool.
hyq_status sizes_ok(const hyq_config* c, const hyq_pages* p) {
  const hyq_status st = hyq_config_check(c);
  if (st != HYQ_OK) return st;
  if (!p || p->n_layers < 1 || p->n_layers > 65535 || p->n_pages < 1 || p->n_pages > HYQ_PAGED_MAX_PAGES ||
      p->n_seqs < 1 || p->n_seqs > (1 << 24) || p->max_blocks < 1 || p->max_blocks > HYQ_PAGED_MAX_BLOCKS)
    return HYQ_ERR_INVALID_ARG;
  return HYQ_OK;
}

hyq_status pages_ok(const hyq_config* c, const hyq_pages* p) {
  const hyq_status st = sizes_ok(c, p);
  if (st != HYQ_OK) return st;
  const void* ps[] = {p->pool, p->bounds, p->table, p->lens, p->refs, p->err};
  for (const void* x : ps)
    if (!x || !aligned(x, 256)) return HYQ_ERR_INVALID_ARG;
  return HYQ_OK;
}

// The arguments that every call on one layer shares.
hyq_status call_ok(const hyq_config* c, const hyq_pages* p, int32_t layer, const int32_t* seqs, int32_t batch) {
  const hyq_status st = pages_ok(c, p);
  if (st != HYQ_OK) return st;
  if (layer < 0 || layer >= p->n_layers || batch < 0 || (seqs && !aligned(seqs, 4))) return HYQ_ERR_INVALID_ARG;
  if (batch > HYQ_PAGED_MAX_BATCH) return HYQ_ERR_UNSUPPORTED;
  return HYQ_OK;
}

hyq_status queries_ok(const hyq_config* c, int32_t n_q, const void* q, int64_t ldq) {
  if (n_q < 1 || !q || !aligned(q, 16)) return HYQ_ERR_INVALID_ARG;
  if (ldq < (int64_t)c->num_q_heads * HYQ_D || ldq % 8) return HYQ_ERR_INVALID_ARG;
  if (n_q > HYQ_PAGED_MAX_Q || (int64_t)n_q * c->num_kv_heads > 65535) return HYQ_ERR_UNSUPPORTED;
  return HYQ_OK;
}

bool ws_ok(const void* ws, size_t have, size_t need) { return ws && aligned(ws, 256) && have >= need; }

}  // namespace

extern "C" hyq_status hyq_pages_sizes(const hyq_config* c, const hyq_pages* p, size_t* out) {
  const hyq_status st = sizes_ok(c, p);
  if (st != HYQ_OK) return st;
  if (!out) return HYQ_ERR_INVALID_ARG;
  const size_t blocks = (size_t)p->n_layers * p->n_pages * c->num_kv_heads;
  out[0] = hyq_align256(blocks * hyq_qblock_bytes(c));
  out[1] = hyq_align256(blocks * HYQ_BOUND_BYTES);
  out[2] = hyq_align256((size_t)p->n_seqs * p->max_blocks * 4);
  out[3] = hyq_align256((size_t)p->n_seqs * 4);
  out[4] = hyq_align256((size_t)p->n_pages * 4);
  out[5] = hyq_align256(4);
  return HYQ_OK;
}

extern "C" size_t hyq_pages_workspace_size(const hyq_config* c, const hyq_pages* p, int op, int32_t batch,
                                           int32_t n_q) {
  if (sizes_ok(c, p) != HYQ_OK || batch < 1 || batch > HYQ_PAGED_MAX_BATCH) return 0;
  const bool q_ok = n_q >= 1 && n_q <= HYQ_PAGED_MAX_Q;
  switch (op) {
    case HYQ_OP_PAGED_ATTENTION: return q_ok ? hyq_paged_attention_ws_bytes(c, batch, n_q) : 0;
    case HYQ_OP_PAGED_SELECT: return q_ok ? hyq_paged_select_ws_bytes(c, p, batch, n_q) : 0;
    case HYQ_OP_PAGES_RESERVE: return hyq_pages_reserve_ws_bytes(p);
    case HYQ_OP_PAGES_COMPACT: return hyq_pages_compact_ws_bytes(p);
    case HYQ_OP_PAGED_SHARED: return q_ok ? hyq_paged_shared_ws_bytes(c, batch, n_q) : 0;
    case HYQ_OP_PAGED_CROSS: return hyq_paged_cross_ws_bytes(c, batch);
    case HYQ_OP_PAGES_EVICT: return hyq_pages_evict_ws_bytes(c, p, batch);
    default: return 0;
  }
}

extern "C" hyq_status hyq_pages_reset(const hyq_config* c, const hyq_pages* p, hyq_stream_t s) {
  const hyq_status st = pages_ok(c, p);
  if (st != HYQ_OK) return st;
  cudaError_t e = cudaMemsetAsync(p->lens, 0, (size_t)p->n_seqs * 4, s);
  if (e == cudaSuccess) e = cudaMemsetAsync(p->refs, 0, (size_t)p->n_pages * 4, s);
  if (e == cudaSuccess) e = cudaMemsetAsync(p->err, 0, 4, s);
  return from_cuda(e);
}

extern "C" hyq_status hyq_pages_reserve(const hyq_config* c, const hyq_pages* p, const int32_t* seqs, int32_t batch,
                                        const int32_t* n_new, void* ws, size_t ws_bytes, hyq_stream_t s) {
  const hyq_status st = call_ok(c, p, 0, seqs, batch);
  if (st != HYQ_OK) return st;
  if ((!seqs && batch > p->n_seqs) || (n_new && !aligned(n_new, 4))) return HYQ_ERR_INVALID_ARG;
  if (batch == 0) return HYQ_OK;
  if (!ws_ok(ws, ws_bytes, hyq_pages_reserve_ws_bytes(p))) return HYQ_ERR_WORKSPACE;
  return from_cuda(hyq_launch_pages_reserve(c, p, seqs, batch, n_new, ws, s));
}

extern "C" hyq_status hyq_pages_fork(const hyq_config* c, const hyq_pages* p, const int32_t* src, const int32_t* dst,
                                     int32_t n, hyq_stream_t s) {
  const hyq_status st = call_ok(c, p, 0, nullptr, n);
  if (st != HYQ_OK) return st;
  if (n == 0) return HYQ_OK;
  if (!int32s(src) || !int32s(dst)) return HYQ_ERR_INVALID_ARG;
  return from_cuda(hyq_launch_pages_fork(p, src, dst, n, s));
}

extern "C" hyq_status hyq_pages_truncate(const hyq_config* c, const hyq_pages* p, const int32_t* seqs,
                                         const int32_t* new_lens, int32_t n, hyq_stream_t s) {
  // without a list nothing is looked for in it: all rows of any table
  const hyq_status st = call_ok(c, p, 0, seqs, seqs || n < 0 ? n : 0);
  if (st != HYQ_OK) return st;
  if ((!seqs && n > p->n_seqs) || (new_lens && !aligned(new_lens, 4))) return HYQ_ERR_INVALID_ARG;
  if (n == 0) return HYQ_OK;
  return from_cuda(hyq_launch_pages_truncate(p, seqs, new_lens, n, s));
}

extern "C" hyq_status hyq_pages_compact(const hyq_config* c, const hyq_pages* p, int32_t* table_out,
                                        int32_t* refs_out, void* ws, size_t ws_bytes, hyq_stream_t s) {
  const hyq_status st = pages_ok(c, p);
  if (st != HYQ_OK) return st;
  if ((table_out && !aligned(table_out, 4)) || (refs_out && !aligned(refs_out, 4))) return HYQ_ERR_INVALID_ARG;
  if (!ws_ok(ws, ws_bytes, hyq_pages_compact_ws_bytes(p))) return HYQ_ERR_WORKSPACE;
  return from_cuda(hyq_launch_pages_compact(c, p, table_out, refs_out, ws, s));
}

extern "C" hyq_status hyq_paged_append(const hyq_config* c, const hyq_pages* p, int32_t layer, const int32_t* seqs,
                                       int32_t batch, const int32_t* cu_rows, int32_t n_rows, const void* k_rows,
                                       const void* v_rows, int64_t ld, void* k_hat, void* v_hat, hyq_stream_t s) {
  const hyq_status st = call_ok(c, p, layer, seqs, batch);
  if (st != HYQ_OK) return st;
  if (n_rows < 0 || (cu_rows ? !aligned(cu_rows, 4) : n_rows != batch)) return HYQ_ERR_INVALID_ARG;
  if (!seqs && batch > p->n_seqs) return HYQ_ERR_INVALID_ARG;
  if (batch == 0 || n_rows == 0) return HYQ_OK;
  if (!k_rows || !v_rows || !aligned(k_rows, 16) || !aligned(v_rows, 16)) return HYQ_ERR_INVALID_ARG;
  if (ld < (int64_t)c->num_kv_heads * HYQ_D || ld % 8) return HYQ_ERR_INVALID_ARG;
  if ((k_hat == nullptr) != (v_hat == nullptr) || !aligned(k_hat, 16) || !aligned(v_hat, 16))
    return HYQ_ERR_INVALID_ARG;
  return from_cuda(hyq_launch_paged_append(c, hyq_page_view(c, p, layer), seqs, batch, cu_rows, n_rows, k_rows, v_rows,
                                           ld, k_hat, v_hat, s));
}

extern "C" hyq_status hyq_paged_attention_lse(const hyq_config* c, const hyq_pages* p, int32_t layer,
                                              const int32_t* seqs, int32_t batch, int32_t n_q, const void* q,
                                              int64_t ldq, void* out, float* lse, void* ws, size_t ws_bytes,
                                              hyq_stream_t s) {
  hyq_status st = call_ok(c, p, layer, seqs, batch);
  if (st != HYQ_OK) return st;
  if (!seqs && batch > p->n_seqs) return HYQ_ERR_INVALID_ARG;
  if (batch == 0) return HYQ_OK;
  st = queries_ok(c, n_q, q, ldq);
  if (st != HYQ_OK) return st;
  if (!out || !aligned(out, 16) || !aligned(lse, 4)) return HYQ_ERR_INVALID_ARG;
  if (!ws_ok(ws, ws_bytes, hyq_paged_attention_ws_bytes(c, batch, n_q))) return HYQ_ERR_WORKSPACE;
  return from_cuda(hyq_launch_paged_attention(c, hyq_page_view(c, p, layer), seqs, batch, n_q, q, ldq, nullptr, 0, out,
                                              lse, nullptr, nullptr, ws, s));
}

extern "C" hyq_status hyq_paged_attention(const hyq_config* c, const hyq_pages* p, int32_t layer, const int32_t* seqs,
                                          int32_t batch, int32_t n_q, const void* q, int64_t ldq, void* out, void* ws,
                                          size_t ws_bytes, hyq_stream_t s) {
  return hyq_paged_attention_lse(c, p, layer, seqs, batch, n_q, q, ldq, out, nullptr, ws, ws_bytes, s);
}

extern "C" hyq_status hyq_paged_attention_shared(const hyq_config* c, const hyq_pages* p, int32_t layer,
                                                 const int32_t* seqs, int32_t batch, int32_t n_q,
                                                 const int32_t* cu_groups, const int32_t* n_shared, int32_t n_groups,
                                                 const void* q, int64_t ldq, void* out, void* ws, size_t ws_bytes,
                                                 hyq_stream_t s) {
  hyq_status st = call_ok(c, p, layer, seqs, batch);
  if (st != HYQ_OK) return st;
  if ((!seqs && batch > p->n_seqs) || n_groups < 0) return HYQ_ERR_INVALID_ARG;
  if (n_groups > HYQ_PAGED_MAX_BATCH) return HYQ_ERR_UNSUPPORTED;
  if (batch == 0) return HYQ_OK;
  st = queries_ok(c, n_q, q, ldq);
  if (st != HYQ_OK) return st;
  if (!out || !aligned(out, 16) || (n_groups && (!int32s(cu_groups) || !int32s(n_shared)))) return HYQ_ERR_INVALID_ARG;
  if (!ws_ok(ws, ws_bytes, hyq_paged_shared_ws_bytes(c, batch, n_q))) return HYQ_ERR_WORKSPACE;
  return from_cuda(hyq_launch_paged_shared(c, hyq_page_view(c, p, layer), seqs, batch, n_q,
                                           SharedRows{cu_groups, n_shared, n_groups}, q, ldq, out, ws, s));
}

extern "C" hyq_status hyq_paged_cross_attention(const hyq_config* c, const hyq_pages* p, int32_t layer,
                                                const int32_t* seqs, int32_t batch, const int32_t* cu_q,
                                                int32_t n_tokens, const void* q, int64_t ldq, void* out, void* ws,
                                                size_t ws_bytes, hyq_stream_t s) {
  hyq_status st = call_ok(c, p, layer, seqs, batch);
  if (st != HYQ_OK) return st;
  if (!seqs && batch > p->n_seqs) return HYQ_ERR_INVALID_ARG;
  if (n_tokens < 0 || (cu_q ? !aligned(cu_q, 4) : n_tokens != batch)) return HYQ_ERR_INVALID_ARG;
  if (batch == 0 || n_tokens == 0) return HYQ_OK;
  st = queries_ok(c, 1, q, ldq);
  if (st != HYQ_OK) return st;
  if (!out || !aligned(out, 16)) return HYQ_ERR_INVALID_ARG;
  if ((int64_t)n_tokens * c->num_q_heads > INT32_MAX) return HYQ_ERR_UNSUPPORTED;
  if (!ws_ok(ws, ws_bytes, hyq_paged_cross_ws_bytes(c, batch))) return HYQ_ERR_WORKSPACE;
  return from_cuda(
      hyq_launch_paged_cross(c, hyq_page_view(c, p, layer), seqs, batch, cu_q, n_tokens, q, ldq, out, ws, s));
}

extern "C" hyq_status hyq_paged_accumulate(const hyq_config* c, const hyq_pages* p, int32_t layer, const int32_t* seqs,
                                           int32_t batch, int32_t n_q, const void* q, int64_t ldq, const float* lse,
                                           const int32_t* n_new, float* mass, hyq_stream_t s) {
  hyq_status st = call_ok(c, p, layer, seqs, batch);
  if (st != HYQ_OK) return st;
  if (!seqs && batch > p->n_seqs) return HYQ_ERR_INVALID_ARG;
  if (batch == 0) return HYQ_OK;
  st = queries_ok(c, n_q, q, ldq);
  if (st != HYQ_OK) return st;
  if (!lse || !aligned(lse, 4) || !mass || !aligned(mass, 16) || !aligned(n_new, 4)) return HYQ_ERR_INVALID_ARG;
  float* mine = mass + (size_t)layer * p->n_pages * c->num_kv_heads * HYQ_PAGE_ROWS;
  return from_cuda(hyq_launch_paged_accumulate(c, hyq_page_view(c, p, layer), p->refs, seqs, batch, n_q, q, ldq, lse,
                                               n_new, mine, s));
}

extern "C" hyq_status hyq_pages_evict(const hyq_config* c, const hyq_pages* p, const int32_t* seqs, int32_t batch,
                                      const int32_t* keep, int32_t n_first, int32_t n_last, float* mass, void* ws,
                                      size_t ws_bytes, hyq_stream_t s) {
  const hyq_status st = call_ok(c, p, 0, seqs, batch);
  if (st != HYQ_OK) return st;
  if (!seqs && batch > p->n_seqs) return HYQ_ERR_INVALID_ARG;
  if (n_first < 0 || n_last < 0 || n_first > INT32_MAX - n_last) return HYQ_ERR_INVALID_ARG;
  if (batch == 0) return HYQ_OK;
  if (!int32s(keep) || !mass || !aligned(mass, 16)) return HYQ_ERR_INVALID_ARG;
  if (!ws_ok(ws, ws_bytes, hyq_pages_evict_ws_bytes(c, p, batch))) return HYQ_ERR_WORKSPACE;
  return from_cuda(hyq_launch_pages_evict(c, p, seqs, batch, keep, n_first, n_last, mass, ws, s));
}

extern "C" hyq_status hyq_paged_attention_blocks(const hyq_config* c, const hyq_pages* p, int32_t layer,
                                                 const int32_t* seqs, int32_t batch, int32_t n_q, const void* q,
                                                 int64_t ldq, const int32_t* sel, int32_t k, void* out, void* ws,
                                                 size_t ws_bytes, hyq_stream_t s) {
  hyq_status st = call_ok(c, p, layer, seqs, batch);
  if (st != HYQ_OK) return st;
  if (!seqs && batch > p->n_seqs) return HYQ_ERR_INVALID_ARG;
  if (batch == 0) return HYQ_OK;
  st = queries_ok(c, n_q, q, ldq);
  if (st != HYQ_OK) return st;
  if (!out || !aligned(out, 16) || !int32s(sel) || k < 1 || k > HYQ_PAGED_MAX_BLOCKS) return HYQ_ERR_INVALID_ARG;
  if (!ws_ok(ws, ws_bytes, hyq_paged_attention_ws_bytes(c, batch, n_q))) return HYQ_ERR_WORKSPACE;
  return from_cuda(
      hyq_launch_paged_attention(c, hyq_page_view(c, p, layer), seqs, batch, n_q, q, ldq, sel, k, out, nullptr, nullptr,
                                 nullptr, ws, s));
}

extern "C" hyq_status hyq_paged_select(const hyq_config* c, const hyq_pages* p, int32_t layer, const int32_t* seqs,
                                       int32_t batch, int32_t n_q, const void* q, int64_t ldq, int32_t k,
                                       int32_t n_first, int32_t n_last, int32_t* sel, void* ws, size_t ws_bytes,
                                       hyq_stream_t s) {
  hyq_status st = call_ok(c, p, layer, seqs, batch);
  if (st != HYQ_OK) return st;
  if (!seqs && batch > p->n_seqs) return HYQ_ERR_INVALID_ARG;
  if (batch == 0) return HYQ_OK;
  st = queries_ok(c, n_q, q, ldq);
  if (st != HYQ_OK) return st;
  if (!int32s(sel) || k < 1 || k > HYQ_PAGED_MAX_BLOCKS || n_first < 0 || n_last < 0 || n_first > k - n_last)
    return HYQ_ERR_INVALID_ARG;
  if (!ws_ok(ws, ws_bytes, hyq_paged_select_ws_bytes(c, p, batch, n_q))) return HYQ_ERR_WORKSPACE;
  return from_cuda(hyq_launch_paged_select(c, hyq_page_view(c, p, layer), seqs, batch, n_q, q, ldq, k, n_first,
                                           n_last, sel, ws, s));
}
