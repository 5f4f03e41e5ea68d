// C ABI of the serving calls (paged cache append, paged attention, experts on
// 4-bit weights): argument checks.  The kernels live in the other .cu files.
#include "experts_w4.cuh"
#include "kv_cache.cuh"

using namespace moe;

namespace {

inline bool aligned(const void *p, uintptr_t a) {
  return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}
inline moe_status_t cuda_status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

// Sizes and types of a cache; its pointers are looked at by check_memory.
moe_status_t check_cache(const moe_kv_cache_t *c) {
  if (!c) return MOE_ERR_INVALID_ARG;
  if (c->num_seqs < 0 || c->q_heads < 1 || c->kv_heads < 1 || c->head_dim < 1 ||
      c->page_size < 1 || c->num_pages < 0 || c->max_pages < 1)
    return MOE_ERR_INVALID_ARG;
  if (c->q_heads % c->kv_heads) return MOE_ERR_INVALID_ARG;
  if (c->dtype != MOE_F32 && c->dtype != MOE_BF16) return MOE_ERR_INVALID_ARG;
  if (c->cache_dtype != c->dtype && !(c->cache_dtype == MOE_E4M3 && c->dtype == MOE_BF16))
    return MOE_ERR_INVALID_ARG;
  if (c->cache_dtype != MOE_E4M3 && (c->k_scale || c->v_scale)) return MOE_ERR_INVALID_ARG;
  if (c->rope_dim < 0 || c->rope_rows < 0 || c->rope_dim > c->head_dim) return MOE_ERR_INVALID_ARG;
  if ((c->rope != nullptr) != (c->rope_dim > 0)) return MOE_ERR_INVALID_ARG;
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return MOE_ERR_UNSUPPORTED;
  if (c->page_size % 16 || c->rope_dim % 16) return MOE_ERR_UNSUPPORTED;
  if (c->num_seqs > kMaxSeqs || c->q_heads > 65536) return MOE_ERR_UNSUPPORTED;
  const long long page = (long long)c->kv_heads * c->page_size * c->head_dim;
  if (c->page_stride < page || page > 0x7fffffffll) return MOE_ERR_INVALID_ARG;
  if (c->page_stride % 16) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

moe_status_t check_memory(const moe_kv_cache_t *c) {
  if (!c->k_cache || !c->v_cache || !c->page_table) return MOE_ERR_INVALID_ARG;
  if (!aligned(c->k_cache, 16) || !aligned(c->v_cache, 16) || !aligned(c->rope, 16) ||
      !aligned(c->page_table, 4) || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4))
    return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

bool row_stride_ok(long long stride, int heads, int dim) {
  return stride >= (long long)heads * dim && stride % 8 == 0;
}

moe_status_t check_w4(const moe_layer_desc_t *desc, int group, Desc *d) {
  moe_status_t st = check_desc(desc, d);
  if (st != MOE_OK) return st;
  if (group != 32 && group != 64 && group != 128) return MOE_ERR_UNSUPPORTED;
  if (!d->bf16 || d->H % 128 || d->I % 128) return MOE_ERR_UNSUPPORTED;
  if (d->I > 0x7fffffff / 2) return MOE_ERR_UNSUPPORTED;  // w13's 2 I columns are an int
  return MOE_OK;
}

}  // namespace

extern "C" {

moe_status_t moe_kv_append(const moe_kv_cache_t *cache, int32_t n, const void *q,
                           int64_t q_stride, const void *k, int64_t k_stride, const void *v,
                           int64_t v_stride, const int32_t *seq_ids, const int32_t *positions,
                           void *q_out, int32_t *status_word, moe_stream_t stream) {
  moe_status_t st = check_cache(cache);
  if (st != MOE_OK) return st;
  if (n < 0) return MOE_ERR_INVALID_ARG;
  if (n == 0) return MOE_OK;
  st = check_memory(cache);
  if (st != MOE_OK) return st;
  if (!k || !v || !seq_ids || !positions || (q != nullptr) != (q_out != nullptr))
    return MOE_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(q_out, 16) ||
      !aligned(seq_ids, 4) || !aligned(positions, 4))
    return MOE_ERR_INVALID_ARG;
  const int D = cache->head_dim;
  // strides matter from the second token on
  if (n > 1 && ((q && !row_stride_ok(q_stride, cache->q_heads, D)) ||
                !row_stride_ok(k_stride, cache->kv_heads, D) ||
                !row_stride_ok(v_stride, cache->kv_heads, D)))
    return MOE_ERR_INVALID_ARG;
  if (q && q == q_out && n > 1 && q_stride != (long long)cache->q_heads * D)
    return MOE_ERR_INVALID_ARG;
  return cuda_status(launch_kv_append(*cache, n, q, q_stride, k, k_stride, v, v_stride, seq_ids,
                                      positions, q_out, status_word, stream));
}

size_t moe_paged_attention_workspace_size(const moe_kv_cache_t *cache) {
  if (check_cache(cache) != MOE_OK) return 0;
  return paged_attention_ws_bytes(*cache);
}

moe_status_t moe_paged_attention(const moe_kv_cache_t *cache, const void *q, int64_t q_stride,
                                 const int32_t *seq_lens, int32_t window, float scale, void *out,
                                 float *lse, void *ws, size_t ws_bytes, int32_t *status_word,
                                 moe_stream_t stream) {
  moe_status_t st = check_cache(cache);
  if (st != MOE_OK) return st;
  if (window < 0 || !(scale > 0.f) || scale > 3.4e38f) return MOE_ERR_INVALID_ARG;
  if (cache->num_seqs == 0) return MOE_OK;
  st = check_memory(cache);
  if (st != MOE_OK) return st;
  if (!q || !seq_lens || !out || !ws) return MOE_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(lse, 4) || !aligned(seq_lens, 4) ||
      !aligned(ws, 256))
    return MOE_ERR_INVALID_ARG;
  if (cache->num_seqs > 1 && !row_stride_ok(q_stride, cache->q_heads, cache->head_dim))
    return MOE_ERR_INVALID_ARG;
  if (ws_bytes < paged_attention_ws_bytes(*cache)) return MOE_ERR_WORKSPACE;
  return cuda_status(launch_paged_attention(*cache, q, q_stride, seq_lens, window, scale, out, lse,
                                            ws, status_word, stream));
}

moe_status_t moe_quantize_weights_w4(const moe_layer_desc_t *desc, int group, const void *w13,
                                     const void *w2, int32_t *w13_q, void *w13_s, int32_t *w2_q,
                                     void *w2_s, moe_stream_t stream) {
  Desc d;
  moe_status_t st = check_w4(desc, group, &d);
  if (st != MOE_OK) return st;
  const void *ptrs[] = {w13, w2, w13_q, w13_s, w2_q, w2_s};
  for (const void *p : ptrs)
    if (!p || !aligned(p, 16)) return MOE_ERR_INVALID_ARG;
  cudaError_t e = launch_quantize_w4(d.E, d.H, 2 * d.I, group, w13, w13_q, w13_s, stream);
  if (e == cudaSuccess) e = launch_quantize_w4(d.E, d.I, d.H, group, w2, w2_q, w2_s, stream);
  return cuda_status(e);
}

size_t moe_experts_w4_workspace_size(const moe_layer_desc_t *desc) {
  Desc d;
  if (check_w4(desc, 128, &d) != MOE_OK || d.nK() > kW4MaxPairs) return 0;
  return experts_w4_ws_bytes(d);
}

size_t moe_w4_tiled_bytes(const moe_layer_desc_t *desc, int group, int which) {
  Desc d;
  if (check_w4(desc, group, &d) != MOE_OK || which < 0 || which > 1) return 0;
  return w4_tiled_bytes(d, group, which);
}

moe_status_t moe_prepare_weights_w4(const moe_layer_desc_t *desc, int group, const int32_t *w13_q,
                                    const void *w13_s, const int32_t *w2_q, const void *w2_s,
                                    void *w13_t, void *w2_t, moe_stream_t stream) {
  Desc d;
  moe_status_t st = check_w4(desc, group, &d);
  if (st != MOE_OK) return st;
  const void *ptrs[] = {w13_q, w13_s, w2_q, w2_s, w13_t, w2_t};
  for (const void *p : ptrs)
    if (!p || !aligned(p, 16)) return MOE_ERR_INVALID_ARG;
  cudaError_t e = launch_prepare_w4(d, group, 0, w13_q, w13_s, w13_t, stream);
  if (e == cudaSuccess) e = launch_prepare_w4(d, group, 1, w2_q, w2_s, w2_t, stream);
  return cuda_status(e);
}

moe_status_t moe_experts_w4(const moe_layer_desc_t *desc, int group, const void *x,
                            const int32_t *topk_idx, const float *topk_w, const void *w13_t,
                            const void *w2_t, void *y, void *ws, size_t ws_bytes,
                            int32_t *status_word, moe_stream_t stream) {
  Desc d;
  moe_status_t st = check_w4(desc, group, &d);
  if (st != MOE_OK) return st;
  if (d.nK() > kW4MaxPairs) return MOE_ERR_UNSUPPORTED;
  if (d.n == 0) return MOE_OK;
  const void *ptrs[] = {x, w13_t, w2_t, y};
  for (const void *p : ptrs)
    if (!p || !aligned(p, 16)) return MOE_ERR_INVALID_ARG;
  if (!topk_idx || !topk_w || !aligned(topk_idx, 4) || !aligned(topk_w, 4))
    return MOE_ERR_INVALID_ARG;
  if (!ws || !aligned(ws, 256)) return MOE_ERR_INVALID_ARG;
  if (ws_bytes < experts_w4_ws_bytes(d)) return MOE_ERR_WORKSPACE;
  return cuda_status(launch_experts_w4(d, group, x, topk_idx, topk_w, w13_t, w2_t, y, ws,
                                       status_word, stream));
}

}  // extern "C"
