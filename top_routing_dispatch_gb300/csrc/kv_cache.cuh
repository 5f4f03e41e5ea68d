// Key-value caches: the checked description shared by the append and the
// attention, and the launchers of their kernels.
#pragma once

#include "common.cuh"

namespace moe {

constexpr int kMaxSeqs = 65536;

// The launchers below are given descriptions that passed check_cache
// (decode_api.cu); every field is as in moe_kv_cache_t.
using KVCache = moe_kv_cache_t;

// ---- kv_append.cu
cudaError_t launch_kv_append(const KVCache &c, int n, const void *q, long long q_stride,
                             const void *k, long long k_stride, const void *v, long long v_stride,
                             const int32_t *seq_ids, const int32_t *positions, void *q_out,
                             int32_t *status, cudaStream_t s);

// ---- paged_attention.cu
size_t paged_attention_ws_bytes(const KVCache &c);
cudaError_t launch_paged_attention(const KVCache &c, const void *q, long long q_stride,
                                   const int32_t *seq_lens, int window, float scale, void *out,
                                   float *lse, void *ws, int32_t *status, cudaStream_t s);

}  // namespace moe
