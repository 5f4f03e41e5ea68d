// Launchers of the experts on 4-bit weights (experts_w4.cu).
#pragma once

#include "common.cuh"

namespace moe {

constexpr int kW4MaxPairs = 4096;

// w (E, rows, cols) bf16 -> codes and scales by column
cudaError_t launch_quantize_w4(int E, int rows, int cols, int group, const void *w, int32_t *q,
                               void *scales, cudaStream_t s);
// codes and scales of w13 (which 0) or w2 (which 1) -> records
size_t w4_tiled_bytes(const Desc &d, int group, int which);
cudaError_t launch_prepare_w4(const Desc &d, int group, int which, const int32_t *q,
                              const void *scales, void *tiled, cudaStream_t s);
size_t experts_w4_ws_bytes(const Desc &d);
cudaError_t launch_experts_w4(const Desc &d, int group, const void *x, const int32_t *topk_idx,
                              const float *topk_w, const void *w13_t, const void *w2_t, void *y,
                              void *ws, int32_t *status, cudaStream_t s);

}  // namespace moe
