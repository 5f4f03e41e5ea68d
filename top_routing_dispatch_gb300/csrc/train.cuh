// Internal declarations of the training operators (layer norm, gradient norm,
// AdamW): norm.cu, adamw.cu, train_api.cu.
#pragma once

#include "common.cuh"

namespace moe {

// Lets a kernel have `bytes` of dynamic shared memory, once a device.
template <typename K>
inline cudaError_t allow_smem(K kernel, int bytes, bool (&ready)[64]) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  bool &r = ready[dev >= 0 && dev < 64 ? dev : 0];
  if (r) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) r = true;
  return e;
}

// launch_pdl of clusters of `size` CTAs
template <typename K, typename A>
inline cudaError_t launch_pdl_cluster(K kernel, int clusters, int size, int threads, int smem,
                                      cudaStream_t s, const A &a) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(clusters * size), cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem, cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = size;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr, cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

// ---- norm.cu, norm_backward.cu
constexpr int kNormMaxH = 1 << 20;  // longest row
size_t norm_backward_ws_bytes(const moe_norm_t &d);
cudaError_t launch_norm(const moe_norm_t &d, const void *x, long long x_stride,
                        const void *residual, long long residual_stride, const void *weight,
                        const void *bias, void *s, void *y, float *stats, cudaStream_t st);
cudaError_t launch_norm_backward(const moe_norm_t &d, const void *dy, long long dy_stride,
                                 const void *s, long long s_stride, const float *stats,
                                 const void *weight, const void *ds, long long ds_stride, void *dx,
                                 float *dweight, float *dbias, void *ws, cudaStream_t st);

// ---- adamw.cu
constexpr int kAdamBlock = 256;  // values of a tensor that share a scale
size_t grad_norm_ws_bytes(int count);
cudaError_t launch_grad_norm(const moe_tensor_t *t, int count, float max_norm, float *norm,
                             float *factor, void *ws, cudaStream_t s);
cudaError_t launch_adamw_set_steps(double beta1, double beta2, long long steps, void *state,
                                   cudaStream_t s);
cudaError_t launch_adamw(const moe_adamw_t &o, const moe_adamw_tensor_t *t, int count, void *state,
                         cudaStream_t s);

}  // namespace moe
