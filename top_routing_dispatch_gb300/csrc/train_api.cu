// C ABI of the training calls (layer norm, gradient norm, AdamW): argument
// checks.  The kernels live in norm.cu and adamw.cu.
#include <math.h>

#include "train.cuh"

using namespace moe;

namespace {

inline bool aligned(const void *p, uintptr_t a) {
  return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}
inline moe_status_t cuda_status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }
inline bool row_type(int dt) { return dt == MOE_F32 || dt == MOE_BF16; }
inline uintptr_t elem(int dt) { return dt == MOE_F32 ? 4 : dt == MOE_BF16 ? 2 : 1; }

constexpr long long kMaxValues = 1ll << 40;
constexpr int kMaxTensors = 65536;

moe_status_t check_norm(const moe_norm_t *d) {
  if (!d || d->n < 0 || d->H < 1 || !row_type(d->dtype)) return MOE_ERR_INVALID_ARG;
  if (d->weight_dtype != MOE_F32 && d->weight_dtype != d->dtype) return MOE_ERR_INVALID_ARG;
  if (!(d->eps >= 0.f) || isinf(d->eps)) return MOE_ERR_INVALID_ARG;
  if (d->H > kNormMaxH) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// A (n, H) argument: rows of the norm's type, `stride` elements apart
bool rows_ok(const moe_norm_t *d, const void *p, int64_t stride) {
  return p && aligned(p, elem(d->dtype)) && (d->n < 2 || stride >= d->H);
}

}  // namespace

extern "C" {

moe_status_t moe_layer_norm(const moe_norm_t *desc, const void *x, int64_t x_stride,
                            const void *residual, int64_t residual_stride, const void *weight,
                            const void *bias, void *s, void *y, float *stats,
                            moe_stream_t stream) {
  moe_status_t st = check_norm(desc);
  if (st != MOE_OK) return st;
  if (desc->n == 0) return MOE_OK;
  const uintptr_t we = elem(desc->weight_dtype);
  if (!rows_ok(desc, x, x_stride) || !rows_ok(desc, y, desc->H)) return MOE_ERR_INVALID_ARG;
  if ((residual != nullptr) != (s != nullptr)) return MOE_ERR_INVALID_ARG;
  if (residual && (!rows_ok(desc, residual, residual_stride) || !rows_ok(desc, s, desc->H)))
    return MOE_ERR_INVALID_ARG;
  if (!weight || !aligned(weight, we) || !aligned(bias, we) || !aligned(stats, 4))
    return MOE_ERR_INVALID_ARG;
  return cuda_status(launch_norm(*desc, x, desc->n < 2 ? desc->H : x_stride, residual,
                                 desc->n < 2 ? desc->H : residual_stride, weight, bias, s, y, stats,
                                 stream));
}

size_t moe_layer_norm_backward_workspace_size(const moe_norm_t *desc) {
  if (check_norm(desc) != MOE_OK) return 0;
  return norm_backward_ws_bytes(*desc);
}

moe_status_t moe_layer_norm_backward(const moe_norm_t *desc, const void *dy, int64_t dy_stride,
                                     const void *s, int64_t s_stride, const float *stats,
                                     const void *weight, const void *ds, int64_t ds_stride,
                                     void *dx, float *dweight, float *dbias, void *ws,
                                     size_t ws_bytes, moe_stream_t stream) {
  moe_status_t st = check_norm(desc);
  if (st != MOE_OK) return st;
  if (!dweight || !aligned(dweight, 4) || !aligned(dbias, 4)) return MOE_ERR_INVALID_ARG;
  if (desc->n == 0)
    return cuda_status(launch_norm_backward(*desc, nullptr, 0, nullptr, 0, nullptr, nullptr,
                                            nullptr, 0, nullptr, dweight, dbias, nullptr, stream));
  if (!rows_ok(desc, dy, dy_stride) || !rows_ok(desc, s, s_stride) || !rows_ok(desc, dx, desc->H) ||
      (ds && !rows_ok(desc, ds, ds_stride)))
    return MOE_ERR_INVALID_ARG;
  if (!stats || !aligned(stats, 4) || !weight || !aligned(weight, elem(desc->weight_dtype)))
    return MOE_ERR_INVALID_ARG;
  if (!ws || !aligned(ws, 16)) return MOE_ERR_INVALID_ARG;
  if (ws_bytes < norm_backward_ws_bytes(*desc)) return MOE_ERR_WORKSPACE;
  const bool one = desc->n < 2;
  return cuda_status(launch_norm_backward(*desc, dy, one ? desc->H : dy_stride, s,
                                          one ? desc->H : s_stride, stats, weight, ds,
                                          one ? desc->H : ds_stride, dx, dweight, dbias, ws,
                                          stream));
}

size_t moe_grad_norm_workspace_size(int32_t count) {
  return count < 0 || count > kMaxTensors ? 0 : grad_norm_ws_bytes(count);
}

moe_status_t moe_grad_norm(const moe_tensor_t *tensors, int32_t count, float max_norm,
                           float *norm, float *factor, void *ws, size_t ws_bytes,
                           moe_stream_t stream) {
  if (count < 0 || (count && !tensors) || !(max_norm > 0.f)) return MOE_ERR_INVALID_ARG;
  if (count > kMaxTensors) return MOE_ERR_UNSUPPORTED;
  long long values = 0;
  for (int i = 0; i < count; ++i) {
    const moe_tensor_t &t = tensors[i];
    if (t.numel < 0 || !row_type(t.dtype)) return MOE_ERR_INVALID_ARG;
    if (t.numel && (!t.data || !aligned(t.data, elem(t.dtype)))) return MOE_ERR_INVALID_ARG;
    if (t.numel > kMaxValues || (values += t.numel) > kMaxValues) return MOE_ERR_UNSUPPORTED;
  }
  if (!norm || !factor || !aligned(norm, 4) || !aligned(factor, 4) || !ws || !aligned(ws, 256))
    return MOE_ERR_INVALID_ARG;
  if (ws_bytes < grad_norm_ws_bytes(count)) return MOE_ERR_WORKSPACE;
  return cuda_status(launch_grad_norm(tensors, count, max_norm, norm, factor, ws, stream));
}

static bool betas_ok(double b1, double b2) { return b1 >= 0 && b1 < 1 && b2 >= 0 && b2 < 1; }

moe_status_t moe_adamw_set_steps(double beta1, double beta2, int64_t steps, void *step_state,
                                 moe_stream_t stream) {
  if (!betas_ok(beta1, beta2) || steps < 0 || !step_state || !aligned(step_state, 16))
    return MOE_ERR_INVALID_ARG;
  return cuda_status(launch_adamw_set_steps(pow(beta1, (double)steps + 1),
                                            pow(beta2, (double)steps + 1), steps, step_state,
                                            stream));
}

moe_status_t moe_adamw_step(const moe_adamw_t *opt, const moe_adamw_tensor_t *tensors,
                            int32_t count, void *step_state, moe_stream_t stream) {
  if (!opt || count < 0 || (count && !tensors)) return MOE_ERR_INVALID_ARG;
  if (opt->state_dtype != MOE_F32 && opt->state_dtype != MOE_E4M3) return MOE_ERR_INVALID_ARG;
  if (opt->rounding < MOE_ROUND_BY_BETA2 || opt->rounding > MOE_ROUND_RANDOM)
    return MOE_ERR_INVALID_ARG;
  if (!betas_ok(opt->beta1, opt->beta2) || !(opt->eps >= 0x1p-126f) || isinf(opt->eps))
    return MOE_ERR_INVALID_ARG;
  if (!(opt->lr >= 0.f) || isinf(opt->lr)) return MOE_ERR_INVALID_ARG;
  if (!aligned(opt->lr_device, 4) || !aligned(opt->grad_scale, 4)) return MOE_ERR_INVALID_ARG;
  if (!step_state || !aligned(step_state, 16)) return MOE_ERR_INVALID_ARG;
  if (count > kMaxTensors) return MOE_ERR_UNSUPPORTED;
  const bool e4m3 = opt->state_dtype == MOE_E4M3;
  const uintptr_t se = e4m3 ? 1 : 4;
  long long values = 0;
  for (int i = 0; i < count; ++i) {
    const moe_adamw_tensor_t &t = tensors[i];
    if (t.numel < 0 || !row_type(t.dtype) || !row_type(t.grad_dtype)) return MOE_ERR_INVALID_ARG;
    if (!(t.weight_decay >= 0.f) || isinf(t.weight_decay)) return MOE_ERR_INVALID_ARG;
    if (!e4m3 && (t.m_scale || t.v_scale)) return MOE_ERR_INVALID_ARG;
    if (t.numel > kMaxValues || (values += t.numel) > kMaxValues) return MOE_ERR_UNSUPPORTED;
    if (t.numel == 0) continue;
    if (!t.param || !t.grad || !t.m || !t.v || (e4m3 && (!t.m_scale || !t.v_scale)))
      return MOE_ERR_INVALID_ARG;
    if (!aligned(t.param, elem(t.dtype)) || !aligned(t.master, 4) ||
        !aligned(t.grad, elem(t.grad_dtype)) || !aligned(t.m, se) || !aligned(t.v, se) ||
        !aligned(t.m_scale, 4) || !aligned(t.v_scale, 4))
      return MOE_ERR_INVALID_ARG;
  }
  return cuda_status(launch_adamw(*opt, tensors, count, step_state, stream));
}

}  // extern "C"
