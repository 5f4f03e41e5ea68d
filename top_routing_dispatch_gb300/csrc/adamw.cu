// The gradients' global norm, and one AdamW step, over many tensors in one
// launch each.
//
//   g = grad f;  m = b1 m + (1 - b1) g;  v = b2 v + ((1 - b2) g) g
//   p = p (1 - lr wd) - lr / (1 - b1^t) m / (sqrt(v) / sqrt(1 - b2^t) + eps)
//
// Every product and sum of m and v is rounded by itself (no contraction), so
// that a state's 8-bit code does not depend on how the compiler fuses them.
//
// 8-bit states: 256 values of a tensor share a float32 scale; m = code scale,
// sqrt(v) = code scale with e4m3 codes, scale = largest / 448.  The root is
// held, not v itself: e4m3 spans 2^-9 .. 448, which as a root covers 2^36 of
// v.  A positive root never becomes zero (its code is at least the smallest),
// because the step divides by it.  Infinities and NaN become NaN codes and do
// not enter the scale, so they stay where they are.
//
// A warp takes 256 values: lane l those at 4 l .. 4 l + 3 and 128 further on.
#include <cuda_fp8.h>

#include "df.cuh"
#include "train.cuh"

namespace moe {
namespace {

constexpr int kUnit = 2048;  // values of a CTA's turn
constexpr int kThreads = kUnit / 8;
constexpr float kInvMax = (float)(1.0 / 448.0);
constexpr float kTiny = 0x1p-100f;  // the least largest value that a scale is made for

// What a step needs of its number; kept on the device, advanced by the step
// itself, so that a captured step counts on when it is replayed.
struct StepState {
  long long steps;  // taken
  double p1, p2;    // beta^(steps + 1)
  float inv1, inv2; // 1 / (1 - beta1^(steps + 1)), 1 / sqrt(1 - beta2^(steps + 1))
  unsigned done;    // CTAs of the running step that have finished
};
static_assert(sizeof(StepState) <= MOE_ADAMW_STATE_BYTES, "state");

__device__ __forceinline__ void derive(StepState *s) {
  s->inv1 = (float)(1.0 / (1.0 - s->p1));
  s->inv2 = (float)(1.0 / sqrt(1.0 - s->p2));
}

__global__ void adamw_set_steps_kernel(double p1, double p2, long long steps, StepState *s) {
  pdl_enter();
  s->steps = steps, s->p1 = p1, s->p2 = p2, s->done = 0;
  derive(s);
}

struct Tensor {
  void *param;
  float *master;
  const void *grad;
  void *m, *v;
  float *ms, *vs;
  long long numel;
  int first;    // turn at which it begins
  int flags;
  float keep;   // weight decay; the kernel multiplies by the learning rate
};
enum { kParamBf16 = 1, kGradBf16 = 2, kVector = 4 };

template <int CAP>
struct StepArgs {
  Tensor t[CAP];
  StepState *state;
  const float *lr_dev, *scale;
  float lr, b1, a1, b2, a2, eps;  // a = 1 - b
  double beta1, beta2;
  int count, turns;
  bool last;  // launch of the step
};

// 4 neighbouring values from `at`, of which `left` exist (the rest are 0)
__device__ __forceinline__ float4 load4(const void *p, bool bf16, bool vec, long long at,
                                        long long left) {
  float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
  float *e = &f.x;
  if (bf16) {
    const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(p) + at;
    if (vec && left >= 4) {
      const uint2 u = *reinterpret_cast<const uint2 *>(q);
      const float2 a = __bfloat1622float2(reinterpret_cast<const __nv_bfloat162 *>(&u)[0]);
      const float2 b = __bfloat1622float2(reinterpret_cast<const __nv_bfloat162 *>(&u)[1]);
      return make_float4(a.x, a.y, b.x, b.y);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < left) e[i] = __bfloat162float(q[i]);
  } else {
    const float *q = static_cast<const float *>(p) + at;
    if (vec && left >= 4) return *reinterpret_cast<const float4 *>(q);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < left) e[i] = q[i];
  }
  return f;
}

__device__ __forceinline__ void store4(void *p, bool bf16, bool vec, long long at, long long left,
                                       float4 f) {
  const float *e = &f.x;
  if (bf16) {
    __nv_bfloat16 *q = static_cast<__nv_bfloat16 *>(p) + at;
    if (vec && left >= 4) {
      uint2 u;
      reinterpret_cast<__nv_bfloat162 *>(&u)[0] = __floats2bfloat162_rn(f.x, f.y);
      reinterpret_cast<__nv_bfloat162 *>(&u)[1] = __floats2bfloat162_rn(f.z, f.w);
      *reinterpret_cast<uint2 *>(q) = u;
      return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < left) q[i] = __float2bfloat16_rn(e[i]);
  } else {
    float *q = static_cast<float *>(p) + at;
    if (vec && left >= 4) {
      *reinterpret_cast<float4 *>(q) = f;
      return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < left) q[i] = e[i];
  }
}

// 4 codes
__device__ __forceinline__ float4 decode4(uint32_t u) {
  const __half2_raw a = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(u & 0xffff), __NV_E4M3);
  const __half2_raw b = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(u >> 16), __NV_E4M3);
  const float2 x = __half22float2(__half2(a)), y = __half22float2(__half2(b));
  return make_float4(x.x, x.y, y.x, y.y);
}
__device__ __forceinline__ uint32_t encode4(float4 f) {
  const uint32_t a = __nv_cvt_float2_to_fp8x2(make_float2(f.x, f.y), __NV_SATFINITE, __NV_E4M3);
  const uint32_t b = __nv_cvt_float2_to_fp8x2(make_float2(f.z, f.w), __NV_SATFINITE, __NV_E4M3);
  return a | b << 16;
}
__device__ __forceinline__ uint32_t load_codes(const void *p, bool vec, long long at,
                                               long long left) {
  const uint8_t *q = static_cast<const uint8_t *>(p) + at;
  if (vec && left >= 4) return *reinterpret_cast<const uint32_t *>(q);
  uint32_t u = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i < left) u |= (uint32_t)q[i] << (8 * i);
  return u;
}
__device__ __forceinline__ void store_codes(void *p, bool vec, long long at, long long left,
                                            uint32_t u) {
  uint8_t *q = static_cast<uint8_t *>(p) + at;
  if (vec && left >= 4) {
    *reinterpret_cast<uint32_t *>(q) = u;
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i < left) q[i] = (uint8_t)(u >> (8 * i));
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o /= 2) v = fmaxf(v, __shfl_xor_sync(~0u, v, o));
  return v;
}

// Magnitude that counts for a scale: that of a finite value
__device__ __forceinline__ float finite_abs(float v) {
  v = fabsf(v);
  return v < INFINITY ? v : 0.f;
}

template <bool E4M3, int CAP>
__global__ void __launch_bounds__(kThreads)
    adamw_kernel(const __grid_constant__ StepArgs<CAP> a) {
  pdl_enter();
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const float lr = a.lr_dev ? __ldg(a.lr_dev) : a.lr;
  const float fac = a.scale ? __ldg(a.scale) : 1.f;
  const float c1 = lr * a.state->inv1, c2 = a.state->inv2;
  int k = 0;
  for (int turn = blockIdx.x; turn < a.turns; turn += gridDim.x) {
    while (k + 1 < a.count && turn >= a.t[k + 1].first) ++k;
    const Tensor &t = a.t[k];
    const long long block = (long long)(turn - t.first) * (kUnit / kAdamBlock) + warp;
    const long long base = block * kAdamBlock;
    if (base >= t.numel) continue;  // whole warps
    const bool pb = t.flags & kParamBf16, gb = t.flags & kGradBf16, vec = t.flags & kVector;
    const float keep = 1.f - lr * t.keep;
    float4 g[2], p[2], m[2], v[2], root[2];
    float ms = 0.f, vs = 0.f;
    if (E4M3) ms = t.ms[block], vs = t.vs[block];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const long long at = base + 128 * h + 4 * lane, left = t.numel - at;
      g[h] = load4(t.grad, gb, vec, at, left);
      p[h] = t.master ? load4(t.master, false, vec, at, left) : load4(t.param, pb, vec, at, left);
      if (E4M3) {
        m[h] = decode4(load_codes(t.m, vec, at, left));
        v[h] = decode4(load_codes(t.v, vec, at, left));
      } else {
        m[h] = load4(t.m, false, vec, at, left);
        v[h] = load4(t.v, false, vec, at, left);
      }
    }
    float top_m = 0.f, top_r = 0.f;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float *ge = &g[h].x, *pe = &p[h].x, *me = &m[h].x, *ve = &v[h].x, *re = &root[h].x;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float gr = a.scale ? __fmul_rn(ge[i], fac) : ge[i];
        float mo = me[i], vo = ve[i];
        if (E4M3) {
          mo = __fmul_rn(mo, ms);
          vo = __fmul_rn(vo, vs);
          vo = __fmul_rn(vo, vo);
        }
        me[i] = __fadd_rn(__fmul_rn(mo, a.b1), __fmul_rn(gr, a.a1));
        ve[i] = __fadd_rn(__fmul_rn(vo, a.b2), __fmul_rn(__fmul_rn(gr, a.a2), gr));
        re[i] = __fsqrt_rn(ve[i]);
        pe[i] = pe[i] * keep - c1 * __fdiv_rn(me[i], fmaf(re[i], c2, a.eps));
        if (E4M3) {
          top_m = fmaxf(top_m, finite_abs(me[i]));
          top_r = fmaxf(top_r, finite_abs(re[i]));
        }
      }
    }
    float im = 0.f, ir = 0.f;
    if (E4M3) {
      ms = __fmul_rn(fmaxf(warp_max(top_m), kTiny), kInvMax);
      vs = __fmul_rn(fmaxf(warp_max(top_r), kTiny), kInvMax);
      im = __frcp_rn(ms), ir = __frcp_rn(vs);
      if (lane == 0) t.ms[block] = ms, t.vs[block] = vs;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const long long at = base + 128 * h + 4 * lane, left = t.numel - at;
      if (t.master) store4(t.master, false, vec, at, left, p[h]);
      store4(t.param, pb, vec, at, left, p[h]);
      if (E4M3) {
        float4 cm, cr;
        float *me = &m[h].x, *re = &root[h].x, *ce = &cm.x, *de = &cr.x;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          // 0 x is 0, and NaN for an infinity
          ce[i] = fmaf(0.f, me[i], __fmul_rn(me[i], im));
          de[i] = fmaxf(__fmul_rn(re[i], ir), re[i] > 0.f ? 0x1p-9f : 0.f);
          de[i] = fmaf(0.f, re[i], de[i]);
        }
        store_codes(t.m, vec, at, left, encode4(cm));
        store_codes(t.v, vec, at, left, encode4(cr));
      } else {
        store4(t.m, false, vec, at, left, m[h]);
        store4(t.v, false, vec, at, left, v[h]);
      }
    }
  }
  if (!a.last) return;
  // the last CTA to finish advances the step: by then every CTA has read it
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    if (atomicAdd(&a.state->done, 1u) == gridDim.x - 1) {
      StepState *s = a.state;
      s->steps += 1;
      s->p1 *= a.beta1;
      s->p2 *= a.beta2;
      derive(s);
      s->done = 0;
    }
  }
}

// ------------------------------------------------------------ global norm
struct Part {
  const void *data;
  long long numel;
  int first, flags;
};
template <int CAP>
struct NormArgs {
  Part t[CAP];
  double *part;  // a sum of squares per CTA
  int count, turns;
};

template <int CAP>
__global__ void __launch_bounds__(kThreads)
    grad_norm_kernel(const __grid_constant__ NormArgs<CAP> a) {
  pdl_enter();
  __shared__ double warps[kThreads / 32];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  double sum = 0.0;
  int k = 0;
  for (int turn = blockIdx.x; turn < a.turns; turn += gridDim.x) {
    while (k + 1 < a.count && turn >= a.t[k + 1].first) ++k;
    const Part &t = a.t[k];
    const bool bf16 = t.flags & kGradBf16, vec = t.flags & kVector;
    float s = 0.f;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const long long at = (long long)(turn - t.first) * kUnit + 4 * (threadIdx.x + kThreads * h);
      const float4 f = load4(t.data, bf16, vec, at, t.numel - at);
      s = fmaf(f.x, f.x, s), s = fmaf(f.y, f.y, s), s = fmaf(f.z, f.z, s), s = fmaf(f.w, f.w, s);
    }
    sum += (double)s;
  }
#pragma unroll
  for (int o = 16; o > 0; o /= 2) sum += __shfl_xor_sync(~0u, sum, o);
  if (lane == 0) warps[warp] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 1; i < kThreads / 32; ++i) sum += warps[i];
    a.part[blockIdx.x] = sum;
  }
}

__global__ void __launch_bounds__(256)
    grad_norm_join_kernel(const double *part, int parts, float max_norm, float *norm,
                          float *factor) {
  pdl_enter();
  __shared__ double warps[8];
  double sum = 0.0;
  for (int i = threadIdx.x; i < parts; i += 256) sum += part[i];
#pragma unroll
  for (int o = 16; o > 0; o /= 2) sum += __shfl_xor_sync(~0u, sum, o);
  if (threadIdx.x % 32 == 0) warps[threadIdx.x / 32] = sum;
  __syncthreads();
  if (threadIdx.x) return;
  for (int i = 1; i < 8; ++i) sum += warps[i];
  const float n = (float)sqrt(sum);
  const float f = max_norm / (n + 1e-6f);
  *norm = n;
  *factor = f < 1.f ? f : f >= 1.f ? 1.f : f;  // NaN stays
}

constexpr int kSmallCap = 48, kLargeCap = 384;  // tensors of a launch
constexpr int kMaxCtas = 608;                   // of a launch of the norm

inline bool on16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
inline long long turns_of(long long numel) { return (numel + kUnit - 1) / kUnit; }

template <bool E4M3, int CAP>
cudaError_t step_launch(const moe_adamw_t &o, const moe_adamw_tensor_t *t, int count, bool last,
                        StepState *state, cudaStream_t s) {
  StepArgs<CAP> a;
  long long turns = 0;
  a.count = 0;
  for (int i = 0; i < count; ++i) {
    const moe_adamw_tensor_t &x = t[i];
    if (x.numel == 0) continue;
    const bool vec = on16(x.param) && on16(x.master) && on16(x.grad) && on16(x.m) && on16(x.v);
    a.t[a.count++] = Tensor{x.param, x.master, x.grad, x.m, x.v, x.m_scale, x.v_scale, x.numel,
                            (int)turns,
                            (x.dtype == MOE_BF16 ? kParamBf16 : 0) |
                                (x.grad_dtype == MOE_BF16 ? kGradBf16 : 0) | (vec ? kVector : 0),
                            x.weight_decay};
    turns += turns_of(x.numel);
  }
  a.state = state;
  a.lr_dev = o.lr_device, a.scale = o.grad_scale;
  a.lr = o.lr, a.eps = o.eps;
  a.b1 = (float)o.beta1, a.a1 = (float)(1.0 - o.beta1);
  a.b2 = (float)o.beta2, a.a2 = (float)(1.0 - o.beta2);
  a.beta1 = o.beta1, a.beta2 = o.beta2;
  a.turns = (int)turns, a.last = last;
  const long long most = 4ll * device_sm_count();
  const unsigned grid = (unsigned)(turns < 1 ? 1 : turns < most ? turns : most);
  return launch_pdl(adamw_kernel<E4M3, CAP>, dim3(grid), dim3(kThreads), 0, s, a);
}

}  // namespace

size_t grad_norm_ws_bytes(int count) {
  const size_t launches = count < 1 ? 1 : (size_t)(count + kLargeCap - 1) / kLargeCap;
  return (launches * kMaxCtas * sizeof(double) + 255) / 256 * 256;
}

template <int CAP>
static cudaError_t norm_launch(const moe_tensor_t *t, int count, double *part, int *parts,
                               cudaStream_t s) {
  NormArgs<CAP> a;
  long long turns = 0;
  a.count = 0;
  for (int i = 0; i < count; ++i) {
    if (t[i].numel == 0) continue;
    a.t[a.count++] = Part{t[i].data, t[i].numel, (int)turns,
                          (t[i].dtype == MOE_BF16 ? kGradBf16 : 0) | (on16(t[i].data) ? kVector : 0)};
    turns += turns_of(t[i].numel);
  }
  if (turns == 0) return cudaSuccess;
  a.part = part + *parts, a.turns = (int)turns;
  const int most = 4 * device_sm_count() < kMaxCtas ? 4 * device_sm_count() : kMaxCtas;
  const int grid = turns < most ? (int)turns : most;
  *parts += grid;
  return launch_pdl(grad_norm_kernel<CAP>, dim3(grid), dim3(kThreads), 0, s, a);
}

cudaError_t launch_grad_norm(const moe_tensor_t *t, int count, float max_norm, float *norm,
                             float *factor, void *ws, cudaStream_t s) {
  double *part = static_cast<double *>(ws);
  int parts = 0;
  cudaError_t e = cudaSuccess;
  if (count <= kSmallCap) {
    e = norm_launch<kSmallCap>(t, count, part, &parts, s);
  } else {
    for (int i = 0; i < count && e == cudaSuccess; i += kLargeCap)
      e = norm_launch<kLargeCap>(t + i, count - i < kLargeCap ? count - i : kLargeCap, part, &parts, s);
  }
  if (e != cudaSuccess) return e;
  return launch_pdl(grad_norm_join_kernel, dim3(1), dim3(256), 0, s, (const double *)part, parts,
                    max_norm, norm, factor);
}

cudaError_t launch_adamw_set_steps(double p1, double p2, long long steps, void *state,
                                   cudaStream_t s) {
  return launch_pdl(adamw_set_steps_kernel, dim3(1), dim3(1), 0, s, p1, p2, steps,
                    static_cast<StepState *>(state));
}

template <bool E4M3>
static cudaError_t step_all(const moe_adamw_t &o, const moe_adamw_tensor_t *t, int count,
                            StepState *state, cudaStream_t s) {
  if (count <= kSmallCap) return step_launch<E4M3, kSmallCap>(o, t, count, true, state, s);
  cudaError_t e = cudaSuccess;
  for (int i = 0; i < count && e == cudaSuccess; i += kLargeCap) {
    const int k = count - i < kLargeCap ? count - i : kLargeCap;
    e = step_launch<E4M3, kLargeCap>(o, t + i, k, i + k == count, state, s);
  }
  return e;
}

cudaError_t launch_adamw(const moe_adamw_t &o, const moe_adamw_tensor_t *t, int count, void *state,
                         cudaStream_t s) {
  StepState *st = static_cast<StepState *>(state);
  return o.state_dtype == MOE_E4M3 ? step_all<true>(o, t, count, st, s)
                                   : step_all<false>(o, t, count, st, s);
}

}  // namespace moe
