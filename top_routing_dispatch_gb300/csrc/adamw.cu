// The gradients' global norm, and one AdamW step, over many tensors in one
// launch each.
//
//   g = grad f;  m = b1 m + (1 - b1) g;  v = b2 v + ((1 - b2) g) g
//   p = p (1 - lr wd) - lr / (1 - b1^t) m / (sqrt(v) / sqrt(1 - b2^t) + eps)
//
// In m and v the gradient's term is rounded, and the rest is one fused multiply-
// add, spelled out so that a state's 8-bit code does not depend on what the
// compiler contracts.
//
// 8-bit states: 256 values of a tensor share a float32 scale; m = code scale,
// sqrt(v) = code scale with e4m3 codes, scale = largest / 448.  The root is
// held, not v itself: e4m3 spans 2^-9 .. 448, which as a root covers 2^36 of
// v.  A positive root never becomes zero (its code is at least the smallest),
// because the step divides by it.  Infinities and NaN become NaN codes and do
// not enter the scale, so they stay where they are.
//
// A warp takes 256 values at a time: lane l those at 4 l .. 4 l + 3 and 128
// further on, in pairs for the two-operation instructions.
//
// Bound: HBM with float32 states (28 bytes a value in float32 throughout);
// instructions come next, which is why the 8-bit form counts them: the largest
// root is the root of the largest v, one warp-wide maximum of integers does for
// a block (positive floats order as their bits), and what only an infinity, a
// NaN, a tiny v or a zero code needs stands apart behind one test.
#include <cuda_fp8.h>

#include "pairs.cuh"
#include "train.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMostBlocks = 8;  // of a warp's turn
constexpr float kInvMax = (float)(1.0 / 448.0);
constexpr float kTiny = 0x1p-100f;  // the least largest value that a scale is made for
constexpr uint32_t kInfBits = 0x7f800000u;

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
  float decay;  // weight decay; the kernel multiplies by the learning rate
  bool vec;     // all on 16 bytes
};

template <int CAP>
struct StepArgs {
  Tensor t[CAP];
  StepState *state;
  const float *lr_dev, *scale;
  float lr, b1, a1, b2, a2, eps;  // a = 1 - b
  double beta1, beta2;
  int count, turns, blocks;  // blocks of a turn
  bool last;                 // launch of the step
};

// sqrt(v), rounded to nearest: one Newton step with a fused residual (Markstein)
// from the approximate reciprocal root; below 2^-96 the residual would
// underflow.  Equal to __fsqrt_rn for every float32 from 2^-102 up (tried).
__device__ __forceinline__ float2 root2(float2 v) {
  const float2 y = make_float2(rsqrtf(v.x), rsqrtf(v.y));
  const float2 s = mul2(v, y);
  return fma2(fma2(mul2(s, both(-1.f)), s, v), mul2(y, both(0.5f)), s);
}
__device__ __forceinline__ bool plain_root(uint32_t bits) {
  return bits >= 0x0f800000u && bits < kInfBits;  // 2^-96 to the largest finite
}

__device__ __forceinline__ float reciprocal(float x) {  // within 2 u
  float y;
  asm("rcp.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 4 neighbouring values from `at` as two pairs; those past `left` are 0
template <typename T, bool FULL>
__device__ __forceinline__ void load4(const void *p, long long at, int left, float2 *f) {
  const T *q = static_cast<const T *>(p) + at;
  if constexpr (FULL && sizeof(T) == 2) {
    const uint2 u = *reinterpret_cast<const uint2 *>(q);
    f[0] = make_float2(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u));
    f[1] = make_float2(__uint_as_float(u.y << 16), __uint_as_float(u.y & 0xffff0000u));
  } else if constexpr (FULL) {
    const float4 u = *reinterpret_cast<const float4 *>(q);
    f[0] = make_float2(u.x, u.y), f[1] = make_float2(u.z, u.w);
  } else {
    float e[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) e[i] = i < left ? (float)q[i] : 0.f;
    f[0] = make_float2(e[0], e[1]), f[1] = make_float2(e[2], e[3]);
  }
}

template <typename T, bool FULL>
__device__ __forceinline__ void store4(void *p, long long at, int left, const float2 *f) {
  T *q = static_cast<T *>(p) + at;
  if constexpr (FULL && sizeof(T) == 2) {
    uint2 u;
    reinterpret_cast<__nv_bfloat162 *>(&u)[0] = __float22bfloat162_rn(f[0]);
    reinterpret_cast<__nv_bfloat162 *>(&u)[1] = __float22bfloat162_rn(f[1]);
    *reinterpret_cast<uint2 *>(q) = u;
  } else if constexpr (FULL) {
    *reinterpret_cast<float4 *>(q) = make_float4(f[0].x, f[0].y, f[1].x, f[1].y);
  } else {
    const float e[4] = {f[0].x, f[0].y, f[1].x, f[1].y};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < left) q[i] = (T)e[i];
  }
}

template <bool FULL>
__device__ __forceinline__ uint32_t load_codes(const void *p, long long at, int left) {
  const uint8_t *q = static_cast<const uint8_t *>(p) + at;
  uint32_t u = 0;
  if constexpr (FULL) {
    u = *reinterpret_cast<const uint32_t *>(q);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < left) u |= (uint32_t)q[i] << (8 * i);
  }
  return u;
}
template <bool FULL>
__device__ __forceinline__ void store_codes(void *p, long long at, int left, uint32_t u) {
  uint8_t *q = static_cast<uint8_t *>(p) + at;
  if constexpr (FULL) {
    *reinterpret_cast<uint32_t *>(q) = u;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < left) q[i] = (uint8_t)(u >> (8 * i));
  }
}

__device__ __forceinline__ void decode4(uint32_t u, float2 *f) {
  const __half2_raw a = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(u & 0xffff), __NV_E4M3);
  const __half2_raw b = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(u >> 16), __NV_E4M3);
  f[0] = __half22float2(__half2(a)), f[1] = __half22float2(__half2(b));
}
__device__ __forceinline__ uint32_t encode4(const float2 *f) {
  const uint32_t a = __nv_cvt_float2_to_fp8x2(f[0], __NV_SATFINITE, __NV_E4M3);
  const uint32_t b = __nv_cvt_float2_to_fp8x2(f[1], __NV_SATFINITE, __NV_E4M3);
  return a | b << 16;
}

// Magnitude that counts for a scale: that of a finite value
__device__ __forceinline__ uint32_t finite_bits(float v) {
  const uint32_t b = __float_as_uint(v) & 0x7fffffffu;
  return b < kInfBits ? b : 0u;
}
__device__ __forceinline__ float nan_if_not_finite(float v, float code) {
  return finite_bits(v) == (__float_as_uint(v) & 0x7fffffffu) ? code : NAN;
}

struct Step {
  float keep, fac, c1, c2, b1, a1, b2, a2, eps;
  bool scaled;
};

// One block of 256 values.  PT, GT: types of parameter and gradient; MASTER:
// a float32 master of a bf16 parameter (a float32 parameter's is a copy).
template <bool E4M3, typename PT, typename GT, bool MASTER, bool FULL>
__device__ __forceinline__ void step_block(const Tensor &t, const Step &c, long long block,
                                           int lane) {
  const long long base = block * kAdamBlock;
  float2 g[4], p[4], m[4], v[4], root[4];
  float ms = 0.f, vs = 0.f;
  int left[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const long long at = base + 128 * h + 4 * lane;
    left[h] = FULL ? 4 : (int)(t.numel - at < 4 ? t.numel - at : 4);
    load4<GT, FULL>(t.grad, at, left[h], g + 2 * h);
    if (MASTER || t.master)
      load4<float, FULL>(t.master, at, left[h], p + 2 * h);
    else
      load4<PT, FULL>(t.param, at, left[h], p + 2 * h);
    if (E4M3) {
      decode4(load_codes<FULL>(t.m, at, left[h]), m + 2 * h);
      decode4(load_codes<FULL>(t.v, at, left[h]), v + 2 * h);
    } else {
      load4<float, FULL>(t.m, at, left[h], m + 2 * h);
      load4<float, FULL>(t.v, at, left[h], v + 2 * h);
    }
  }
  if (E4M3) ms = t.ms[block], vs = t.vs[block];
  uint32_t top_v = 0, low_v = ~0u;
  float top_m = 0.f;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (c.scaled) g[k] = mul2(g[k], both(c.fac));
    if (E4M3) {
      m[k] = mul2(m[k], both(ms));
      v[k] = mul2(v[k], both(vs));
      v[k] = mul2(v[k], v[k]);
    }
    m[k] = fma2(m[k], both(c.b1), mul2(g[k], both(c.a1)));
    v[k] = fma2(v[k], both(c.b2), mul2(mul2(g[k], both(c.a2)), g[k]));
    const uint32_t x = __float_as_uint(v[k].x), y = __float_as_uint(v[k].y);
    low_v = min(low_v, min(x, y));
    top_v = max(top_v, max(x, y));
    if (E4M3) top_m = fmaxf(top_m, fmaxf(fabsf(m[k].x), fabsf(m[k].y)));
    root[k] = root2(v[k]);
  }
  if (!plain_root(low_v) || !plain_root(top_v)) {  // also a NaN, whose bits are larger
#pragma unroll
    for (int k = 0; k < 4; ++k)
      root[k] = make_float2(__fsqrt_rn(v[k].x), __fsqrt_rn(v[k].y));
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    float2 d = fma2(root[k], both(c.c2), both(c.eps));
    d = mul2(m[k], make_float2(reciprocal(d.x), reciprocal(d.y)));
    p[k] = fma2(d, both(-c.c1), mul2(p[k], both(c.keep)));
  }
  if (E4M3) {
    uint32_t bm = __reduce_max_sync(~0u, __float_as_uint(top_m));
    uint32_t bv = __reduce_max_sync(~0u, top_v);
    const bool bad = bm >= kInfBits || bv >= kInfBits;
    if (bad) {
      bm = bv = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        bm = max(bm, max(finite_bits(m[k].x), finite_bits(m[k].y)));
        bv = max(bv, max(finite_bits(v[k].x), finite_bits(v[k].y)));
      }
      bm = __reduce_max_sync(~0u, bm);
      bv = __reduce_max_sync(~0u, bv);
    }
    ms = __fmul_rn(fmaxf(__uint_as_float(bm), kTiny), kInvMax);
    vs = __fmul_rn(fmaxf(__fsqrt_rn(__uint_as_float(bv)), kTiny), kInvMax);
    const float2 im = both(__frcp_rn(ms)), iv = both(__frcp_rn(vs));
    if (lane == 0) t.ms[block] = ms, t.vs[block] = vs;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 x = mul2(m[k], im), y = mul2(root[k], iv);
      if (bad) {
        v[k] = make_float2(nan_if_not_finite(root[k].x, y.x), nan_if_not_finite(root[k].y, y.y));
        m[k] = make_float2(nan_if_not_finite(m[k].x, x.x), nan_if_not_finite(m[k].y, x.y));
      } else {
        v[k] = y, m[k] = x;
      }
    }
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const long long at = base + 128 * h + 4 * lane;
    if (MASTER || t.master) store4<float, FULL>(t.master, at, left[h], p + 2 * h);
    store4<PT, FULL>(t.param, at, left[h], p + 2 * h);
    if (E4M3) {
      uint32_t r = encode4(v + 2 * h);
      // a positive root keeps at least the smallest code
      if ((r - 0x01010101u) & ~r & 0x80808080u) {
        const float2 *q = root + 2 * h;
        const float e[4] = {q[0].x, q[0].y, q[1].x, q[1].y};
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (!(r >> (8 * i) & 0xff) && e[i] > 0.f) r |= 1u << (8 * i);
      }
      store_codes<FULL>(t.m, at, left[h], encode4(m + 2 * h));
      store_codes<FULL>(t.v, at, left[h], r);
    } else {
      store4<float, FULL>(t.m, at, left[h], m + 2 * h);
      store4<float, FULL>(t.v, at, left[h], v + 2 * h);
    }
  }
}

template <bool E4M3, typename PT, typename GT, bool MASTER, int CAP>
__global__ void __launch_bounds__(kThreads, 4)
    adamw_kernel(const __grid_constant__ StepArgs<CAP> a) {
  pdl_enter();
  const int lane = threadIdx.x % 32;
  const float lr = a.lr_dev ? __ldg(a.lr_dev) : a.lr;
  Step c = {1.f, a.scale ? __ldg(a.scale) : 1.f, lr * a.state->inv1, a.state->inv2, a.b1, a.a1,
            a.b2, a.a2, a.eps, a.scale != nullptr};
  const int warps = gridDim.x * kWarps;
  int k = 0;
  // neighbouring turns on neighbouring CTAs' warps
  for (int turn = threadIdx.x / 32 * gridDim.x + blockIdx.x; turn < a.turns; turn += warps) {
    while (k + 1 < a.count && turn >= a.t[k + 1].first) ++k;
    const Tensor &t = a.t[k];
    c.keep = 1.f - lr * t.decay;
    long long block = (long long)(turn - t.first) * a.blocks;
    const long long whole = t.vec ? t.numel / kAdamBlock : 0;
    for (int i = 0; i < a.blocks; ++i, ++block) {
      if (block < whole)
        step_block<E4M3, PT, GT, MASTER, true>(t, c, block, lane);
      else if (block * kAdamBlock < t.numel)
        step_block<E4M3, PT, GT, MASTER, false>(t, c, block, lane);
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
constexpr int kNormUnit = 8192;  // values of a CTA's turn
constexpr int kNormCtas = 1216;  // of a launch, at most

struct Part {
  const void *data;
  long long numel;
  int first;
  bool bf16, vec;
};
template <int CAP>
struct NormArgs {
  Part t[CAP];
  double *part;  // a sum of squares per CTA
  int count, turns;
};

// Bound: HBM.  A thread asks for all 16-byte pieces of its turn (128 bytes of
// float32) before it uses one.
template <int CAP>
__global__ void __launch_bounds__(kThreads)
    grad_norm_kernel(const __grid_constant__ NormArgs<CAP> a) {
  pdl_enter();
  __shared__ double warps[kWarps];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  double sum = 0.0;
  int k = 0;
  for (int turn = blockIdx.x; turn < a.turns; turn += gridDim.x) {
    while (k + 1 < a.count && turn >= a.t[k + 1].first) ++k;
    const Part &t = a.t[k];
    const long long base = (long long)(turn - t.first) * kNormUnit;
    float2 s[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
    if (t.vec && base + kNormUnit <= t.numel) {
      uint4 u[8];
      const int pieces = t.bf16 ? 4 : 8;
      const uint4 *q = reinterpret_cast<const uint4 *>(static_cast<const char *>(t.data) +
                                                       base * (t.bf16 ? 2 : 4)) + threadIdx.x;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < pieces) u[i] = __ldg(q + i * kThreads);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (i >= pieces) break;
        const uint32_t w[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
        if (t.bf16) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 f = make_float2(__uint_as_float(w[j] << 16),
                                         __uint_as_float(w[j] & 0xffff0000u));
            s[j % 2] = fma2(f, f, s[j % 2]);
          }
        } else {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float2 f = make_float2(__uint_as_float(w[2 * j]), __uint_as_float(w[2 * j + 1]));
            s[j] = fma2(f, f, s[j]);
          }
        }
      }
    } else {
      for (int i = threadIdx.x; i < kNormUnit && base + i < t.numel; i += kThreads) {
        const float f = t.bf16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(t.data)[base + i])
                               : static_cast<const float *>(t.data)[base + i];
        s[0].x = fmaf(f, f, s[0].x);
      }
    }
    s[0] = add2(s[0], s[1]);
    sum += (double)(s[0].x + s[0].y);
  }
#pragma unroll
  for (int o = 16; o > 0; o /= 2) sum += __shfl_xor_sync(~0u, sum, o);
  if (lane == 0) warps[warp] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 1; i < kWarps; ++i) sum += warps[i];
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

// ---------------------------------------------------------------- launches
constexpr int kSmallCap = 48, kLargeCap = 384;  // tensors of a launch

inline bool on16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
inline long long ceil_of(long long a, long long b) { return (a + b - 1) / b; }

template <int CAP>
cudaError_t norm_launch(const moe_tensor_t *t, int count, double *part, int *parts,
                        cudaStream_t s) {
  NormArgs<CAP> a;
  long long turns = 0;
  a.count = 0;
  for (int i = 0; i < count; ++i) {
    if (t[i].numel == 0) continue;
    a.t[a.count++] = Part{t[i].data, t[i].numel, (int)turns, t[i].dtype == MOE_BF16,
                          on16(t[i].data)};
    turns += ceil_of(t[i].numel, kNormUnit);
  }
  if (turns == 0) return cudaSuccess;
  a.part = part + *parts, a.turns = (int)turns;
  const long long most = 8ll * device_sm_count() < kNormCtas ? 8ll * device_sm_count() : kNormCtas;
  const int grid = (int)(turns < most ? turns : most);
  *parts += grid;
  return launch_pdl(grad_norm_kernel<CAP>, dim3(grid), dim3(kThreads), 0, s, a);
}

// What a kernel is made for; the tensors of a step are launched kind by kind.
struct Kind {
  bool param_bf16, grad_bf16, master;
};
inline Kind kind_of(const moe_adamw_tensor_t &t) {
  const bool b = t.dtype == MOE_BF16;
  return Kind{b, t.grad_dtype == MOE_BF16, b && t.master};
}

struct Pending {  // tensors of one kind, by index
  int index[kLargeCap];
  int count = 0;
};

template <bool E4M3, typename PT, typename GT, bool MASTER, int CAP>
cudaError_t step_cap(const moe_adamw_t &o, const moe_adamw_tensor_t *t, const Pending &q, bool last,
                     StepState *state, cudaStream_t s) {
  StepArgs<CAP> a;
  const int sms = device_sm_count();
  long long blocks = 0;
  for (int i = 0; i < q.count; ++i) blocks += ceil_of(t[q.index[i]].numel, kAdamBlock);
  // short turns while there are few of them, so that every warp has some
  const long long share = blocks / (sms * 64ll);
  a.blocks = (int)(share < 1 ? 1 : share < kMostBlocks ? share : kMostBlocks);
  long long turns = 0;
  a.count = 0;
  for (int i = 0; i < q.count; ++i) {
    const moe_adamw_tensor_t &x = t[q.index[i]];
    const bool vec = on16(x.param) && on16(x.master) && on16(x.grad) && on16(x.m) && on16(x.v);
    a.t[a.count++] = Tensor{x.param, x.master, x.grad, x.m, x.v, x.m_scale, x.v_scale, x.numel,
                            (int)turns, x.weight_decay, vec};
    turns += ceil_of(ceil_of(x.numel, kAdamBlock), a.blocks);
  }
  a.state = state;
  a.lr_dev = o.lr_device, a.scale = o.grad_scale;
  a.lr = o.lr, a.eps = o.eps;
  a.b1 = (float)o.beta1, a.a1 = (float)(1.0 - o.beta1);
  a.b2 = (float)o.beta2, a.a2 = (float)(1.0 - o.beta2);
  a.beta1 = o.beta1, a.beta2 = o.beta2;
  a.turns = (int)turns, a.last = last;
  const long long ctas = ceil_of(turns, kWarps), most = 4ll * sms;
  const unsigned grid = (unsigned)(ctas < 1 ? 1 : ctas < most ? ctas : most);
  return launch_pdl(adamw_kernel<E4M3, PT, GT, MASTER, CAP>, dim3(grid), dim3(kThreads), 0, s, a);
}

template <bool E4M3, typename PT, typename GT, bool MASTER>
cudaError_t step_kind(const moe_adamw_t &o, const moe_adamw_tensor_t *t, const Pending &q,
                      bool last, StepState *state, cudaStream_t s) {
  return q.count <= kSmallCap ? step_cap<E4M3, PT, GT, MASTER, kSmallCap>(o, t, q, last, state, s)
                              : step_cap<E4M3, PT, GT, MASTER, kLargeCap>(o, t, q, last, state, s);
}

template <bool E4M3>
cudaError_t step_launch(const moe_adamw_t &o, const moe_adamw_tensor_t *t, Kind k, Pending &q,
                        bool last, StepState *st, cudaStream_t s) {
  using B = __nv_bfloat16;
  cudaError_t e;
  if (!k.param_bf16)
    e = k.grad_bf16 ? step_kind<E4M3, float, B, false>(o, t, q, last, st, s)
                    : step_kind<E4M3, float, float, false>(o, t, q, last, st, s);
  else if (k.master)
    e = k.grad_bf16 ? step_kind<E4M3, B, B, true>(o, t, q, last, st, s)
                    : step_kind<E4M3, B, float, true>(o, t, q, last, st, s);
  else
    e = k.grad_bf16 ? step_kind<E4M3, B, B, false>(o, t, q, last, st, s)
                    : step_kind<E4M3, B, float, false>(o, t, q, last, st, s);
  q.count = 0;
  return e;
}

template <bool E4M3>
cudaError_t step_all(const moe_adamw_t &o, const moe_adamw_tensor_t *t, int count,
                     StepState *state, cudaStream_t s) {
  // every kind's tensors, and which kind has the last launch
  int of[8] = {0};
  for (int i = 0; i < count; ++i) {
    const Kind k = kind_of(t[i]);
    if (t[i].numel) ++of[k.param_bf16 * 4 + k.grad_bf16 * 2 + k.master];
  }
  int left = 0;
  for (int n : of) left += n;
  Pending q;
  if (left == 0) return step_launch<E4M3>(o, t, Kind{false, false, false}, q, true, state, s);
  cudaError_t e = cudaSuccess;
  for (int id = 0; id < 8; ++id) {
    if (!of[id]) continue;
    const Kind k = {(id & 4) != 0, (id & 2) != 0, (id & 1) != 0};
    for (int i = 0; i < count && e == cudaSuccess; ++i) {
      const Kind x = kind_of(t[i]);
      if (!t[i].numel || x.param_bf16 != k.param_bf16 || x.grad_bf16 != k.grad_bf16 ||
          x.master != k.master)
        continue;
      q.index[q.count++] = i;
      --left, --of[id];
      if (q.count == kLargeCap || of[id] == 0) e = step_launch<E4M3>(o, t, k, q, left == 0, state, s);
    }
  }
  return e;
}

}  // namespace

size_t grad_norm_ws_bytes(int count) {
  const size_t launches = count < 1 ? 1 : (size_t)ceil_of(count, kLargeCap);
  return (launches * kNormCtas * sizeof(double) + 255) / 256 * 256;
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

cudaError_t launch_adamw(const moe_adamw_t &o, const moe_adamw_tensor_t *t, int count, void *state,
                         cudaStream_t s) {
  StepState *st = static_cast<StepState *>(state);
  return o.state_dtype == MOE_E4M3 ? step_all<true>(o, t, count, st, s)
                                   : step_all<false>(o, t, count, st, s);
}

}  // namespace moe
