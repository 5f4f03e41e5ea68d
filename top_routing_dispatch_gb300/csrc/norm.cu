// Layer norm of rows, and its gradients:
//   s = x + residual (rounded to the rows' type), mu = sum s / H (0 in the root
//   mean square form), r = 1 / sqrt(sum (s - mu)^2 / H + eps),
//   y = (s - mu) r w + b;
//   xh = (s - mu) r, t = dy w, dx = r (t - sum t / H - xh sum(t xh) / H) + ds,
//   dw = sum over rows of dy xh, db = sum over rows of dy.
//
// A row belongs to a group of GS threads of one CTA and stays in their
// registers between the sums and the result.
#include "train.cuh"

namespace moe {
namespace {

// Values of a row in 16-byte chunks (VEC), or one by one where rows do not
// start on 16-byte boundaries: then neighbouring threads hold neighbouring
// values, so that a warp still reads whole sectors.
template <typename T>
constexpr int kPer = 16 / (int)sizeof(T);

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f<float>(float v) {
  return v;
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}

template <typename T, int GS, bool VEC>
struct Rows {
  static constexpr int V = kPer<T>;
  // position of value j of chunk c of the group's thread t
  static __device__ __forceinline__ int at(int c, int j, int t) {
    return VEC ? (c * GS + t) * V + j : (c * V + j) * GS + t;
  }
  static __device__ __forceinline__ void load(const T *row, int c, int t, int H, bool on,
                                              float (&f)[V]) {
    if (VEC) {
      uint4 u = make_uint4(0, 0, 0, 0);
      if (on && at(c, 0, t) < H) u = __ldg(reinterpret_cast<const uint4 *>(row + at(c, 0, t)));
      const T *p = reinterpret_cast<const T *>(&u);
#pragma unroll
      for (int j = 0; j < V; ++j) f[j] = to_f(p[j]);
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) f[j] = on && at(c, j, t) < H ? to_f(row[at(c, j, t)]) : 0.f;
    }
  }
  static __device__ __forceinline__ void store(T *row, int c, int t, int H, bool on,
                                               const float (&f)[V]) {
    if (VEC) {
      uint4 u;
      T *p = reinterpret_cast<T *>(&u);
#pragma unroll
      for (int j = 0; j < V; ++j) p[j] = from_f<T>(f[j]);
      if (on && at(c, 0, t) < H) *reinterpret_cast<uint4 *>(row + at(c, 0, t)) = u;
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (on && at(c, j, t) < H) row[at(c, j, t)] = from_f<T>(f[j]);
    }
  }
  // weight or bias at the same places
  static __device__ __forceinline__ void param(const void *w, bool wide, int c, int t, int H,
                                               float (&f)[V]) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int i = at(c, j, t);
      f[j] = i >= H ? 0.f
             : wide ? __ldg(static_cast<const float *>(w) + i)
                    : to_f(static_cast<const T *>(w)[i]);
    }
  }
};

// Sums of two values over the group, the same in every thread of it.  Groups
// of more than a warp are whole CTAs: `part` holds a value per warp, and two
// of them are used in turn so that one barrier a sum is enough.
template <int GS>
__device__ __forceinline__ float2 group_sum(float2 v, float2 *part) {
#pragma unroll
  for (int o = (GS < 32 ? GS : 32) / 2; o > 0; o /= 2) {
    v.x += __shfl_xor_sync(~0u, v.x, o);
    v.y += __shfl_xor_sync(~0u, v.y, o);
  }
  if (GS <= 32) return v;
  constexpr int W = GS > 32 ? GS / 32 : 1;
  if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = v;
  __syncthreads();
  float2 a = threadIdx.x % 32 < W ? part[threadIdx.x % 32] : make_float2(0.f, 0.f);
#pragma unroll
  for (int o = 16; o > 0; o /= 2) {
    a.x += __shfl_xor_sync(~0u, a.x, o);
    a.y += __shfl_xor_sync(~0u, a.y, o);
  }
  return a;
}

struct NormArgs {
  const void *x, *res, *w, *b;
  long long xs, rs;  // elements between rows
  void *s, *y;
  float *stats;
  int n, H;
  bool wide, rms;  // float32 weight; no mean
  float eps;
};

// CH chunks a thread in registers; CH = 0: rows of any length, read again for
// each of the three passes.
template <typename T, int GS, int CH, bool VEC>
__global__ void __launch_bounds__(GS < 128 ? 128 : GS) norm_kernel(const NormArgs a) {
  pdl_enter();
  using R = Rows<T, GS, VEC>;
  constexpr int V = R::V, CTA = GS < 128 ? 128 : GS, LIVE = CH ? CH : 1;
  __shared__ float2 part[2][32];
  const int t = threadIdx.x % GS;
  const long long row = (long long)blockIdx.x * (CTA / GS) + threadIdx.x / GS;
  const bool on = row < a.n;
  const T *x = static_cast<const T *>(a.x) + row * a.xs;
  const T *res = a.res ? static_cast<const T *>(a.res) + row * a.rs : nullptr;
  T *s = a.res ? static_cast<T *>(a.s) + row * a.H : nullptr;
  T *y = static_cast<T *>(a.y) + row * a.H;
  const int chunks = CH ? CH : (a.H + GS * V - 1) / (GS * V);
  const float inv = 1.f / (float)a.H;
  float f[LIVE][V];
  auto fetch = [&](int c, float(&g)[V], bool first) {
    if (!res || first) R::load(x, c, t, a.H, on, g);
    if (!res) return;
    if (first) {  // the sum, rounded as it is stored
      float q[V];
      R::load(res, c, t, a.H, on, q);
#pragma unroll
      for (int j = 0; j < V; ++j) g[j] = to_f(from_f<T>(g[j] + q[j]));
      R::store(s, c, t, a.H, on, g);
    } else {  // written by this thread; not through the read-only path
#pragma unroll
      for (int j = 0; j < V; ++j)
        g[j] = on && R::at(c, j, t) < a.H ? to_f(s[R::at(c, j, t)]) : 0.f;
    }
  };
  float2 sum = make_float2(0.f, 0.f);
#pragma unroll
  for (int c = 0; c < chunks; ++c) {
    fetch(c, f[CH ? c : 0], true);
    if (!a.rms) {
#pragma unroll
      for (int j = 0; j < V; ++j) sum.x += f[CH ? c : 0][j];
    }
  }
  // mean, then squares of the deviations from it.  The deviations' own sum
  // takes out what rounding left in the mean.
  float mu = a.rms ? 0.f : group_sum<GS>(sum, part[0]).x * inv;
  sum = make_float2(0.f, 0.f);
#pragma unroll
  for (int c = 0; c < chunks; ++c) {
    if (!CH) fetch(c, f[0], false);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const float d = R::at(c, j, t) < a.H ? f[CH ? c : 0][j] - mu : 0.f;
      sum.x += d;
      sum.y = fmaf(d, d, sum.y);
    }
  }
  sum = group_sum<GS>(sum, part[1]);
  float var = sum.y * inv;
  if (!a.rms) {
    const float off = sum.x * inv;
    var = fmaf(-off, off, var);
    var = var < 0.f ? 0.f : var;  // a NaN stays one
    mu += off;
  }
  const float r = 1.f / sqrtf(var + a.eps);
#pragma unroll
  for (int c = 0; c < chunks; ++c) {
    if (!CH) fetch(c, f[0], false);
    float w[V], b[V], o[V];
    R::param(a.w, a.wide, c, t, a.H, w);
    if (a.b) R::param(a.b, a.wide, c, t, a.H, b);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const float xh = (f[CH ? c : 0][j] - mu) * r;
      o[j] = a.b ? fmaf(xh, w[j], b[j]) : xh * w[j];
    }
    R::store(y, c, t, a.H, on, o);
  }
  if (a.stats && on && t == 0) {
    a.stats[row] = mu;
    a.stats[(size_t)a.n + row] = r;
  }
}

struct NormBackArgs {
  const void *dy, *s, *w, *ds;
  long long dys, ss, dss;
  const float *stats;
  void *dx;
  float *part;  // (2, parts, H) sums of row ranges for dweight and dbias
  int n, H, parts;
  bool wide, rms, bias;
};

// dx of a row
template <typename T, int GS, int CH, bool VEC>
__global__ void __launch_bounds__(GS < 128 ? 128 : GS) norm_dx_kernel(const NormBackArgs a) {
  pdl_enter();
  using R = Rows<T, GS, VEC>;
  constexpr int V = R::V, CTA = GS < 128 ? 128 : GS, LIVE = CH ? CH : 1;
  __shared__ float2 part[1][32];
  const int t = threadIdx.x % GS;
  const long long row = (long long)blockIdx.x * (CTA / GS) + threadIdx.x / GS;
  const bool on = row < a.n;
  const T *x = static_cast<const T *>(a.s) + row * a.ss;
  const T *dy = static_cast<const T *>(a.dy) + row * a.dys;
  const int chunks = CH ? CH : (a.H + GS * V - 1) / (GS * V);
  const float inv = 1.f / (float)a.H;
  const float mu = on && !a.rms ? a.stats[row] : 0.f;
  const float r = on ? a.stats[(size_t)a.n + row] : 0.f;
  float xh[LIVE][V], tw[LIVE][V];
  auto fetch = [&](int c, float(&h)[V], float(&g)[V]) {
    float w[V];
    R::load(x, c, t, a.H, on, h);
    R::load(dy, c, t, a.H, on, g);
    R::param(a.w, a.wide, c, t, a.H, w);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      h[j] = (h[j] - mu) * r;
      g[j] *= w[j];  // 0 behind the row's end
    }
  };
  float2 sum = make_float2(0.f, 0.f);
#pragma unroll
  for (int c = 0; c < chunks; ++c) {
    const int k = CH ? c : 0;
    fetch(c, xh[k], tw[k]);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      if (R::at(c, j, t) < a.H) {
        sum.x += tw[k][j];
        sum.y = fmaf(tw[k][j], xh[k][j], sum.y);
      }
    }
  }
  sum = group_sum<GS>(sum, part[0]);
  const float c1 = a.rms ? 0.f : sum.x * inv, c2 = sum.y * inv;
#pragma unroll
  for (int c = 0; c < chunks; ++c) {
    const int k = CH ? c : 0;
    if (!CH) fetch(c, xh[0], tw[0]);
    float o[V];
#pragma unroll
    for (int j = 0; j < V; ++j) o[j] = r * (tw[k][j] - c1 - xh[k][j] * c2);
    if (a.ds) {
      float d[V];
      R::load(static_cast<const T *>(a.ds) + row * a.dss, c, t, a.H, on, d);
#pragma unroll
      for (int j = 0; j < V; ++j) o[j] += d[j];
    }
    R::store(static_cast<T *>(a.dx) + row * a.H, c, t, a.H, on, o);
  }
}

constexpr int kWarps = 8;       // of a column kernel's CTA
constexpr int kMaxParts = 304;  // row ranges whose sums are added at the end

// Sums of dy xh and of dy over a range of rows, 32 columns a CTA
template <typename T>
__global__ void __launch_bounds__(32 * kWarps) norm_columns_kernel(const NormBackArgs a) {
  pdl_enter();
  __shared__ float sw[kWarps][32], sb[kWarps][32];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int col = blockIdx.x * 32 + lane;
  const int r0 = (int)((long long)a.n * blockIdx.y / a.parts);
  const int r1 = (int)((long long)a.n * (blockIdx.y + 1) / a.parts);
  float dw = 0.f, db = 0.f;
  if (col < a.H) {
    for (int row = r0 + warp; row < r1; row += kWarps) {
      const float mu = a.rms ? 0.f : a.stats[row], r = a.stats[(size_t)a.n + row];
      const float x = to_f(static_cast<const T *>(a.s)[row * a.ss + col]);
      const float dy = to_f(static_cast<const T *>(a.dy)[row * a.dys + col]);
      dw = fmaf(dy, (x - mu) * r, dw);
      db += dy;
    }
  }
  sw[warp][lane] = dw, sb[warp][lane] = db;
  __syncthreads();
  if (warp || col >= a.H) return;
#pragma unroll
  for (int i = 1; i < kWarps; ++i) dw += sw[i][lane], db += sb[i][lane];
  a.part[(size_t)blockIdx.y * a.H + col] = dw;
  if (a.bias) a.part[((size_t)a.parts + blockIdx.y) * a.H + col] = db;
}

// dweight (blockIdx.y 0) and dbias (1): the parts in a fixed order
__global__ void __launch_bounds__(32 * kWarps)
    norm_join_kernel(const float *part, int parts, int H, float *dweight, float *dbias) {
  pdl_enter();
  __shared__ float acc[kWarps][32];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int col = blockIdx.x * 32 + lane;
  float *out = blockIdx.y ? dbias : dweight;
  const float *p = part + (size_t)blockIdx.y * parts * H + col;
  float v = 0.f;
  if (out && col < H)
    for (int i = warp; i < parts; i += kWarps) v += p[(size_t)i * H];
  acc[warp][lane] = v;
  __syncthreads();
  if (warp || !out || col >= H) return;
#pragma unroll
  for (int i = 1; i < kWarps; ++i) v += acc[i][lane];
  out[col] = v;
}

int parts_of(int n) { return n < 1 ? 1 : n < kMaxParts ? n : kMaxParts; }

// The group of threads that takes a row: the smallest that holds it at up to
// four chunks a thread.
template <template <typename, int, int, bool> class Launch, typename T, bool VEC, typename A>
cudaError_t by_length(const A &a, cudaStream_t st) {
  const int c = (a.H + kPer<T> - 1) / kPer<T>;
  if (c <= 8) return Launch<T, 8, 1, VEC>::go(a, st);
  if (c <= 16) return Launch<T, 16, 1, VEC>::go(a, st);
  if (c <= 32) return Launch<T, 32, 1, VEC>::go(a, st);
  if (c <= 64) return Launch<T, 32, 2, VEC>::go(a, st);
  if (c <= 128) return Launch<T, 32, 4, VEC>::go(a, st);
  if (c <= 512) return Launch<T, 128, 4, VEC>::go(a, st);
  if (c <= 1024) return Launch<T, 256, 4, VEC>::go(a, st);
  if (c <= 2048) return Launch<T, 512, 4, VEC>::go(a, st);
  return Launch<T, 1024, 0, VEC>::go(a, st);
}

template <int GS>
dim3 rows_grid(int n) {
  constexpr int per = GS < 128 ? 128 / GS : 1;
  return dim3((unsigned)((n + per - 1) / per));
}

template <typename T, int GS, int CH, bool VEC>
struct Forward {
  static cudaError_t go(const NormArgs &a, cudaStream_t st) {
    return launch_pdl(norm_kernel<T, GS, CH, VEC>, rows_grid<GS>(a.n), dim3(GS < 128 ? 128 : GS), 0,
                      st, a);
  }
};
template <typename T, int GS, int CH, bool VEC>
struct Backward {
  static cudaError_t go(const NormBackArgs &a, cudaStream_t st) {
    return launch_pdl(norm_dx_kernel<T, GS, CH, VEC>, rows_grid<GS>(a.n),
                      dim3(GS < 128 ? 128 : GS), 0, st, a);
  }
};

bool on16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

}  // namespace

size_t norm_backward_ws_bytes(const moe_norm_t &d) {
  return 2 * sizeof(float) * (size_t)parts_of(d.n) * d.H;
}

cudaError_t launch_norm(const moe_norm_t &d, const void *x, long long x_stride,
                        const void *residual, long long residual_stride, const void *weight,
                        const void *bias, void *s, void *y, float *stats, cudaStream_t st) {
  if (d.n == 0) return cudaSuccess;
  NormArgs a = {x, residual, weight, bias, x_stride, residual_stride, s, y, stats, d.n, d.H,
                d.weight_dtype == MOE_F32, d.rms != 0, d.eps};
  const int per = d.dtype == MOE_F32 ? 4 : 8;
  const bool vec = d.H % per == 0 && x_stride % per == 0 && on16(x) && on16(y) && on16(weight) &&
                   on16(bias) && (!residual || (residual_stride % per == 0 && on16(residual) && on16(s)));
  if (d.dtype == MOE_F32)
    return vec ? by_length<Forward, float, true>(a, st) : by_length<Forward, float, false>(a, st);
  return vec ? by_length<Forward, __nv_bfloat16, true>(a, st)
             : by_length<Forward, __nv_bfloat16, false>(a, st);
}

cudaError_t launch_norm_backward(const moe_norm_t &d, const void *dy, long long dy_stride,
                                 const void *s, long long s_stride, const float *stats,
                                 const void *weight, const void *ds, long long ds_stride, void *dx,
                                 float *dweight, float *dbias, void *ws, cudaStream_t st) {
  if (d.n == 0) {
    cudaError_t e = cudaMemsetAsync(dweight, 0, sizeof(float) * d.H, st);
    if (e == cudaSuccess && dbias) e = cudaMemsetAsync(dbias, 0, sizeof(float) * d.H, st);
    return e;
  }
  NormBackArgs a = {dy, s, weight, ds, dy_stride, s_stride, ds_stride, stats, dx,
                    static_cast<float *>(ws), d.n, d.H, parts_of(d.n),
                    d.weight_dtype == MOE_F32, d.rms != 0, dbias != nullptr};
  const int per = d.dtype == MOE_F32 ? 4 : 8;
  const bool vec = d.H % per == 0 && dy_stride % per == 0 && s_stride % per == 0 && on16(dy) &&
                   on16(s) && on16(dx) && on16(weight) &&
                   (!ds || (ds_stride % per == 0 && on16(ds)));
  const dim3 cols((d.H + 31) / 32, a.parts), cta(32 * kWarps);
  // the sums first: dx may lie where ds does
  cudaError_t e = d.dtype == MOE_F32
                      ? launch_pdl(norm_columns_kernel<float>, cols, cta, 0, st, a)
                      : launch_pdl(norm_columns_kernel<__nv_bfloat16>, cols, cta, 0, st, a);
  if (e == cudaSuccess)
    e = launch_pdl(norm_join_kernel, dim3((d.H + 31) / 32, dbias ? 2 : 1), cta, 0, st,
                   (const float *)a.part, a.parts, d.H, dweight, dbias);
  if (e != cudaSuccess) return e;
  if (d.dtype == MOE_F32)
    return vec ? by_length<Backward, float, true>(a, st) : by_length<Backward, float, false>(a, st);
  return vec ? by_length<Backward, __nv_bfloat16, true>(a, st)
             : by_length<Backward, __nv_bfloat16, false>(a, st);
}

}  // namespace moe
