// Layer norm of rows:
//   s = x + residual (rounded to the rows' type), mu = sum s / H (0 in the root
//   mean square form), r = 1 / sqrt(sum (s - mu)^2 / H + eps),
//   y = (s - mu) r w + b
//
// Bound: HBM, every value read once and written once.  A row stays in its
// group's registers between the sums and the result; weight and bias stay there
// over all rows of a persistent CTA.  One CTA an SM: its groups are at
// different points of their rows, which overlaps loads, sums and stores.
//
// Measured: 4096 rows of 2048 bf16 with residual (67 MB) 11.9 us, 5.6 TB/s;
// 8192 rows of 7168 42 us (5.6 TB/s), with residual 79 (5.9); 1777 rows of 1031
// float32 6.7 us, 4097 of 4099 bf16 with residual 34; one row of 2048 2.0.  A CTA
// per row without a ring took 34 us for the first; the float32 operations one by
// one, 63 for the second.
#include "norm.cuh"

namespace moe {
namespace {

struct NormArgs {
  const void *x, *res, *w, *b;
  long long xs, rs;  // elements between rows
  void *s, *y;
  float *stats;
  int n, H;
  bool wide, rms;  // float32 weight; no mean
  float eps;
  int phase;  // values from a row's beginning within 16 bytes to the next row's
  bool vec;   // weight and bias on 16 bytes
};

// N: tensors read (x; x and residual)
template <typename T, int GS, int VALS, bool SHIFT, int N, int D>
__global__ void __launch_bounds__(kCta<GS>) norm_kernel(const NormArgs a) {
  using IO = RowIO<T, GS, VALS, SHIFT, false>;
  pdl_enter();
  extern __shared__ __align__(16) char ring[];
  __shared__ __align__(16) float2 parts[2][kCta<GS> / 32];
  const int t = threadIdx.x % GS, group = threadIdx.x / GS, groups = blockDim.x / GS;
  const int H = a.H, first = threadIdx.x / GS * GS / 32;  // the group's first warp
  char *mine = ring + group * (D * N * IO::BYTES);
  const uint32_t mine32 = ptx::smem_u32(mine);
  const long long step = (long long)gridDim.x * groups;
  long long row = blockIdx.x + (long long)gridDim.x * group, ahead = row;
  const T *x_in = static_cast<const T *>(a.x) + row * a.xs;
  const T *res_in = static_cast<const T *>(a.res) + (N == 2 ? row * a.rs : 0);
  T *y = static_cast<T *>(a.y) + row * H, *s = static_cast<T *>(a.s) + (N == 2 ? row * H : 0);
  const IO io(H, t, (int)(row * a.phase % IO::V), 0, 0);
  auto issue = [&](int slot) {
    if (ahead < a.n) {
      const uint32_t to = mine32 + slot * (N * IO::BYTES);
      io.issue(to, x_in, a.xs, a.n - 1 - ahead);
      if (N == 2) io.issue(to + IO::BYTES, res_in, a.rs, a.n - 1 - ahead);
    }
    ptx::cp_async_commit();
    ahead += step, x_in += step * a.xs, res_in += N == 2 ? step * a.rs : 0;
  };
#pragma unroll 1
  for (int i = 0; i < D - 1; ++i) issue(i);
  float2 w[IO::P], b[IO::P];
  io.param(a.w, a.wide, a.vec, w);
  if (a.b) io.param(a.b, a.wide, a.vec, b);
  const float inv = 1.f / (float)H;
  // all groups of a CTA take the same number of turns: those of a warp share
  // its shuffles
  const int turns = (int)((a.n - blockIdx.x + step - 1) / step);
#pragma unroll 1
  for (int i = 0; i < turns; ++i) {
    issue((i + D - 1) % D);
    ptx::cp_async_wait<D - 1>();
    const bool on = row < a.n;
    const char *slot = mine + i % D * (N * IO::BYTES);
    float2 f[IO::P];
    io.template read<N == 1>(slot, f);
    if (N == 2) {
      float2 g[IO::P];
      io.template read<false>(slot + IO::BYTES, g);
#pragma unroll
      for (int k = 0; k < IO::P; ++k) f[k] = add2(f[k], g[k]);
#pragma unroll
      for (int c = 0; c < IO::PIECES; ++c) io.mask(c, f);
      IO::round(f);
      if (on) io.store(s, f);
    }
    float mu = 0.f, off = 0.f, var;
    if (!a.rms) {
      float2 sum = f[0];
#pragma unroll
      for (int k = 1; k < IO::P; ++k) sum = add2(sum, f[k]);
      mu = group_sum<GS>(sum.x + sum.y, parts[0] + first, group) * inv;
      // squares of the deviations from the mean; the deviations' own sum takes
      // out what rounding left in it
      float2 d = make_float2(0.f, 0.f), q = d;
      const float2 m = both(-mu);
#pragma unroll
      for (int k = 0; k < IO::P; ++k) f[k] = add2(f[k], m);
#pragma unroll
      for (int c = 0; c < IO::PIECES; ++c) io.mask(c, f);
      io.each([&](int, int k) {
        d = add2(d, f[k]);
        q = fma2(f[k], f[k], q);
      });
      const float2 v = group_sum<GS>(make_float2(d.x + d.y, q.x + q.y), parts[1] + first, group);
      off = v.x * inv;
      var = fmaf(-off, off, v.y * inv);
      var = var < 0.f ? 0.f : var;  // a NaN stays one
      mu += off;
    } else {
      float2 q = mul2(f[0], f[0]);
#pragma unroll
      for (int k = 1; k < IO::P; ++k) q = fma2(f[k], f[k], q);
      // one sum a row: places in turn
      var = group_sum<GS>(q.x + q.y, parts[i & 1] + first, group) * inv;
    }
    const float r = rsqrt_of(var + a.eps);
    if (on) {
      const float2 r2 = both(r), o2 = both(-off);
#pragma unroll
      for (int k = 0; k < IO::P; ++k) f[k] = mul2(a.rms ? f[k] : add2(f[k], o2), r2);
      if (a.b) {
#pragma unroll
        for (int k = 0; k < IO::P; ++k) f[k] = fma2(f[k], w[k], b[k]);
      } else {
#pragma unroll
        for (int k = 0; k < IO::P; ++k) f[k] = mul2(f[k], w[k]);
      }
      io.store(y, f);
      if (a.stats && t == 0) {
        a.stats[row] = mu;
        a.stats[(size_t)a.n + row] = r;
      }
    }
    row += step, y += step * H;
    if (N == 2) s += step * H;
  }
}

// Rows of any length and alignment: a CTA a row, read again for each of the
// three passes.
template <typename T>
__global__ void __launch_bounds__(1024) norm_long_kernel(const NormArgs a) {
  pdl_enter();
  __shared__ __align__(16) float2 parts[2][32];
  const long long row = blockIdx.x;
  const T *x = static_cast<const T *>(a.x) + row * a.xs;
  const T *res = a.res ? static_cast<const T *>(a.res) + row * a.rs : nullptr;
  T *s = a.res ? static_cast<T *>(a.s) + row * a.H : nullptr;
  T *y = static_cast<T *>(a.y) + row * a.H;
  const float inv = 1.f / (float)a.H;
  float2 sum = make_float2(0.f, 0.f);
  for (int i = threadIdx.x; i < a.H; i += 1024) {
    float f = to_f(x[i]);
    if (res) {
      const T v = from_f<T>(f + to_f(res[i]));
      s[i] = v;
      f = to_f(v);
    }
    sum.x += f;
  }
  const T *in = res ? s : x;  // a thread's own values
  float mu = group_sum<1024>(sum.x, parts[0], 0) * inv;
  if (a.rms) mu = 0.f;
  sum = make_float2(0.f, 0.f);
  for (int i = threadIdx.x; i < a.H; i += 1024) {
    const float d = to_f(in[i]) - mu;
    sum.x += d;
    sum.y = fmaf(d, d, sum.y);
  }
  sum = group_sum<1024>(sum, parts[1], 0);
  float var = sum.y * inv;
  if (!a.rms) {
    const float off = sum.x * inv;
    var = fmaf(-off, off, var);
    var = var < 0.f ? 0.f : var;
    mu += off;
  }
  const float r = rsqrt_of(var + a.eps);
  auto param = [&](const void *p, int i) {
    return a.wide ? static_cast<const float *>(p)[i] : to_f(static_cast<const T *>(p)[i]);
  };
  for (int i = threadIdx.x; i < a.H; i += 1024) {
    const float xh = (to_f(in[i]) - mu) * r, w = param(a.w, i);
    y[i] = from_f<T>(a.b ? fmaf(xh, w, param(a.b, i)) : xh * w);
  }
  if (a.stats && threadIdx.x == 0) {
    a.stats[row] = mu;
    a.stats[(size_t)a.n + row] = r;
  }
}

template <typename T, int GS, int VALS, bool SHIFT, bool>
struct Forward {
  template <int N>
  static bool with(const NormArgs &a, cudaStream_t s, cudaError_t *e) {
    // 4096 rows of 2048 bf16 with residual: three slots 11.7 us, two 12.1, four
    // 13.2; shifted, bf16 with residual: 4097 x 4099 four 34 us, three 35; 21859 x
    // 1535 49 and 57; 11646 x 2881 51 and 59 (14588 x 2300 45 and 43; float32 the
    // same on both)
    constexpr int D = ring_slots<T, GS, VALS, N>(SHIFT ? 4 : 3);
    if constexpr (D == 0) {
      return false;
    } else {
      const NormGrid g = norm_grid<GS>(a.n, device_sm_count());
      constexpr int one = D * N * RowIO<T, GS, VALS, SHIFT, false>::BYTES;
      auto kernel = norm_kernel<T, GS, VALS, SHIFT, N, D>;
      static bool ready[64] = {false};
      *e = allow_smem(kernel, one * (kCta<GS> / GS), ready);
      if (*e == cudaSuccess)
        *e = launch_pdl(kernel, dim3(g.ctas), dim3(g.groups * GS), one * g.groups, s, a);
      return true;
    }
  }
  static bool go(const NormArgs &a, int, cudaStream_t s, cudaError_t *e) {
    return a.res ? with<2>(a, s, e) : with<1>(a, s, e);
  }
};

template <typename T>
cudaError_t forward(NormArgs &a, cudaStream_t s) {
  Phases ph(kPer<T>);
  ph.add(a.x, a.xs), ph.add(a.res, a.rs), ph.add(a.s, a.H), ph.add(a.y, a.H);
  a.phase = ph.step;
  a.vec = on_bytes(a.w, 16) && on_bytes(a.b, 16);
  cudaError_t e = cudaSuccess;
  if (ph.one && (ph.step || a.H % kPer<T> ? by_length<false, T, true, Forward>(a, s, &e)
                                      : by_length<false, T, false, Forward>(a, s, &e))) return e;
  return launch_pdl(norm_long_kernel<T>, dim3(a.n), dim3(1024), 0, s, a);
}

}  // namespace

cudaError_t launch_norm(const moe_norm_t &d, const void *x, long long x_stride,
                        const void *residual, long long residual_stride, const void *weight,
                        const void *bias, void *s, void *y, float *stats, cudaStream_t st) {
  if (d.n == 0) return cudaSuccess;
  NormArgs a = {x, residual, weight, bias, x_stride, residual_stride, s, y, stats, d.n, d.H,
                d.weight_dtype == MOE_F32, d.rms != 0, d.eps, 0, false};
  return d.dtype == MOE_F32 ? forward<float>(a, st) : forward<__nv_bfloat16>(a, st);
}

}  // namespace moe
