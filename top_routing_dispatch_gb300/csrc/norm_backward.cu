// Gradients of the layer norm: xh = (s - mu) r, t = dy w,
//   dx = r (t - sum t / H - xh sum(t xh) / H) + ds,
//   dw = sum over rows of dy xh, db = sum over rows of dy.
//
// Bound: HBM, every value read once and written once; instructions come next
// (31 a value of a long row).  A group of threads keeps its columns' sums for dw
// and db in registers over all its rows; the groups of a CTA join them in
// shared memory, the CTAs through one float32 row each in the workspace, added
// in a fixed order by a second kernel.  A separate pass for dw and db would read
// s and dy twice.
//
// Rows of more than 8192 values belong to clusters of CTAs; their sums' barrier
// bounds them (bf16 with ds, a row of a cluster: 2.4 us at 8200 values and 3.0 at
// 16384 on two CTAs, 3.3 at 32768 on four, 4.0 at 65528 on eight).
//
// Measured, both kernels: 4096 rows of 2048 bf16 with ds (67 MB) 16.9 us, of
// which 1.6 store the ranges' sums and 2.6 add them; 8192 rows of 7168 (470 MB)
// 79 us, 6.0 TB/s; 4096 rows of 16384 (537 MB) 158 us, 3.4 TB/s; 152 rows of
// 7168 7.5 us; 301 rows of 1031 float32 7.2.  Two passes (a CTA a row, then
// columns) took 58 us for the first and 286 for the second.
#include "norm.cuh"

namespace moe {
namespace {

struct BackArgs {
  const void *dy, *s, *w, *ds;
  long long dys, ss, dss;  // elements between rows
  const float *stats;
  void *dx;
  float *part;  // (2, parts, H) sums for dweight and dbias
  int n, H, parts;
  bool wide, rms, bias;
  int phase;  // as in the forward
  bool vec;   // weight on 16 bytes
};

// N: tensors read (dy and s; and ds)
template <typename T, int GS, int VALS, bool SHIFT, bool CLUSTER, int N, int D>
__global__ void __launch_bounds__(kCta<GS>) norm_back_kernel(const BackArgs a) {
  using IO = RowIO<T, GS, VALS, SHIFT, CLUSTER>;
  pdl_enter();
  extern __shared__ __align__(16) char ring[];
  __shared__ __align__(16) float2 parts[2][(CLUSTER ? kMostCluster : 1) * kCta<GS> / 32];
  const int t = threadIdx.x % GS, group = threadIdx.x / GS, groups = blockDim.x / GS;
  const int H = a.H, first = threadIdx.x / GS * GS / 32;
  char *mine = ring + group * (D * N * IO::BYTES);
  const uint32_t mine32 = ptx::smem_u32(mine);
  const Share<GS, VALS, IO::V, CLUSTER> share(H + (SHIFT ? IO::V - 1 : 0));
  const long long step = (long long)share.count * groups;
  long long row = share.index + (long long)share.count * group, ahead = row;
  const T *dy_in = static_cast<const T *>(a.dy) + row * a.dys;
  const T *s_in = static_cast<const T *>(a.s) + row * a.ss;
  const T *ds_in = static_cast<const T *>(a.ds) + (N == 3 ? row * a.dss : 0);
  const IO io(H, t, (int)(row * a.phase % IO::V), share.base, share.part);
  T *dx = static_cast<T *>(a.dx) + row * H;
  auto issue = [&](int slot) {
    if (ahead < a.n) {
      const uint32_t to = mine32 + slot * (N * IO::BYTES);
      const long long behind = a.n - 1 - ahead;
      io.issue(to, dy_in, a.dys, behind);
      io.issue(to + IO::BYTES, s_in, a.ss, behind);
      if (N == 3) io.issue(to + 2 * IO::BYTES, ds_in, a.dss, behind);
    }
    ptx::cp_async_commit();
    ahead += step, dy_in += step * a.dys, s_in += step * a.ss;
    if (N == 3) ds_in += step * a.dss;
  };
#pragma unroll 1
  for (int i = 0; i < D - 1; ++i) issue(i);
  if (CLUSTER) __syncwarp(), ptx::cluster_sync();  // the other CTAs' shared memory is there
  auto sum_of = [&](auto v, float2 *places) {
    if constexpr (CLUSTER)
      return cluster_sum<GS>(v, places, share.size, share.rank);
    else
      return group_sum<GS>(v, places + first, group);
  };
  float2 w[IO::P], dw[IO::P], db[IO::P];
  io.param(a.w, a.wide, a.vec, w);
#pragma unroll
  for (int k = 0; k < IO::P; ++k) dw[k] = db[k] = make_float2(0.f, 0.f);
  const float inv = 1.f / (float)H;
  const int turns = (int)((a.n - share.index + step - 1) / step);
  // the statistics of the next row are on their way during a row
  float mu_in = 0.f, r_in = 0.f;
  auto stats = [&](long long at) {
    if (at < a.n) {
      if (!a.rms) mu_in = __ldg(a.stats + at);
      r_in = __ldg(a.stats + a.n + at);
    }
  };
  stats(row);
#pragma unroll 1
  for (int i = 0; i < turns; ++i) {
    const bool on = row < a.n;
    const float2 mu = both(-mu_in), r = both(r_in);
    stats(row + step);
    issue((i + D - 1) % D);
    ptx::cp_async_wait<D - 1>();
    const char *slot = mine + i % D * (N * IO::BYTES);
    // with d = s - mu and g = dy r: r t = g w, and the sums of r t and r t d
    // give r c1 and c2
    float2 g[IO::P], d[IO::P];
    float2 s1 = make_float2(0.f, 0.f), s2 = s1;
    // `sums` is always true, but without it the compiler orders this part of the
    // kernel on 1024 threads so that 4096 rows of 8192 bf16 take 56 us instead of
    // 47 (the other group sizes and the clusters take the same)
    auto fetch = [&](bool sums) {
      io.template read<true>(slot, g);
      io.template read<false>(slot + IO::BYTES, d);
#pragma unroll
      for (int k = 0; k < IO::P; ++k) d[k] = add2(d[k], mu);
#pragma unroll
      for (int c = 0; c < IO::PIECES; ++c) io.mask(c, d);
      io.each([&](int, int k) {
        if (sums) db[k] = add2(db[k], g[k]);
        g[k] = mul2(g[k], r);
        if (sums) dw[k] = fma2(g[k], d[k], dw[k]);
        g[k] = mul2(g[k], w[k]);
        if (sums) s1 = add2(s1, g[k]), s2 = fma2(g[k], d[k], s2);
      });
    };
    if (on) fetch(true);
    s1 = sum_of(make_float2(s1.x + s1.y, s2.x + s2.y), parts[i & 1]);
    if (on) {
      const float2 c1 = both(a.rms ? 0.f : -s1.x * inv), c2 = both(-s1.y * inv * r.x * r.x);
#pragma unroll
      for (int k = 0; k < IO::P; ++k) g[k] = fma2(d[k], c2, add2(g[k], c1));
      if (N == 3) {
        io.template read<false>(slot + 2 * IO::BYTES, d);
#pragma unroll
        for (int k = 0; k < IO::P; ++k) g[k] = add2(g[k], d[k]);
      }
      io.store(dx, g);
    }
    row += step, dx += step * H;
  }
  // the CTA's (or cluster's) sums, group by group
  float *out = a.part + (size_t)share.index * H;
  if (groups > 1) {
    ptx::cp_async_wait<0>();
    __syncthreads();
    float *all = reinterpret_cast<float *>(ring), *all_b = all + groups * H;
    io.put(all + group * H, H % 4 == 0, dw);
    if (a.bias) io.put(all_b + group * H, H % 4 == 0, db);
    __syncthreads();
    for (int c = threadIdx.x; c < H; c += blockDim.x) {
      float v = all[c];
      for (int q = 1; q < groups; ++q) v += all[q * H + c];
      out[c] = v;
      if (a.bias) {
        v = all_b[c];
        for (int q = 1; q < groups; ++q) v += all_b[q * H + c];
        out[(size_t)a.parts * H + c] = v;
      }
    }
    return;
  }
  io.put(out, H % 4 == 0, dw);
  if (a.bias) io.put(out + (size_t)a.parts * H, H % 4 == 0, db);
}

// Rows of any length and alignment, second part: dx, a CTA a row.
template <typename T>
__global__ void __launch_bounds__(1024) norm_back_long_kernel(const BackArgs a) {
  pdl_enter();
  __shared__ __align__(16) float2 parts[32];
  const long long row = blockIdx.x;
  const T *dy = static_cast<const T *>(a.dy) + row * a.dys;
  const T *s = static_cast<const T *>(a.s) + row * a.ss;
  const T *ds = a.ds ? static_cast<const T *>(a.ds) + row * a.dss : nullptr;
  T *dx = static_cast<T *>(a.dx) + row * a.H;
  const float mu = a.rms ? 0.f : a.stats[row], r = a.stats[(size_t)a.n + row];
  const float inv = 1.f / (float)a.H;
  auto weight = [&](int i) {
    return a.wide ? static_cast<const float *>(a.w)[i] : to_f(static_cast<const T *>(a.w)[i]);
  };
  float2 sum = make_float2(0.f, 0.f);
  for (int i = threadIdx.x; i < a.H; i += 1024) {
    const float v = to_f(dy[i]) * weight(i);
    sum.x += v;
    sum.y = fmaf(v, (to_f(s[i]) - mu) * r, sum.y);
  }
  sum = group_sum<1024>(sum, parts, 0);
  const float c1 = a.rms ? 0.f : sum.x * inv, c2 = sum.y * inv;
  for (int i = threadIdx.x; i < a.H; i += 1024) {
    const float v = r * (to_f(dy[i]) * weight(i) - c1 - (to_f(s[i]) - mu) * r * c2);
    dx[i] = from_f<T>(ds ? v + to_f(ds[i]) : v);
  }
}

constexpr int kWarps = 8;  // of a column kernel's CTA

// First part: sums of dy xh and of dy over a range of rows, 32 columns a CTA
template <typename T>
__global__ void __launch_bounds__(32 * kWarps) norm_columns_kernel(const BackArgs a) {
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

// dweight (blockIdx.y 0) and dbias (1): the parts in a fixed order, 32 columns a
// CTA.  Bound: latency.  Every warp's few parts are asked for at once, then
// each warp adds one column's sums (4096 x 2048: 32 warps 2.9 us, 8 4.6).
__global__ void __launch_bounds__(1024)
    norm_join_kernel(const float *part, int parts, int H, float *dweight, float *dbias) {
  pdl_enter();
  __shared__ float acc[32][33];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int col = blockIdx.x * 32 + lane;
  float *out = blockIdx.y ? dbias : dweight;
  const float *p = part + (size_t)blockIdx.y * parts * H + col;
  float v = 0.f;
  if (col < H) {
#pragma unroll 5
    for (int i = warp; i < parts; i += 32) v += p[(size_t)i * H];
  }
  acc[warp][lane] = v;
  __syncthreads();
  v = acc[lane][warp];
#pragma unroll
  for (int o = 16; o > 0; o /= 2) v += __shfl_xor_sync(~0u, v, o);
  if (lane == 0 && blockIdx.x * 32 + warp < H) out[blockIdx.x * 32 + warp] = v;
}

template <typename T, int GS, int VALS, bool SHIFT, bool CLUSTER>
struct Backward {
  template <int N>
  static bool with(BackArgs &a, int size, cudaStream_t s, cudaError_t *e) {
    // 8192 rows of 7168 bf16 with ds: four slots 84 us, three 101
    constexpr int D = ring_slots<T, GS, VALS, N>(4);
    if constexpr (D == 0) {
      return false;
    } else {
      constexpr int one = D * N * RowIO<T, GS, VALS, SHIFT, CLUSTER>::BYTES;
      // the groups' sums are joined in the ring
      static_assert(one >= 2 * GS * VALS * 4, "ring");
      auto kernel = norm_back_kernel<T, GS, VALS, SHIFT, CLUSTER, N, D>;
      static bool ready[64] = {false};
      *e = allow_smem(kernel, one * (kCta<GS> / GS), ready);
      if (*e != cudaSuccess) return true;
      if constexpr (CLUSTER) {
        static int resident[64][kMostCluster + 1] = {};
        *e = cluster_grid(kernel, GS, one, size, a.n, kNormParts, SHIFT ? kPer<T> : 1, resident, &a.parts);
        if (*e == cudaSuccess) *e = launch_pdl_cluster(kernel, a.parts, size, GS, one, s, a);
      } else {
        const int sms = device_sm_count();
        const NormGrid g = norm_grid<GS>(a.n, sms < kNormParts ? sms : kNormParts);
        a.parts = g.ctas;
        *e = launch_pdl(kernel, dim3(g.ctas), dim3(g.groups * GS), one * g.groups, s, a);
      }
      return true;
    }
  }
  static bool go(BackArgs &a, int size, cudaStream_t s, cudaError_t *e) {
    return a.ds ? with<3>(a, size, s, e) : with<2>(a, size, s, e);
  }
};

template <typename T>
cudaError_t backward(BackArgs &a, float *dweight, float *dbias, cudaStream_t s) {
  Phases ph(kPer<T>);
  ph.add(a.dy, a.dys), ph.add(a.s, a.ss), ph.add(a.ds, a.dss), ph.add(a.dx, a.H);
  a.phase = ph.step;
  a.vec = on_bytes(a.w, 16);
  cudaError_t e = cudaSuccess;
  if (!ph.one || !(ph.step || a.H % kPer<T> ? by_length<true, T, true, Backward>(a, s, &e)
                                          : by_length<true, T, false, Backward>(a, s, &e))) {
    e = launch_pdl(norm_columns_kernel<T>, dim3((a.H + 31) / 32, a.parts), dim3(32 * kWarps), 0,
                   s, a);
    if (e == cudaSuccess)
      e = launch_pdl(norm_back_long_kernel<T>, dim3(a.n), dim3(1024), 0, s, a);
  }
  if (e != cudaSuccess) return e;
  return launch_pdl(norm_join_kernel, dim3((a.H + 31) / 32, dbias ? 2 : 1), dim3(1024), 0, s,
                     (const float *)a.part, a.parts, a.H, dweight, dbias);
}

}  // namespace

size_t norm_backward_ws_bytes(const moe_norm_t &d) {
  const int parts = d.n < 1 ? 1 : d.n < kNormParts ? d.n : kNormParts;
  return 2 * sizeof(float) * (size_t)parts * d.H;
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
  BackArgs a = {dy, s, weight, ds, dy_stride, s_stride, ds_stride, stats, dx,
                static_cast<float *>(ws), d.n, d.H, d.n < kNormParts ? d.n : kNormParts,
                d.weight_dtype == MOE_F32, d.rms != 0, dbias != nullptr, 0, false};
  return d.dtype == MOE_F32 ? backward<float>(a, dweight, dbias, st)
                            : backward<__nv_bfloat16>(a, dweight, dbias, st);
}

}  // namespace moe
