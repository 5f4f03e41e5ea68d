// Appending keys and values to a paged cache, with the position rotation of
// queries and keys on the way:
//   q_out[t] = rot(q[t]), K[page][h][slot] = rot(k[t]), V[page][h][slot] = v[t]
// with rot(x)_i = x_i cos - x_j sin, rot(x)_j = x_j cos + x_i sin over the
// rotated pairs (i, j), page and slot from the token's sequence and position.
//
// Bound: HBM for a prefill chunk (every value is read once and written once),
// latency for a decode batch (ids -> page -> store is a chain of dependent
// loads).  A CTA owns one token, so the chain is walked once per CTA and the
// token's cosines and sines are read once per thread and used for every head:
// thread (row lane, j) moves the j-th 16 values of the head rows row lane,
// row lane + lanes, ...  16 values are two vectors of 8 that rotate with each
// other (i and i + rope_dim/2, or 16 neighbours when pairs are interleaved),
// so no value is loaded twice and q may be rotated in place.
//
// Measured: 8191 tokens of 16 + 2 * 16 heads of 128, bf16 (206 MB): 37.5 us,
// 5.5 TB/s, as long as a plain device copy of the same bytes takes; with the
// rows asked for after the page is known 40 us.  The same into an e4m3 cache
// (172 MB) 45.7 us, 3.8 TB/s; all in float32 (407 MB) 72.6 us, 5.6 TB/s.  61
// tokens of 32 + 2 * 8 heads into an e4m3 cache: 3 us.
#include <cuda_fp8.h>

#include "kv_cache.cuh"

namespace moe {
namespace {

constexpr int AT = 128;  // threads per CTA
constexpr int AU = 4;    // head rows in flight per thread

struct AppendArgs {
  const void *q, *k, *v;
  long long qs, ks, vs;  // elements between tokens
  const int32_t *seq_ids, *positions, *table;
  const float *rope, *kscale, *vscale;
  void *qout, *kc, *vc;
  long long page_stride;
  int num_seqs, Hq, Hkv, P, num_pages, max_pages, rope_rows, R, interleaved;
  int rows_per_cta;  // head rows (q, k and v) of one CTA
  int32_t *status;
};

struct Vec8 {
  float f[8];
};

// 8 values as they lie in memory; widened when they are used
template <typename T>
struct Raw8;
template <>
struct Raw8<__nv_bfloat16> {
  uint4 u;
  __device__ __forceinline__ void load(const __nv_bfloat16 *p) {
    u = __ldcs(reinterpret_cast<const uint4 *>(p));
  }
  __device__ __forceinline__ Vec8 widen() const {
    const __nv_bfloat162 *h = reinterpret_cast<const __nv_bfloat162 *>(&u);
    Vec8 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 x = __bfloat1622float2(h[i]);
      v.f[2 * i] = x.x;
      v.f[2 * i + 1] = x.y;
    }
    return v;
  }
};
template <>
struct Raw8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float *p) {
    a = __ldcs(reinterpret_cast<const float4 *>(p));
    b = __ldcs(reinterpret_cast<const float4 *>(p) + 1);
  }
  __device__ __forceinline__ Vec8 widen() const {
    return Vec8{{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
  }
};

// Stored values are rounded once from float32; scale is used by e4m3 only.
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const Vec8 &v, float) {
  uint4 u;
  __nv_bfloat162 *h = reinterpret_cast<__nv_bfloat162 *>(&u);
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(v.f[2 * i], v.f[2 * i + 1]);
  *reinterpret_cast<uint4 *>(p) = u;
}

__device__ __forceinline__ void store8(float *p, const Vec8 &v, float) {
  *reinterpret_cast<float4 *>(p) = *reinterpret_cast<const float4 *>(v.f);
  *reinterpret_cast<float4 *>(p + 4) = *reinterpret_cast<const float4 *>(v.f + 4);
}

__device__ __forceinline__ void store8(__nv_fp8_e4m3 *p, const Vec8 &v, float scale) {
  uint2 u;
  __nv_fp8x2_storage_t *h = reinterpret_cast<__nv_fp8x2_storage_t *>(&u);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    h[i] = __nv_cvt_float2_to_fp8x2(
        make_float2(__fdiv_rn(v.f[2 * i], scale), __fdiv_rn(v.f[2 * i + 1], scale)),
        __NV_SATFINITE, __NV_E4M3);
  *reinterpret_cast<uint2 *>(p) = u;
}

// One pair: products and sums are rounded one by one, so a value does not
// depend on how the compiler contracts them.
__device__ __forceinline__ void rotate(float &a, float &b, float c, float s) {
  const float x = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
  b = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
  a = x;
}

template <int D, typename T, typename C>
__global__ void __launch_bounds__(AT) kv_append_kernel(const AppendArgs a) {
  pdl_enter();
  constexpr int JT = D / 16, RL = AT / JT;
  const int t = blockIdx.x;
  const int j = threadIdx.x % JT, rl = threadIdx.x / JT;
  const int seq = __ldg(a.seq_ids + t), pos = __ldg(a.positions + t);
  // this thread's 16 dimensions of every head row, as two vectors of 8
  const int half = a.R >> 1;
  const bool rot = 16 * j < a.R;
  const bool split = rot && !a.interleaved;
  const int d0 = split ? 8 * j : 16 * j;
  const int d1 = split ? half + 8 * j : d0 + 8;
  const int r0 = blockIdx.y * a.rows_per_cta;
  const int r1 = min(r0 + a.rows_per_cta, a.Hq + 2 * a.Hkv);
  const int rk = a.Hq, rv = a.Hq + a.Hkv;  // first key row, first value row
  Raw8<T> lo[AU], hi[AU];
  auto fetch = [&](int rb) {
#pragma unroll
    for (int u = 0; u < AU; ++u) {
      const int r = rb + u * RL;
      if (r >= r1 || (r < rk && !a.q)) continue;
      const T *src = r < rk   ? (const T *)a.q + t * a.qs + r * D
                     : r < rv ? (const T *)a.k + t * a.ks + (r - rk) * D
                              : (const T *)a.v + t * a.vs + (r - rv) * D;
      lo[u].load(src + (r >= rv ? 16 * j : d0));  // values are not rotated: neighbours
      hi[u].load(src + (r >= rv ? 16 * j + 8 : d1));
    }
  };
  // the rows do not depend on where the token goes: they are on their way
  // while its sequence, position and page are looked up
  fetch(r0 + rl);
  if (seq < 0) return;  // padding
  const int col = pos / a.P;
  bool ok = seq < a.num_seqs && pos >= 0 && col < a.max_pages && (a.R == 0 || pos < a.rope_rows);
  int page = -1;
  Vec8 cs = {}, sn = {};
  if (ok) {
    page = __ldg(a.table + (size_t)seq * a.max_pages + col);
    if (rot) {
      const float4 *row = reinterpret_cast<const float4 *>(a.rope + (size_t)pos * a.R + 8 * j);
      *reinterpret_cast<float4 *>(cs.f) = __ldg(row);
      *reinterpret_cast<float4 *>(cs.f + 4) = __ldg(row + 1);
      *reinterpret_cast<float4 *>(sn.f) = __ldg(row + half / 4);
      *reinterpret_cast<float4 *>(sn.f + 4) = __ldg(row + half / 4 + 1);
    }
  }
  ok = ok && page >= 0 && page < a.num_pages;
  if (!ok) {
    if (threadIdx.x == 0 && blockIdx.y == 0) flag_status(a.status, MOE_DEV_BAD_CACHE);
    return;
  }
  const size_t slot = (size_t)page * a.page_stride + (size_t)(pos - col * a.P) * D;
  const int head_step = a.P * D;
  for (int rb = r0 + rl; rb < r1;) {
#pragma unroll
    for (int u = 0; u < AU; ++u) {
      const int r = rb + u * RL;
      if (r >= r1 || (r < rk && !a.q)) continue;
      Vec8 x = lo[u].widen(), y = hi[u].widen();
      if (r >= rv) {
        const int h = r - rv;
        const float sc = a.vscale ? __ldg(a.vscale + h) : 1.f;
        C *dst = (C *)a.vc + slot + (size_t)h * head_step + 16 * j;
        store8(dst, x, sc);
        store8(dst + 8, y, sc);
        continue;
      }
      if (split) {
#pragma unroll
        for (int i = 0; i < 8; ++i) rotate(x.f[i], y.f[i], cs.f[i], sn.f[i]);
      } else if (rot) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          rotate(x.f[2 * i], x.f[2 * i + 1], cs.f[i], sn.f[i]);
          rotate(y.f[2 * i], y.f[2 * i + 1], cs.f[4 + i], sn.f[4 + i]);
        }
      }
      if (r < rk) {
        T *dst = (T *)a.qout + ((size_t)t * a.Hq + r) * D;
        store8(dst + d0, x, 1.f);
        store8(dst + d1, y, 1.f);
      } else {
        const int h = r - rk;
        const float sc = a.kscale ? __ldg(a.kscale + h) : 1.f;
        C *dst = (C *)a.kc + slot + (size_t)h * head_step;
        store8(dst + d0, x, sc);
        store8(dst + d1, y, sc);
      }
    }
    rb += AU * RL;
    if (rb < r1) fetch(rb);
  }
}

template <int D, typename T, typename C>
cudaError_t append_d(AppendArgs &a, int n, cudaStream_t s) {
  constexpr int RL = AT / (D / 16);
  const int rows = a.Hq + 2 * a.Hkv;
  // few tokens: their head rows are spread over CTAs, one row per thread, so
  // that a token is not the work of one SM; many: one CTA per token, which looks
  // its place up once (48 rows of 128 a token: 61 tokens 2.34 us spread, 2.66
  // not; 200 2.91 and 3.07; 300 4.06 and 3.10; other layouts not measured)
  const int parts = (rows + RL - 1) / RL;
  const bool spread = (long long)n * parts <= 4ll * device_sm_count();
  a.rows_per_cta = spread ? RL : rows;
  return launch_pdl(kv_append_kernel<D, T, C>, dim3(n, spread ? parts : 1), dim3(AT), 0, s, a);
}

template <typename T, typename C>
cudaError_t append_t(AppendArgs &a, int D, int n, cudaStream_t s) {
  if (D == 64) return append_d<64, T, C>(a, n, s);
  if (D == 128) return append_d<128, T, C>(a, n, s);
  return append_d<256, T, C>(a, n, s);
}

}  // namespace

cudaError_t launch_kv_append(const KVCache &c, int n, const void *q, long long q_stride,
                             const void *k, long long k_stride, const void *v, long long v_stride,
                             const int32_t *seq_ids, const int32_t *positions, void *q_out,
                             int32_t *status, cudaStream_t s) {
  if (n == 0) return cudaSuccess;
  AppendArgs a = {};
  a.q = q, a.k = k, a.v = v;
  a.qs = q_stride, a.ks = k_stride, a.vs = v_stride;
  a.seq_ids = seq_ids, a.positions = positions, a.table = c.page_table;
  a.rope = c.rope, a.kscale = c.k_scale, a.vscale = c.v_scale;
  a.qout = q_out, a.kc = c.k_cache, a.vc = c.v_cache;
  a.page_stride = c.page_stride;
  a.num_seqs = c.num_seqs, a.Hq = c.q_heads, a.Hkv = c.kv_heads, a.P = c.page_size;
  a.num_pages = c.num_pages, a.max_pages = c.max_pages;
  a.rope_rows = c.rope_rows, a.R = c.rope ? c.rope_dim : 0, a.interleaved = c.rope_interleaved;
  a.status = status;
  if (c.dtype == MOE_F32) return append_t<float, float>(a, c.head_dim, n, s);
  if (c.cache_dtype == MOE_E4M3)
    return append_t<__nv_bfloat16, __nv_fp8_e4m3>(a, c.head_dim, n, s);
  return append_t<__nv_bfloat16, __nv_bfloat16>(a, c.head_dim, n, s);
}

}  // namespace moe
