// What the norm's forward and backward kernels share.
//
// A row belongs to a group of GS threads (part of a warp, a warp, or several),
// VALS values to a thread.  A persistent CTA holds several groups; each copies
// its next rows asynchronously into a ring of D slots of its own in shared
// memory, so the loads of D - 1 rows are on their way while one row's sums go
// through the group.  Three ways into the ring:
//   VEC            16 bytes a copy; a thread copies what it will read itself,
//                  so no barrier is needed.
//   words, float   4 bytes a copy, likewise.
//   words, bf16    rows that do not start on 16 bytes, perhaps not even on 4:
//                  the 4-byte words that cover the row, one barrier a row, and
//                  values read at the row's offset in its first word.
#pragma once

#include "ptx.cuh"
#include "train.cuh"

namespace moe {

constexpr int kNormThreads = 512;  // of a CTA of groups, at most
constexpr int kNormParts = 304;    // CTAs of the backward, at most

template <typename T>
constexpr int kPer = 16 / (int)sizeof(T);  // values of 16 bytes

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

__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}

// Two float32 operations in one instruction, each rounded as its single form
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<unsigned long long &>(d))
      : "l"(reinterpret_cast<unsigned long long &>(a)), "l"(reinterpret_cast<unsigned long long &>(b)));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<unsigned long long &>(d))
      : "l"(reinterpret_cast<unsigned long long &>(a)), "l"(reinterpret_cast<unsigned long long &>(b)));
  return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(reinterpret_cast<unsigned long long &>(d))
      : "l"(reinterpret_cast<unsigned long long &>(a)), "l"(reinterpret_cast<unsigned long long &>(b)),
        "l"(reinterpret_cast<unsigned long long &>(c)));
  return d;
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// A thread's VALS values of a row, in pairs.
template <typename T, bool VEC, int GS, int VALS>
struct RowIO {
  static constexpr int V = VEC ? kPer<T> : 1;
  static constexpr bool SHARED = !VEC && sizeof(T) == 2;  // slots are read by other threads
  static constexpr int BYTES = GS * VALS * (int)sizeof(T);
  static constexpr int P = VALS / 2;       // pairs
  static constexpr int RUN = VEC ? V / 2 : 1;  // pairs that lie inside the row or outside together
  // column of the k-th value of the group's thread t
  static __device__ __forceinline__ int at(int k, int t) {
    return VEC ? (k / V * GS + t) * V + k % V : k * GS + t;
  }
  static __device__ __forceinline__ int odd(const T *row) {
    return SHARED ? (int)(reinterpret_cast<uintptr_t>(row) >> 1) & 1 : 0;
  }
  static __device__ __forceinline__ void issue(uint32_t slot, const T *row, int H, int t) {
    if (SHARED) {
      const int o = odd(row), end = H + o;
#pragma unroll
      for (int k = 0; k < VALS / 2; ++k) {
        const int j = k * GS + t;  // word; the last may hold one value of the row
        if (2 * j < end) cp_async4(slot + 4 * j, row - o + 2 * j, 2 * j + 2 <= end ? 4 : 2);
      }
    } else if (VEC) {
#pragma unroll
      for (int k = 0; k < VALS; k += V)
        if (at(k, t) < H) ptx::cp_async_cg16(slot + at(k, t) * (int)sizeof(T), row + at(k, t));
    } else {
#pragma unroll
      for (int k = 0; k < VALS; ++k)
        if (at(k, t) < H) cp_async4(slot + 4 * at(k, t), row + at(k, t), 4);
    }
  }
  static __device__ __forceinline__ float2 pair(uint32_t u) {  // of bf16
    return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
  }
  // 16 bytes as pairs, from pair i of f on
  static __device__ __forceinline__ void widen(uint4 u, float2 *f) {
    if (sizeof(T) == 2) {
      f[0] = pair(u.x), f[1] = pair(u.y), f[2] = pair(u.z), f[3] = pair(u.w);
    } else {
      f[0] = make_float2(__uint_as_float(u.x), __uint_as_float(u.y));
      f[1] = make_float2(__uint_as_float(u.z), __uint_as_float(u.w));
    }
  }
  // values behind the row's end are 0
  static __device__ __forceinline__ void read(const char *slot, int o, int H, int t,
                                              float2 (&f)[P]) {
    const T *p = reinterpret_cast<const T *>(slot) + (SHARED ? o : 0);
    if (VEC) {
#pragma unroll
      for (int k = 0; k < VALS; k += V) {
        uint4 u = make_uint4(0, 0, 0, 0);
        if (at(k, t) < H) u = *reinterpret_cast<const uint4 *>(p + at(k, t));
        widen(u, f + k / 2);
      }
    } else {
#pragma unroll
      for (int k = 0; k < P; ++k) {
        f[k].x = at(2 * k, t) < H ? to_f(p[at(2 * k, t)]) : 0.f;
        f[k].y = at(2 * k + 1, t) < H ? to_f(p[at(2 * k + 1, t)]) : 0.f;
      }
    }
  }
  static __device__ __forceinline__ uint4 narrow(const float2 *f) {
    uint4 u;
    if (sizeof(T) == 2) {
      __nv_bfloat162 *h = reinterpret_cast<__nv_bfloat162 *>(&u);
#pragma unroll
      for (int i = 0; i < 4; ++i) h[i] = __float22bfloat162_rn(f[i]);
    } else {
      u = make_uint4(__float_as_uint(f[0].x), __float_as_uint(f[0].y), __float_as_uint(f[1].x),
                     __float_as_uint(f[1].y));
    }
    return u;
  }
  // the values rounded to T
  static __device__ __forceinline__ void round(float2 (&f)[P]) {
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int k = 0; k < P; ++k) {
        const __nv_bfloat162 h = __float22bfloat162_rn(f[k]);
        f[k] = pair(reinterpret_cast<const uint32_t &>(h));
      }
    }
  }
  static __device__ __forceinline__ void store(T *row, int H, int t, const float2 (&f)[P]) {
    if (VEC) {
#pragma unroll
      for (int k = 0; k < VALS; k += V)
        if (at(k, t) < H) *reinterpret_cast<uint4 *>(row + at(k, t)) = narrow(f + k / 2);
    } else {
#pragma unroll
      for (int k = 0; k < P; ++k) {
        if (at(2 * k, t) < H) row[at(2 * k, t)] = from_f<T>(f[k].x);
        if (at(2 * k + 1, t) < H) row[at(2 * k + 1, t)] = from_f<T>(f[k].y);
      }
    }
  }
  // weight or bias at the same columns, from global memory
  static __device__ __forceinline__ void param(const void *w, bool wide, int H, int t,
                                               float2 (&f)[P]) {
    if (VEC) {
#pragma unroll
      for (int k = 0; k < VALS; k += V) {
        const int i = at(k, t);
        if (i >= H) {
#pragma unroll
          for (int j = 0; j < V / 2; ++j) f[k / 2 + j] = make_float2(0.f, 0.f);
        } else if (wide) {
#pragma unroll
          for (int j = 0; j < V; j += 4)
            *reinterpret_cast<float4 *>(&f[(k + j) / 2]) =
                __ldg(reinterpret_cast<const float4 *>(static_cast<const float *>(w) + i + j));
        } else {
          widen(__ldg(reinterpret_cast<const uint4 *>(static_cast<const T *>(w) + i)), f + k / 2);
        }
      }
    } else {
#pragma unroll
      for (int k = 0; k < VALS; ++k) {
        const int i = at(k, t);
        (k % 2 ? f[k / 2].y : f[k / 2].x) = i >= H ? 0.f
                                            : wide ? __ldg(static_cast<const float *>(w) + i)
                                                   : to_f(static_cast<const T *>(w)[i]);
      }
    }
  }
  // f(k) for every pair k with values inside the row; of the strided forms
  // the second value of a pair may lie behind the row's end
  template <typename F>
  static __device__ __forceinline__ void each(int H, int t, F f) {
#pragma unroll
    for (int k = 0; k < P; k += RUN) {
      if (at(2 * k, t) < H) {
#pragma unroll
        for (int j = 0; j < RUN; ++j) f(k + j);
      }
    }
  }
  // whether both values of pair k lie inside the row
  static __device__ __forceinline__ bool whole(int k, int H, int t) {
    return VEC || at(2 * k + 1, t) < H;
  }
};

// 1 / sqrt(v), within 2 u: one Newton step from the approximation
__device__ __forceinline__ float rsqrt_of(float v) {
  const float r = rsqrtf(v);
  const float e = fmaf(-v * r, r, 1.f);
  return v > 0.f && v < INFINITY ? fmaf(0.5f * r, e, r) : r;
}

// Barrier of the group's threads
template <int GS>
__device__ __forceinline__ void group_sync(int group) {
  if (GS <= 32)
    __syncwarp();
  else
    asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "n"(GS) : "memory");
}

__device__ __forceinline__ float plus(float a, float b) { return a + b; }
__device__ __forceinline__ float2 plus(float2 a, float2 b) { return add2(a, b); }
__device__ __forceinline__ float from_lane(float v, int o) { return __shfl_xor_sync(~0u, v, o); }
__device__ __forceinline__ float2 from_lane(float2 v, int o) {
  return make_float2(__shfl_xor_sync(~0u, v.x, o), __shfl_xor_sync(~0u, v.y, o));
}

// Sum of a value (or of two) over the group, the same in every thread of it.
// `places`: one per warp of the group, which the next sum must not use.
template <int GS, typename F>
__device__ __forceinline__ F group_sum(F v, float2 *places, int group) {
#pragma unroll
  for (int o = (GS < 32 ? GS : 32) / 2; o > 0; o /= 2) v = plus(v, from_lane(v, o));
  if (GS <= 32) return v;
  constexpr int W = GS > 32 ? GS / 32 : 2;
  F *part = reinterpret_cast<F *>(places);
  if (threadIdx.x % 32 == 0) part[threadIdx.x / 32 % W] = v;
  group_sync<GS>(group);
  if (W <= 4) {
    v = part[0];
#pragma unroll
    for (int i = 1; i < W; ++i) v = plus(v, part[i]);
    return v;
  }
  v = part[threadIdx.x % W];
#pragma unroll
  for (int o = W / 2; o > 0; o /= 2) v = plus(v, from_lane(v, o));
  return v;
}

// Slots of the ring for N tensors: as many of 8, 4 or 2 as fit in 200 KB
// beside the other groups' (0: none of them, rows too long).
template <typename T, int VALS, int N>
constexpr int ring_slots() {
  constexpr int one = kNormThreads * VALS * (int)sizeof(T) * N;
  return one * 8 <= 200 * 1024 ? 8 : one * 4 <= 200 * 1024 ? 4 : one * 2 <= 200 * 1024 ? 2 : 0;
}

// The group for rows of H values: the smallest of which a thread takes 16, or
// 512 threads of 32 values; G<...>::go, or false where rows are longer.
template <typename T, bool VEC, template <typename, bool, int, int> class G, typename A>
bool by_length(const A &a, cudaStream_t s, cudaError_t *e) {
  const int H = a.H + (!VEC && sizeof(T) == 2);  // a word may begin one value early
  if (H <= 8 * 16) return G<T, VEC, 8, 16>::go(a, s, e);
  if (H <= 32 * 16) return G<T, VEC, 32, 16>::go(a, s, e);
  if (H <= 64 * 16) return G<T, VEC, 64, 16>::go(a, s, e);
  if (H <= 128 * 16) return G<T, VEC, 128, 16>::go(a, s, e);
  if (H <= 256 * 16) return G<T, VEC, 256, 16>::go(a, s, e);
  if (H <= 512 * 16) return G<T, VEC, 512, 16>::go(a, s, e);
  if (H <= 512 * 32) return G<T, VEC, 512, 32>::go(a, s, e);
  return false;
}

// CTAs and groups of a launch over n rows: the rows of a round lie beside each
// other over the CTAs, so that few rows use many SMs.
struct NormGrid {
  int ctas, groups;
};
template <int GS>
inline NormGrid norm_grid(int n, int most) {
  NormGrid g;
  g.ctas = n < most ? n : most;
  const int rows = (int)(((long long)n + g.ctas - 1) / g.ctas), all = kNormThreads / GS;
  constexpr int warp = GS < 32 ? 32 / GS : 1;  // whole warps
  g.groups = rows < all ? (rows + warp - 1) / warp * warp : all;
  return g;
}

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

inline bool on_bytes(const void *p, uintptr_t b) {
  return (reinterpret_cast<uintptr_t>(p) & (b - 1)) == 0;
}

}  // namespace moe
