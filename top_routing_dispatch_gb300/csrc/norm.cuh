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

template <typename T, bool VEC, int GS, int VALS>
struct RowIO {
  static constexpr int V = VEC ? kPer<T> : 1;
  static constexpr bool SHARED = !VEC && sizeof(T) == 2;  // slots are read by other threads
  static constexpr int BYTES = GS * VALS * (int)sizeof(T);
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
  // values behind the row's end are 0
  static __device__ __forceinline__ void read(const char *slot, const T *row, int H, int t,
                                              float (&f)[VALS]) {
    const T *p = reinterpret_cast<const T *>(slot) + odd(row);
    if (VEC) {
#pragma unroll
      for (int k = 0; k < VALS; k += V) {
        uint4 u = make_uint4(0, 0, 0, 0);
        if (at(k, t) < H) u = *reinterpret_cast<const uint4 *>(p + at(k, t));
        const T *e = reinterpret_cast<const T *>(&u);
#pragma unroll
        for (int j = 0; j < V; ++j) f[k + j] = to_f(e[j]);
      }
    } else {
#pragma unroll
      for (int k = 0; k < VALS; ++k) f[k] = at(k, t) < H ? to_f(p[at(k, t)]) : 0.f;
    }
  }
  static __device__ __forceinline__ void store(T *row, int H, int t, const float (&f)[VALS]) {
    if (VEC) {
#pragma unroll
      for (int k = 0; k < VALS; k += V) {
        uint4 u;
        T *e = reinterpret_cast<T *>(&u);
#pragma unroll
        for (int j = 0; j < V; ++j) e[j] = from_f<T>(f[k + j]);
        if (at(k, t) < H) *reinterpret_cast<uint4 *>(row + at(k, t)) = u;
      }
    } else {
#pragma unroll
      for (int k = 0; k < VALS; ++k)
        if (at(k, t) < H) row[at(k, t)] = from_f<T>(f[k]);
    }
  }
  // weight or bias at the same columns, from global memory
  static __device__ __forceinline__ void param(const void *w, bool wide, int H, int t,
                                               float (&f)[VALS]) {
    if (VEC) {
#pragma unroll
      for (int k = 0; k < VALS; k += V) {
        const int i = at(k, t);
        if (i >= H) {
#pragma unroll
          for (int j = 0; j < V; ++j) f[k + j] = 0.f;
        } else if (wide) {
#pragma unroll
          for (int j = 0; j < V; j += 4)
            *reinterpret_cast<float4 *>(&f[k + j]) =
                __ldg(reinterpret_cast<const float4 *>(static_cast<const float *>(w) + i + j));
        } else {
          const uint4 u = __ldg(reinterpret_cast<const uint4 *>(static_cast<const T *>(w) + i));
          const T *e = reinterpret_cast<const T *>(&u);
#pragma unroll
          for (int j = 0; j < V; ++j) f[k + j] = to_f(e[j]);
        }
      }
    } else {
#pragma unroll
      for (int k = 0; k < VALS; ++k) {
        const int i = at(k, t);
        f[k] = i >= H ? 0.f
               : wide ? __ldg(static_cast<const float *>(w) + i)
                      : to_f(static_cast<const T *>(w)[i]);
      }
    }
  }
};

// Barrier of the group's threads
template <int GS>
__device__ __forceinline__ void group_sync(int group) {
  if (GS <= 32)
    __syncwarp();
  else
    asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "n"(GS) : "memory");
}

// Sums of two values over the group, the same in every thread of it.  `part`:
// a place per warp of the group, which the next sum must not use.
template <int GS>
__device__ __forceinline__ float2 group_sum(float2 v, float2 *part, int group) {
#pragma unroll
  for (int o = (GS < 32 ? GS : 32) / 2; o > 0; o /= 2) {
    v.x += __shfl_xor_sync(~0u, v.x, o);
    v.y += __shfl_xor_sync(~0u, v.y, o);
  }
  if (GS <= 32) return v;
  constexpr int W = GS > 32 ? GS / 32 : 2;
  if (threadIdx.x % 32 == 0) part[threadIdx.x / 32 % W] = v;
  group_sync<GS>(group);
  if (W <= 8) {
    const float4 *p = reinterpret_cast<const float4 *>(part);
    float4 a = p[0];
#pragma unroll
    for (int i = 1; i < W / 2; ++i) {
      const float4 b = p[i];
      a.x += b.x, a.y += b.y, a.z += b.z, a.w += b.w;
    }
    return make_float2(a.x + a.z, a.y + a.w);
  }
  v = part[threadIdx.x % W];
#pragma unroll
  for (int o = W / 2; o > 0; o /= 2) {
    v.x += __shfl_xor_sync(~0u, v.x, o);
    v.y += __shfl_xor_sync(~0u, v.y, o);
  }
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
