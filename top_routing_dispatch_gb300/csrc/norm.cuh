// What the norm's forward and backward kernels share.
//
// A row belongs to a group of GS threads (part of a warp, a warp, or several),
// VALS values to a thread.  A persistent CTA holds several groups; each copies
// its next rows asynchronously into a ring of D slots of its own in shared
// memory, so the loads of D - 1 rows are on their way while one row's sums go
// through the group.  A thread copies the 16-byte pieces that it will read
// itself, so the ring needs no barrier.
//
// Rows of odd length do not begin on 16 bytes.  A group's rows are a multiple
// of 8 apart, so they all begin at the same place within 16 bytes (the phase):
// the group works on the aligned pieces that cover a row, its columns shifted
// by the phase, and masks the row's ends.
//
// In the backward, rows too long for one CTA belong to a cluster of up to 8, a
// CTA being the group of its part of the row; the sums go through the cluster's
// shared memory.
#pragma once

#include "pairs.cuh"
#include "ptx.cuh"
#include "roots.cuh"
#include "train.cuh"

namespace moe {

// Threads of a CTA, at most: whole groups of about 512 threads, with 128 registers
// each (two groups of 320: the forward is content with 96; float32 with residual
// spills 28 bytes)
template <int GS>
constexpr int kCta = GS > 512 ? GS : GS == 320 ? 640 : 512 / GS * GS;
constexpr int kNormParts = 304;    // CTAs (or clusters) of the backward, at most
constexpr int kMostCluster = 8;    // CTAs of a cluster, at most

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

// 16 bytes, of which `bytes` are read and the rest are zeros
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}

// A thread's VALS values of a row, in pairs: pieces of V values, GS apart.
// SHIFT: rows have phases; else every piece lies inside the row or outside.
// CLUSTER: the group has `part` columns of a row, from `base` on.
template <typename T, int GS, int VALS, bool SHIFT, bool CLUSTER>
struct RowIO {
  static constexpr int V = kPer<T>, PIECES = VALS / V, P = VALS / 2;
  static constexpr int BYTES = GS * VALS * (int)sizeof(T);
  int H, t, o;       // row length, thread of the group, phase
  int base;          // of the group's part of a row, without the phase
  bool full[PIECES]; // all of the piece lies inside the row
  bool live[PIECES]; // some of it does, and it belongs to the group's part

  __device__ __forceinline__ RowIO(int H_, int t_, int o_, int base_, int part)
      : H(H_), t(t_), o(SHIFT ? o_ : 0), base(CLUSTER ? base_ : 0) {
#pragma unroll
    for (int c = 0; c < PIECES; ++c) {
      live[c] = first(c) < H;  // begins less than a piece before the row
      full[c] = SHIFT ? first(c) >= 0 && first(c) + V <= H : live[c];
      if (CLUSTER && (c * GS + t) * V >= part) live[c] = full[c] = false;
    }
  }
  // column of a piece's first value
  __device__ __forceinline__ int first(int c) const {
    return base + (c * GS + t) * V - (SHIFT ? o : 0);
  }
  // column of value k, and whether the row has it
  __device__ __forceinline__ int at(int k) const { return first(k / V) + k % V; }
  __device__ __forceinline__ bool has(int k) const { return (unsigned)at(k) < (unsigned)H; }

  // Asks for a row with `behind` rows behind it in the tensor.  A piece may begin
  // before the row, inside the rows before it (the first row has phase 0), and
  // may end behind it, but not behind the tensor.
  __device__ __forceinline__ void issue(uint32_t slot, const T *row, long long stride,
                                        long long behind) const {
    const int room = behind >= V || behind * stride >= V ? V : (int)(behind * stride);
#pragma unroll
    for (int c = 0; c < PIECES; ++c) {
      if (!live[c]) continue;
      const uint32_t to = slot + (c * GS + t) * 16;
      const int left = H + room - first(c);
      if (!SHIFT || left >= V)
        ptx::cp_async_cg16(to, row + first(c));
      else
        cp_async16(to, row + first(c), left * (int)sizeof(T));
    }
  }
  static __device__ __forceinline__ float2 pair(uint32_t u) {  // of bf16
    return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
  }
  // 16 bytes as pairs
  static __device__ __forceinline__ void widen(uint4 u, float2 *f) {
    if constexpr (sizeof(T) == 2) {
      f[0] = pair(u.x), f[1] = pair(u.y), f[2] = pair(u.z), f[3] = pair(u.w);
    } else {
      f[0] = make_float2(__uint_as_float(u.x), __uint_as_float(u.y));
      f[1] = make_float2(__uint_as_float(u.z), __uint_as_float(u.w));
    }
  }
  static __device__ __forceinline__ uint4 narrow(const float2 *f) {
    uint4 u;
    if constexpr (sizeof(T) == 2) {
      __nv_bfloat162 *h = reinterpret_cast<__nv_bfloat162 *>(&u);
#pragma unroll
      for (int i = 0; i < 4; ++i) h[i] = __float22bfloat162_rn(f[i]);
    } else {
      u = make_uint4(__float_as_uint(f[0].x), __float_as_uint(f[0].y), __float_as_uint(f[1].x),
                     __float_as_uint(f[1].y));
    }
    return u;
  }
  // zeros for the values of piece c that the row does not have
  __device__ __forceinline__ void mask(int c, float2 (&f)[P]) const {
    if constexpr (SHIFT) {
      if (full[c]) return;
#pragma unroll
      for (int k = c * V; k < (c + 1) * V; ++k)
        if (!has(k)) (k % 2 ? f[k / 2].y : f[k / 2].x) = 0.f;
    }
  }
  // CLEAN: with zeros for what the row does not have, else other rows' values
  template <bool CLEAN>
  __device__ __forceinline__ void read(const char *slot, float2 (&f)[P]) const {
#pragma unroll
    for (int c = 0; c < PIECES; ++c) {
      uint4 u = make_uint4(0, 0, 0, 0);
      if (live[c]) u = *reinterpret_cast<const uint4 *>(slot + (c * GS + t) * 16);
      widen(u, f + c * V / 2);
      if (CLEAN && live[c]) mask(c, f);
    }
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
  __device__ __forceinline__ void store(T *row, const float2 (&f)[P]) const {
#pragma unroll
    for (int c = 0; c < PIECES; ++c) {
      if (full[c]) {
        *reinterpret_cast<uint4 *>(row + first(c)) = narrow(f + c * V / 2);
      } else if (SHIFT && live[c]) {
#pragma unroll
        for (int k = c * V; k < (c + 1) * V; ++k)
          if (has(k)) row[at(k)] = from_f<T>(k % 2 ? f[k / 2].y : f[k / 2].x);
      }
    }
  }
  // weight or bias at the same columns, from global memory; wide: float32
  __device__ __forceinline__ void param(const void *w, bool wide, bool aligned,
                                        float2 (&f)[P]) const {
#pragma unroll
    for (int c = 0; c < PIECES; ++c) {
      if (aligned && (!SHIFT || o == 0) && full[c]) {
        if (wide) {
#pragma unroll
          for (int j = 0; j < V; j += 4)
            *reinterpret_cast<float4 *>(&f[(c * V + j) / 2]) = __ldg(
                reinterpret_cast<const float4 *>(static_cast<const float *>(w) + first(c) + j));
        } else {
          widen(__ldg(reinterpret_cast<const uint4 *>(static_cast<const T *>(w) + first(c))),
                f + c * V / 2);
        }
        continue;
      }
#pragma unroll
      for (int k = c * V; k < (c + 1) * V; ++k)
        (k % 2 ? f[k / 2].y : f[k / 2].x) =
            !has(k) ? 0.f
            : wide  ? __ldg(static_cast<const float *>(w) + at(k))
                    : to_f(static_cast<const T *>(w)[at(k)]);
    }
  }
  // column sums in float32 at the same columns; aligned: out + first(c) on 16 bytes
  __device__ __forceinline__ void put(float *out, bool aligned, const float2 (&f)[P]) const {
#pragma unroll
    for (int c = 0; c < PIECES; ++c) {
      if ((!SHIFT || o == 0) && aligned && full[c]) {
#pragma unroll
        for (int j = 0; j < V; j += 4)
          *reinterpret_cast<float4 *>(out + first(c) + j) =
              *reinterpret_cast<const float4 *>(&f[(c * V + j) / 2]);
      } else if (live[c]) {
#pragma unroll
        for (int k = c * V; k < (c + 1) * V; ++k)
          if (has(k)) out[at(k)] = k % 2 ? f[k / 2].y : f[k / 2].x;
      }
    }
  }
  // f(c, k) for the pairs k of every piece c that the row has some of
  template <typename F>
  __device__ __forceinline__ void each(F f) const {
#pragma unroll
    for (int c = 0; c < PIECES; ++c) {
      if (live[c]) {
#pragma unroll
        for (int k = c * V / 2; k < (c + 1) * V / 2; ++k) f(c, k);
      }
    }
  }
};

// Whether rows of the given strides keep one phase: 16-byte aligned, and
// strides equal modulo the values of 16 bytes.
struct Phases {
  int per, step;
  bool one = true, first = true;
  explicit Phases(int per_) : per(per_), step(0) {}
  void add(const void *p, long long stride) {
    if (!p) return;
    if (first) step = (int)(stride % per), first = false;
    one = one && (reinterpret_cast<uintptr_t>(p) & 15) == 0 && stride % per == step;
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
  if (W <= 5) {
    v = part[0];
#pragma unroll
    for (int i = 1; i < W; ++i) v = plus(v, part[i]);
    return v;
  }
  if constexpr ((W & (W - 1)) == 0) {
    v = part[threadIdx.x % W];
#pragma unroll
    for (int o = W / 2; o > 0; o /= 2) v = plus(v, from_lane(v, o));
  } else {
    v = threadIdx.x % 32 < W ? part[threadIdx.x % 32] : F{};
#pragma unroll
    for (int o = 16; o > 0; o /= 2) v = plus(v, from_lane(v, o));
  }
  return v;
}

// A CTA's place among those that share its rows: the part of a row that it
// takes, and which rows.
template <int GS, int VALS, int V, bool CLUSTER>
struct Share {
  int size = 1, rank = 0, base = 0, part = GS * VALS;
  int index = blockIdx.x, count = gridDim.x;  // of the CTA, or of the cluster
  // span: columns of a row with its phases
  __device__ __forceinline__ explicit Share(int span) {
    if constexpr (CLUSTER) {
      asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(size));
      rank = (int)ptx::cluster_ctarank();
      part = ((span + V - 1) / V + size - 1) / size * V;  // equal parts, of whole pieces
      base = rank * part;
      index /= size, count /= size;
    }
  }
};

// Sum of a value (or of two) over the cluster, the same in every thread of it:
// each warp's sum goes to all CTAs, each warp adds all of them.  `places`: one
// per warp of the cluster, which the next sum must not use.
template <int GS, typename F>
__device__ __forceinline__ F cluster_sum(F v, float2 *places, int size, int rank) {
  constexpr int W = GS / 32;
  const int lane = threadIdx.x % 32;
#pragma unroll
  for (int o = 16; o > 0; o /= 2) v = plus(v, from_lane(v, o));
  F *part = reinterpret_cast<F *>(places);
  if (lane < size) {
    const uint32_t to =
        ptx::mapa_shared(ptx::smem_u32(part + rank * W + threadIdx.x / 32), (uint32_t)lane);
    if constexpr (sizeof(F) == 8) {
      ptx::st_cluster_v2(to, v.x, v.y);
    } else {
      ptx::st_cluster_u32(to, __float_as_uint(v));
    }
  }
  __syncwarp();
  ptx::cluster_sync();
  v = lane < size * W ? part[lane] : F{};
  for (int i = lane + 32; i < size * W; i += 32) v = plus(v, part[i]);
#pragma unroll
  for (int o = 16; o > 0; o /= 2) v = plus(v, from_lane(v, o));
  return v;
}

// Slots of the ring for N tensors: `most`, or as many as fit in 200 KB (0:
// rows too long).
template <typename T, int GS, int VALS, int N>
constexpr int ring_slots(int most) {
  const int one = kCta<GS> * VALS * (int)sizeof(T) * N;
  const int fit = 200 * 1024 / one;
  return fit < 2 ? 0 : fit < most ? fit : most;
}

// The group for rows of H values: the smallest of which a thread takes 16, and
// beyond 4096 by what was measured.  False where rows are longer.
//
// Sizes between the powers of two: with phases a length just above (or, counting
// the phase, just below) one leaves half of a larger group's threads to masks,
// so there such sizes are worth it (bf16 with residual: 32736 x 1025 on 96
// threads 54 us, its backward 68, on 128 82 and 97; 16376 x 2049 on 160 45 and
// 58, on 256 75 and 90; 8186 x 4099 on 320 47, on 512 78; float32 within 10 % of
// the larger ones, 1025 values 45 and 59).  Without phases idle threads cost little: 96 and 160 threads were slower
// (21845 x 1536 backward 51 us, on 128 45).
template <bool BACK, typename T, bool SHIFT, template <typename, int, int, bool, bool> class G,
          typename A>
bool by_length(A &a, cudaStream_t s, cudaError_t *e) {
  const int H = a.H + (SHIFT ? kPer<T> - 1 : 0);
  if (H <= 8 * 16) return G<T, 8, 16, SHIFT, false>::go(a, 1, s, e);
  // 246723 x 136 bf16 with residual 46 us, on 32 threads 74
  if (H <= 16 * 16) return G<T, 16, 16, SHIFT, false>::go(a, 1, s, e);
  if (H <= 32 * 16) return G<T, 32, 16, SHIFT, false>::go(a, 1, s, e);
  if (H <= 64 * 16) return G<T, 64, 16, SHIFT, false>::go(a, 1, s, e);
  if constexpr (SHIFT)
    if (H <= 96 * 16) return G<T, 96, 16, SHIFT, false>::go(a, 1, s, e);
  if (H <= 128 * 16) return G<T, 128, 16, SHIFT, false>::go(a, 1, s, e);
  if constexpr (SHIFT)
    if (H <= 160 * 16) return G<T, 160, 16, SHIFT, false>::go(a, 1, s, e);
  if (H <= 256 * 16) return G<T, 256, 16, SHIFT, false>::go(a, 1, s, e);
  // Rows of up to 8192: the backward on as many threads of 8 values as a row
  // needs, which leaves it twice the warps beside its columns' sums (bf16 with
  // ds: 8192 x 7168 on 896 79 us, on 1024 83, 512 of 16 values 94; 6553 x 5120
  // on 640 49, 1024 65; float32 the same on all).  With phases the long ones are
  // on 512 of 16, where fewer warps wait for those at a row's ends (4680 x 7169
  // bf16 69 us, 1024 of 8 80).  The forward on 512 of 16 (8192 x 7168 45 us,
  // 1024 of 8 50).
  if constexpr (BACK && (SHIFT || sizeof(T) == 2)) {
    if (H <= 640 * 8) return G<T, 640, 8, SHIFT, false>::go(a, 1, s, e);
    if (H <= 768 * 8) return G<T, 768, 8, SHIFT, false>::go(a, 1, s, e);
  }
  if constexpr (BACK && !SHIFT && sizeof(T) == 2)
    if (H <= 896 * 8) return G<T, 896, 8, SHIFT, false>::go(a, 1, s, e);
  if constexpr (SHIFT && !BACK)
    if (H <= 320 * 16) return G<T, 320, 16, SHIFT, false>::go(a, 1, s, e);
  constexpr int GS = BACK && !SHIFT ? 1024 : 512;
  if (H <= 8192) return G<T, GS, 8192 / GS, SHIFT, false>::go(a, 1, s, e);
  if constexpr (BACK) {
    // Longer ones on a cluster of 2, 4 or 8 such CTAs (with ds, bf16: 4096 x
    // 16384 158 us, 512 threads of 32 values 175; 2048 x 32768 175, a CTA a row
    // 760; three CTAs, for which the device has fewer places, cost more than
    // four: 2730 x 24576 292 and 211).
    int size = 2;
    while (size * 8192 < H) size *= 2;
    if (size <= kMostCluster) return G<T, 1024, 8, SHIFT, true>::go(a, size, s, e);
  } else if (H <= 16384) {
    // 1024 threads of 16, where two rows fit into the ring (3001 x 16384 bf16
    // with residual 65 us, 512 of 32 values 73).  With 64 registers bf16 spills
    // 80 bytes a thread, 144 with residual; half idle, just above 8192 values,
    // it runs at 56 % of the copy rate
    return G<T, 1024, 16, SHIFT, false>::go(a, 1, s, e);
  }
  return false;
}

// CTAs and groups of a launch over n rows: the rows of a round lie beside each
// other over the CTAs, so that few rows use many SMs.  A group's next row is a
// multiple of 8 on.
struct NormGrid {
  int ctas, groups;
};
template <int GS>
inline NormGrid norm_grid(int n, int most) {
  NormGrid g;
  most = most < 8 ? 8 : most - most % 8;
  g.ctas = n < most ? n : most;
  const int rows = (int)(((long long)n + g.ctas - 1) / g.ctas), all = kCta<GS> / GS;
  constexpr int warp = GS < 32 ? 32 / GS : 1;  // whole warps
  g.groups = rows < all ? (rows + warp - 1) / warp * warp : all;
  return g;
}

// Clusters of a launch over n rows, at most `most` and as many as the device
// holds at a time.  A cluster's next row keeps its phase where rows have one.
template <typename K>
inline cudaError_t cluster_grid(K kernel, int threads, int smem, int size, int n, int most, int per,
                                int (&resident)[64][kMostCluster + 1], int *clusters) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  int &r = resident[dev >= 0 && dev < 64 ? dev : 0][size];
  if (r == 0) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr;
    cfg.gridDim = dim3(size), cfg.blockDim = dim3(threads), cfg.dynamicSmemBytes = smem;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = size, attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr, cfg.numAttrs = 1;
    int found = 0;
    e = cudaOccupancyMaxActiveClusters(&found, kernel, &cfg);
    if (e != cudaSuccess) return e;
    r = found < 1 ? 1 : found;
  }
  most = r < most ? r : most;
  most = most < per ? per : most - most % per;
  *clusters = n < most ? n : most;
  return cudaSuccess;
}

inline bool on_bytes(const void *p, uintptr_t b) {
  return (reinterpret_cast<uintptr_t>(p) & (b - 1)) == 0;
}

}  // namespace moe
