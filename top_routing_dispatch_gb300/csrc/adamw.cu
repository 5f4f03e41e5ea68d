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
// Rounding of the codes.  To nearest, what moves a moment by less than half a
// step (3 to 6 %) is lost, step after step: beta2 = 0.999 moves a root by a
// thousandth.  At random (RANDOM), the chance of the upper code is such that the
// expectation of m, and of v (not of its root), is what was rounded, so the
// codes follow the recurrences on average.  65536 values of unit gradients, a
// quarter of each block 100 times smaller after 500 steps, 14 / (1 - beta2) later:
// sum of v against float32 states, for the quarter and for the others; and, where
// the quarter's gradients become zero, its movement 3000 steps later:
//   beta2 0.999: nearest 1e4, 1.04; random 0.999, 1.000
//   beta2 0.98: nearest 2e4, 2.4; random 1.000, 0.999
//   beta2 0.95: nearest 2.4, 1.12, 0.17 lr a step (m stays at its smallest
//   codes); random 0.999, 0.999, none
// (5 to 95 % of the single roots: 0.75 to 1.27 at random.)  With only the roots at
// random, m's smallest codes would move those parameters by 0.44 lr.  So beta2
// above 31/32 is rounded at random unless the caller says otherwise.  That costs
// 22 operations a value: the large layer below 1.12 instead of 1.10 ms, 38 million
// values in bf16 throughout 92 instead of 76 us.
// The chance comes from a hash of the step's number, the place in the block and
// v's bits: a step repeats itself, captured or not, wherever the block lies.
//
// A warp takes 256 values at a time: lane l those at 4 l .. 4 l + 3 and 128
// further on, in pairs for the two-operation instructions.
//
// Bound: HBM with float32 states (28 bytes a value in float32 throughout);
// instructions and the loads' latency come next, which is why the 8-bit form
// counts operations (36 a value): the largest root is the root of the largest
// v, one warp-wide maximum of integers does for a block (positive floats order
// as their bits), and what only an infinity, a NaN, a tiny v or a zero code
// needs stands apart behind one test.  24 warps an SM: with more the memory
// serves less (32: 403 million values 1.20 instead of 1.10 ms).
//
// Measured, 403 million values (bf16 parameters, float32 masters and
// gradients): float32 states 1.87 ms, 6.5 TB/s; 8-bit 1.10 ms, 6.6 TB/s.  38
// million in bf16 throughout with 8-bit states 76 us, 5.0 TB/s; 3.2 million
// float32 in 64 tensors 17.7 us.  Not kept: loads of the next block during this
// one's work in registers (the 8-bit layer 1.25 ms: registers spill) and by
// asynchronous copies of 4 to 16 bytes a lane into shared memory (1.3 ms).
#include <cuda_fp8.h>

#include <type_traits>

#include "pairs.cuh"
#include "roots.cuh"
#include "train.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kCtas = 3;         // of an SM
constexpr int kMostBlocks = 16;  // of a warp's turn
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

// The tensor that a turn belongs to, from k on: the last that does not begin
// behind it.
template <typename A>
__device__ __forceinline__ int tensor_of(const A &a, int turn, int k) {
  if (k + 1 >= a.count || turn < a.t[k + 1].first) return k;
  int lo = k + 1, hi = a.count;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    (turn < a.t[mid].first ? hi : lo) = mid;
  }
  return lo;
}

__device__ __forceinline__ bool plain_root(uint32_t bits) {
  return bits >= 0x0f800000u && bits < kInfBits;  // 2^-96 to the largest finite
}

// 4 neighbouring values as they lie in memory; those past `left` are 0
template <typename T>
struct Raw4 {
  static constexpr int W = (int)sizeof(T);  // words
  uint32_t w[W];
  template <bool FULL>
  __device__ __forceinline__ void load(const T *q, int left) {
    if constexpr (FULL && sizeof(T) == 4) {
      const uint4 u = *reinterpret_cast<const uint4 *>(q);
      w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
    } else if constexpr (FULL && sizeof(T) == 2) {
      const uint2 u = *reinterpret_cast<const uint2 *>(q);
      w[0] = u.x, w[1] = u.y;
    } else if constexpr (FULL) {
      w[0] = *reinterpret_cast<const uint32_t *>(q);
    } else {
      T e[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) e[i] = i < left ? q[i] : T{};
#pragma unroll
      for (int i = 0; i < W; ++i) w[i] = reinterpret_cast<const uint32_t *>(e)[i];
    }
  }
  template <bool FULL>
  __device__ __forceinline__ void store(T *q, int left) const {
    if constexpr (FULL && sizeof(T) == 4) {
      *reinterpret_cast<uint4 *>(q) = make_uint4(w[0], w[1], w[2], w[3]);
    } else if constexpr (FULL && sizeof(T) == 2) {
      *reinterpret_cast<uint2 *>(q) = make_uint2(w[0], w[1]);
    } else if constexpr (FULL) {
      *reinterpret_cast<uint32_t *>(q) = w[0];
    } else {
      const T *e = reinterpret_cast<const T *>(w);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < left) q[i] = e[i];
    }
  }
  __device__ __forceinline__ void get(float2 *f) const {
    if constexpr (sizeof(T) == 4) {
      f[0] = make_float2(__uint_as_float(w[0]), __uint_as_float(w[1]));
      f[1] = make_float2(__uint_as_float(w[2]), __uint_as_float(w[3]));
    } else if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        f[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
            (__nv_fp8x2_storage_t)(w[0] >> (16 * i) & 0xffff), __NV_E4M3);
        f[i] = __half22float2(__half2(h));
      }
    }
  }
  __device__ __forceinline__ void set(const float2 *f) {
    if constexpr (sizeof(T) == 4) {
      w[0] = __float_as_uint(f[0].x), w[1] = __float_as_uint(f[0].y);
      w[2] = __float_as_uint(f[1].x), w[3] = __float_as_uint(f[1].y);
    } else if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        reinterpret_cast<__nv_bfloat162 *>(w)[i] = __float22bfloat162_rn(f[i]);
    } else {
      const uint32_t x = __nv_cvt_float2_to_fp8x2(f[0], __NV_SATFINITE, __NV_E4M3);
      const uint32_t y = __nv_cvt_float2_to_fp8x2(f[1], __NV_SATFINITE, __NV_E4M3);
      w[0] = x | y << 16;
    }
  }
};

// Bits that look random, the upper ones most: xor-shifts and products with odd
// constants (fractions of the roots of 2, 3 and 5)
__device__ __forceinline__ uint32_t mixed(uint32_t x, uint32_t salt) {
  x = x * 0x6a09e667u + salt;
  x ^= x >> 15;
  x *= 0xbb67ae85u;
  x ^= x >> 16;
  return x * 0x3c6ef373u;
}
constexpr uint32_t kPlaceSalt = 0x9e3779b9u;  // for the next place of a block

// Rounding at random works on bits: 2^-120 of a value in units of the scale has
// float32's subnormals where e4m3 has its own, so codes are what the upper 12
// bits hold, and the lower 20 are the way from one to the next.
constexpr float kDown = 0x1p-120f, kUp = 0x1p120f;
constexpr uint32_t kGap = 1u << 20;
__device__ __forceinline__ float code_of(uint32_t bits) {
  return __uint_as_float(bits & ~(kGap - 1));
}
// Codes beside x: its mean over the chances (upper 20 bits) is x
__device__ __forceinline__ float2 random_codes(float2 x, uint32_t ca, uint32_t cb) {
  x = mul2(x, both(kDown));
  return mul2(make_float2(code_of(__float_as_uint(x.x) + (ca >> 12)),
                          code_of(__float_as_uint(x.y) + (cb >> 12))),
              both(kUp));
}
// Codes beside y >= 0, of which the mean square over the chances (upper 23 bits)
// is y^2: the upper one where y^2 - lo^2 is more than the chance times hi^2 - lo^2
__device__ __forceinline__ float2 random_roots(float2 y, uint32_t ca, uint32_t cb) {
  const float2 x = mul2(y, both(kDown));
  const uint32_t a = __float_as_uint(x.x) & ~(kGap - 1), b = __float_as_uint(x.y) & ~(kGap - 1);
  const float2 lo = mul2(make_float2(__uint_as_float(a), __uint_as_float(b)), both(kUp));
  const float2 hi = mul2(make_float2(__uint_as_float(a + kGap), __uint_as_float(b + kGap)), both(kUp));
  const float2 ll = mul2(mul2(lo, both(-1.f)), lo);
  const float2 u = add2(make_float2(__uint_as_float(ca >> 9 | 0x3f800000u),
                                    __uint_as_float(cb >> 9 | 0x3f800000u)), both(-1.f));
  const float2 way = fma2(y, y, ll), part = mul2(u, fma2(hi, hi, ll));
  return make_float2(way.x > part.x ? hi.x : lo.x, way.y > part.y ? hi.y : lo.y);
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
  uint32_t salt;  // of the step's number and the lane
};

// A lane's part of a block of 256 values.  PT, GT: types of parameter and
// gradient; MASTER: a bf16 parameter's float32 master (a float32 parameter's
// is a copy, written where there is one); RANDOM: codes rounded at random.
template <bool E4M3, bool RANDOM, typename PT, typename GT, bool MASTER>
struct Block {
  using ST = typename std::conditional<E4M3, uint8_t, float>::type;
  using WT = typename std::conditional<MASTER, float, PT>::type;  // what the step starts from
  Raw4<GT> g[2];
  Raw4<WT> p[2];
  Raw4<ST> m[2], v[2];
  float ms, vs;

  // the lane's place in the tensors; a block's halves are 128 values apart
  struct Place {
    const GT *g;
    PT *p;
    float *w;  // master, or NULL
    ST *m, *v;
    float *ms, *vs;
    int left[2];  // values that the lane has of a partial block
    __device__ __forceinline__ Place(const Tensor &t, long long block, int lane) {
      const long long at = block * kAdamBlock + 4 * lane;
      g = static_cast<const GT *>(t.grad) + at;
      p = static_cast<PT *>(t.param) + at;
      w = MASTER || (sizeof(PT) == 4 && t.master) ? t.master + at : nullptr;
      m = static_cast<ST *>(t.m) + at, v = static_cast<ST *>(t.v) + at;
      ms = t.ms + block, vs = t.vs + block;
      const long long rest = t.numel - at;
      left[0] = rest < 4 ? (int)rest : 4;
      left[1] = rest < 132 ? (int)rest - 128 : 4;
    }
    __device__ __forceinline__ void next() {
      g += kAdamBlock, p += kAdamBlock, m += kAdamBlock, v += kAdamBlock;
      if (MASTER || (sizeof(PT) == 4 && w)) w += kAdamBlock;
      if (E4M3) ++ms, ++vs;
    }
  };

  template <bool FULL>
  __device__ __forceinline__ void load(const Place &t) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int n = t.left[h];
      g[h].template load<FULL>(t.g + 128 * h, n);
      if constexpr (MASTER)
        p[h].template load<FULL>(t.w + 128 * h, n);
      else if constexpr (sizeof(PT) == 4)
        p[h].template load<FULL>((t.w ? t.w : t.p) + 128 * h, n);
      else
        p[h].template load<FULL>(t.p + 128 * h, n);
      m[h].template load<FULL>(t.m + 128 * h, n);
      v[h].template load<FULL>(t.v + 128 * h, n);
    }
    if (E4M3) ms = *t.ms, vs = *t.vs;
  }

  template <bool FULL>
  __device__ __forceinline__ void step(const Place &t, const Step &c, int lane) {
    float2 G[4], P[4], M[4], V[4], root[4];
#pragma unroll
    for (int h = 0; h < 2; ++h)
      g[h].get(G + 2 * h), p[h].get(P + 2 * h), m[h].get(M + 2 * h), v[h].get(V + 2 * h);
    uint32_t top_v = 0, low_v = ~0u;
    float top_m = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (c.scaled) G[k] = mul2(G[k], both(c.fac));
      if (E4M3) {
        M[k] = mul2(M[k], both(ms));
        V[k] = mul2(V[k], both(vs));
        V[k] = mul2(V[k], V[k]);
      }
      M[k] = fma2(M[k], both(c.b1), mul2(G[k], both(c.a1)));
      V[k] = fma2(V[k], both(c.b2), mul2(mul2(G[k], both(c.a2)), G[k]));
      const uint32_t x = __float_as_uint(V[k].x), y = __float_as_uint(V[k].y);
      low_v = min(low_v, min(x, y));
      top_v = max(top_v, max(x, y));
      if (E4M3) top_m = fmaxf(top_m, fmaxf(fabsf(M[k].x), fabsf(M[k].y)));
      root[k] = root2(V[k]);
    }
    if (!plain_root(low_v) || !plain_root(top_v)) {  // also a NaN, whose bits are larger
#pragma unroll
      for (int k = 0; k < 4; ++k)
        root[k] = make_float2(__fsqrt_rn(V[k].x), __fsqrt_rn(V[k].y));
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float2 d = fma2(root[k], both(c.c2), both(c.eps));
      d = mul2(M[k], make_float2(approx_rcp(d.x), approx_rcp(d.y)));
      P[k] = fma2(d, both(-c.c1), mul2(P[k], both(c.keep)));
    }
    if (E4M3) {
      uint32_t bm = __reduce_max_sync(~0u, __float_as_uint(top_m));
      uint32_t bv = __reduce_max_sync(~0u, top_v);
      const bool bad = bm >= kInfBits || bv >= kInfBits;
      if (bad) {
        bm = bv = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          bm = max(bm, max(finite_bits(M[k].x), finite_bits(M[k].y)));
          bv = max(bv, max(finite_bits(V[k].x), finite_bits(V[k].y)));
        }
        bm = __reduce_max_sync(~0u, bm);
        bv = __reduce_max_sync(~0u, bv);
      }
      const float sm = __fmul_rn(fmaxf(__uint_as_float(bm), kTiny), kInvMax);
      const float big = __uint_as_float(bv);
      const float sv = __fmul_rn(
          fmaxf(plain_root(bv) ? root2(make_float2(big, big)).x : __fsqrt_rn(big), kTiny), kInvMax);
      const float2 im = both(reciprocal(sm)), iv = both(reciprocal(sv));
      if (lane == 0) *t.ms = sm, *t.vs = sv;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float2 x = mul2(M[k], im), y = mul2(root[k], iv);
        if constexpr (RANDOM) {
          const uint32_t salt = c.salt + (k / 2 * 128 + k % 2 * 2) * kPlaceSalt;
          const uint32_t g = mixed(__float_as_uint(V[k].x), salt);
          const uint32_t h = mixed(__float_as_uint(V[k].y), salt + kPlaceSalt);
          x = random_codes(x, g * kPlaceSalt, h * kPlaceSalt);
          y = random_roots(y, g, h);
        }
        if (bad) {
          V[k] = make_float2(nan_if_not_finite(root[k].x, y.x), nan_if_not_finite(root[k].y, y.y));
          M[k] = make_float2(nan_if_not_finite(M[k].x, x.x), nan_if_not_finite(M[k].y, x.y));
        } else {
          V[k] = y, M[k] = x;
        }
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int n = t.left[h];
      Raw4<float> w;
      Raw4<PT> q;
      w.set(P + 2 * h), q.set(P + 2 * h);
      if (MASTER || (sizeof(PT) == 4 && t.w)) w.template store<FULL>(t.w + 128 * h, n);
      q.template store<FULL>(t.p + 128 * h, n);
      m[h].set(M + 2 * h), v[h].set(V + 2 * h);
      if constexpr (E4M3) {
        // a positive root keeps at least the smallest code
        uint32_t &r = v[h].w[0];
        if ((r - 0x01010101u) & ~r & 0x80808080u) {
          const float2 *z = root + 2 * h;
          const float e[4] = {z[0].x, z[0].y, z[1].x, z[1].y};
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (!(r >> (8 * i) & 0xff) && e[i] > 0.f) r |= 1u << (8 * i);
        }
      }
      m[h].template store<FULL>(t.m + 128 * h, n);
      v[h].template store<FULL>(t.v + 128 * h, n);
    }
  }
};

template <bool E4M3, bool RANDOM, typename PT, typename GT, bool MASTER, int CAP>
__global__ void __launch_bounds__(kThreads, kCtas)
    adamw_kernel(const __grid_constant__ StepArgs<CAP> a) {
  using B = Block<E4M3, RANDOM, PT, GT, MASTER>;
  pdl_enter();
  const int lane = threadIdx.x % 32;
  const float lr = a.lr_dev ? __ldg(a.lr_dev) : a.lr;
  Step c = {1.f, a.scale ? __ldg(a.scale) : 1.f, lr * a.state->inv1, a.state->inv2, a.b1, a.a1,
            a.b2, a.a2, a.eps, a.scale != nullptr, 0u};
  if constexpr (RANDOM) {
    const unsigned long long steps = (unsigned long long)a.state->steps;
    c.salt = mixed((uint32_t)steps, mixed((uint32_t)(steps >> 32), 1u)) + 4 * lane * kPlaceSalt;
  }
  int k = 0;
  // neighbouring turns on neighbouring CTAs' warps
  for (int turn = threadIdx.x / 32 * gridDim.x + blockIdx.x; turn < a.turns;
       turn += gridDim.x * kWarps) {
    k = tensor_of(a, turn, k);
    const Tensor &t = a.t[k];
    c.keep = 1.f - lr * t.decay;
    const long long block = (long long)(turn - t.first) * a.blocks;
    const long long rest = t.numel - block * kAdamBlock;
    int whole = 0;
    if (t.vec) whole = rest / kAdamBlock < a.blocks ? (int)(rest / kAdamBlock) : a.blocks;
    typename B::Place at(t, block, lane);
    B x;
#pragma unroll 1
    for (int i = 0; i < whole; ++i, at.next()) {
      x.template load<true>(at);
      x.template step<true>(at, c, lane);
    }
#pragma unroll 1
    for (int i = whole; i < a.blocks && (long long)i * kAdamBlock < rest; ++i) {
      const typename B::Place part(t, block + i, lane);
      x.template load<false>(part);
      x.template step<false>(part, c, lane);
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
constexpr int kPieces = 8;                    // of 16 bytes, of a thread's turn
constexpr int kNormUnit = kPieces * kThreads;  // of a CTA's turn
constexpr int kNormCtas = 1216;                // of a launch, at most
constexpr float kFewBits = 0x1p-118f;           // smaller sums of a turn lose too many

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

// A thread's sum of squares in a turn whose values lie where float32 cannot add
// the squares as they are: of `scale` times the values, which are read again.  A
// square that float32 does not hold makes the sum infinite.
__device__ __noinline__ double scaled_squares(const Part &t, long long first, long long pieces,
                                              long long tail, float scale) {
  const int per = t.bf16 ? 8 : 4;
  float s[4] = {0.f, 0.f, 0.f, 0.f};
  auto add = [&](long long at, float &to) {
    float f = t.bf16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(t.data)[at])
                     : static_cast<const float *>(t.data)[at];
    if (isinf(f * f)) f = INFINITY;
    f *= scale;
    to = fmaf(f, f, to);
  };
  if (tail < t.numel) add(tail, s[0]);
#pragma unroll 1
  for (int i = 0; i < kPieces && first + i * kThreads < pieces; ++i) {
    const long long at = (first + i * kThreads) * per;
#pragma unroll 1
    for (int j = 0; j < per; j += 4) {
#pragma unroll
      for (int k = 0; k < 4; ++k) add(at + j + k, s[k]);
    }
  }
  return (double)((s[0] + s[2]) + (s[1] + s[3])) / ((double)scale * scale);
}

// Bound: HBM.  A thread asks for all the pieces of its turn (128 bytes) before
// it uses one: 1.6 GB of float32 in 231 us, 103 % of the copy rate (reading
// alone is a little faster than copying); with 32 bytes 376 us.
//
// A turn's sum is float32 as it is from 2^-118 (what 65 squares below float32's
// normal numbers lose, at most 2^-144, is then less than its rounding) to the
// largest finite; else, unless all values are 0, of scaled values (403 million
// float32 values of 1e-21: 444 us, of ordinary size 223).
template <int CAP>
__global__ void __launch_bounds__(kThreads)
    grad_norm_kernel(const __grid_constant__ NormArgs<CAP> a) {
  pdl_enter();
  __shared__ double warps[kWarps];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  double sum = 0.0;
  int k = 0;
  for (int turn = blockIdx.x; turn < a.turns; turn += gridDim.x) {
    k = tensor_of(a, turn, k);
    const Part &t = a.t[k];
    const int per = t.bf16 ? 8 : 4;  // values of a piece
    const long long first = (long long)(turn - t.first) * kNormUnit + threadIdx.x;
    const long long pieces = t.numel / per;
    float2 s[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
    uint4 u[kPieces];
    if (t.vec) {
      const uint4 *q = static_cast<const uint4 *>(t.data) + first;
#pragma unroll
      for (int i = 0; i < kPieces; ++i)
        u[i] = first + i * kThreads < pieces ? __ldg(q + i * kThreads) : make_uint4(0, 0, 0, 0);
    } else {  // value by value
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        uint32_t w[4] = {0, 0, 0, 0};
        if (first + i * kThreads < pieces) {
          const long long at = (first + i * kThreads) * per;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (t.bf16) {
              const uint16_t *q = static_cast<const uint16_t *>(t.data) + at + 2 * j;
              w[j] = q[0] | (uint32_t)q[1] << 16;
            } else {
              w[j] = static_cast<const uint32_t *>(t.data)[at + j];
            }
          }
        }
        u[i] = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
    // the values behind the last piece, in the last turn
    const long long tail = turn - t.first == pieces / kNormUnit ? pieces * per + threadIdx.x : t.numel;
    uint32_t any = 0;  // bits of the values but their signs
    if (tail < t.numel)
      s[0].x = t.bf16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(t.data)[tail])
                      : static_cast<const float *>(t.data)[tail];
    any |= __float_as_uint(s[0].x);
    s[0].x *= s[0].x;
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const uint32_t w[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
      any |= w[0] | w[1] | w[2] | w[3];
      if (t.bf16) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 f =
              make_float2(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xffff0000u));
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
    s[0] = add2(s[0], s[1]);
    const float turn_sum = s[0].x + s[0].y;
    if (turn_sum >= kFewBits && turn_sum < INFINITY)
      sum += (double)turn_sum;
    else if (any & (t.bf16 ? 0x7fff7fffu : 0x7fffffffu))  // also a NaN
      sum += scaled_squares(t, first, pieces, tail, turn_sum < kFewBits ? 0x1p100f : 0x1p-10f);
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
  // without a limit nothing is clipped, whatever the norm; a NaN stays
  const float f = max_norm < INFINITY ? max_norm / (n + 1e-6f) : n == n ? 1.f : n;
  *norm = n;
  *factor = f > 1.f ? 1.f : f;
}

// ---------------------------------------------------------------- launches
constexpr int kSmallCap = 48, kLargeCap = 384;          // tensors of a step's launch
constexpr int kNormSmallCap = 128, kNormLargeCap = 1024;  // and of the norm's

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
    // a turn for the pieces and for what is left behind them
    turns += t[i].numel / (t[i].dtype == MOE_BF16 ? 8 : 4) / kNormUnit + 1;
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

template <bool E4M3, bool RANDOM, typename PT, typename GT, bool MASTER, int CAP>
cudaError_t step_cap(const moe_adamw_t &o, const moe_adamw_tensor_t *t, const Pending &q, bool last,
                     StepState *state, cudaStream_t s) {
  StepArgs<CAP> a;
  const int sms = device_sm_count();
  long long blocks = 0;
  for (int i = 0; i < q.count; ++i) blocks += ceil_of(t[q.index[i]].numel, kAdamBlock);
  const long long most = (long long)kCtas * sms, warps = most * kWarps;
  // The blocks of a turn.  8-bit states: eight neighbouring blocks' scales are
  // one sector of memory and their codes a run of 2 KB, so short turns cost
  // more (38 million values in bf16 throughout: two blocks 93 us, fourteen 77),
  // about 0.4 / n of the time; against that stands the longest share of a warp.
  // float32: a sixteenth of a share (3 million values: 17.0 us, the other rule
  // 18.2).
  a.blocks = 1;
  if (E4M3) {
    double best = 1e300;
    for (int n = 1; n <= kMostBlocks; ++n) {
      const double cost = (double)(ceil_of(ceil_of(blocks, n), warps) * n) * (1.0 + 0.4 / n);
      if (cost < best) a.blocks = n, best = cost;
    }
  } else {
    const long long share = blocks / (warps * 16);
    a.blocks = (int)(share < 1 ? 1 : share < kMostBlocks ? share : kMostBlocks);
  }
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
  const long long ctas = ceil_of(turns, kWarps);
  const unsigned grid = (unsigned)(ctas < 1 ? 1 : ctas < most ? ctas : most);
  return launch_pdl(adamw_kernel<E4M3, RANDOM, PT, GT, MASTER, CAP>, dim3(grid), dim3(kThreads), 0, s,
                    a);
}

template <bool E4M3, bool RANDOM, typename PT, typename GT, bool MASTER>
cudaError_t step_kind(const moe_adamw_t &o, const moe_adamw_tensor_t *t, const Pending &q,
                      bool last, StepState *state, cudaStream_t s) {
  return q.count <= kSmallCap
             ? step_cap<E4M3, RANDOM, PT, GT, MASTER, kSmallCap>(o, t, q, last, state, s)
             : step_cap<E4M3, RANDOM, PT, GT, MASTER, kLargeCap>(o, t, q, last, state, s);
}

template <bool E4M3, bool RANDOM>
cudaError_t step_launch(const moe_adamw_t &o, const moe_adamw_tensor_t *t, Kind k, Pending &q,
                        bool last, StepState *st, cudaStream_t s) {
  using B = __nv_bfloat16;
  cudaError_t e;
  if (!k.param_bf16)
    e = k.grad_bf16 ? step_kind<E4M3, RANDOM, float, B, false>(o, t, q, last, st, s)
                    : step_kind<E4M3, RANDOM, float, float, false>(o, t, q, last, st, s);
  else if (k.master)
    e = k.grad_bf16 ? step_kind<E4M3, RANDOM, B, B, true>(o, t, q, last, st, s)
                    : step_kind<E4M3, RANDOM, B, float, true>(o, t, q, last, st, s);
  else
    e = k.grad_bf16 ? step_kind<E4M3, RANDOM, B, B, false>(o, t, q, last, st, s)
                    : step_kind<E4M3, RANDOM, B, float, false>(o, t, q, last, st, s);
  q.count = 0;
  return e;
}

template <bool E4M3, bool RANDOM>
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
  if (left == 0) return step_launch<E4M3, RANDOM>(o, t, Kind{false, false, false}, q, true, state, s);
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
      if (q.count == kLargeCap || of[id] == 0)
        e = step_launch<E4M3, RANDOM>(o, t, k, q, left == 0, state, s);
    }
  }
  return e;
}

}  // namespace

size_t grad_norm_ws_bytes(int count) {
  const size_t launches = count < 1 ? 1 : (size_t)ceil_of(count, kNormLargeCap);
  return (launches * kNormCtas * sizeof(double) + 255) / 256 * 256;
}

cudaError_t launch_grad_norm(const moe_tensor_t *t, int count, float max_norm, float *norm,
                             float *factor, void *ws, cudaStream_t s) {
  double *part = static_cast<double *>(ws);
  int parts = 0;
  cudaError_t e = cudaSuccess;
  if (count <= kNormSmallCap) {
    e = norm_launch<kNormSmallCap>(t, count, part, &parts, s);
  } else {
    for (int i = 0; i < count && e == cudaSuccess; i += kNormLargeCap)
      e = norm_launch<kNormLargeCap>(t + i, count - i < kNormLargeCap ? count - i : kNormLargeCap, part, &parts, s);
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
  if (o.state_dtype != MOE_E4M3) return step_all<false, false>(o, t, count, st, s);
  const bool random = o.rounding == MOE_ROUND_RANDOM ||
                      (o.rounding == MOE_ROUND_BY_BETA2 && o.beta2 > 31.0 / 32.0);
  return random ? step_all<true, true>(o, t, count, st, s)
                : step_all<true, false>(o, t, count, st, s);
}

}  // namespace moe
