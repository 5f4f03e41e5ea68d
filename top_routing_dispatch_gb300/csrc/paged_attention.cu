// Attention of one new token per sequence over a paged key-value cache:
//   out[s][h] = sum_j p_j V[j] / sum_j p_j,  p_j = exp(scale q . K[j] - m),
// j over the sequence's cached tokens (or its last `window` ones), K and V of
// the kv head that query head h shares with q_heads / kv_heads - 1 others.
//
// Bound: HBM.  Each cached value is used once per query head of its group, at
// most 16 multiply-adds a byte here, far below the tensor cores' rate, so the
// kernel is built to keep copies in flight and to spend few instructions:
//
//  - The scores and the weighted sum run on warp-level matrix instructions
//    (m16n8k16) with the cached values as the 16-row operand and up to 8 query
//    heads as the 8 columns: S^T = K Q^T, O^T = V^T P^T.  A single head costs
//    what eight cost.  The instruction's 8-column form suits a handful of
//    heads; the 128-row tensor-memory form would spend a tile's set-up on
//    operands that are read once.
//  - The order of the summed index is free, so every lane loads whole 16-byte
//    pieces of K and V rows straight into the registers the instruction wants
//    (no transposing loads): for K, lane (g, t) takes pieces t, t + 4, ... of
//    row g; for V, pieces g, g + 8, ... of rows 2t, 2t+1, 2t+8, 2t+9, paired
//    by byte permutes.
//  - Those pieces travel through shared memory only as a queue: each lane
//    copies its own pieces asynchronously into its own slots and reads them
//    back, several steps later, itself.  No barrier and no bank conflict, and
//    the queue runs on across the ends of sequences and heads.
//  - The work of all sequences and kv heads is one row of units (a unit: the
//    tokens that the CTA's warps take in one step), cut into equal ranges for
//    one wave of CTAs.  A range may end inside a sequence: its part (maximum,
//    sum and unnormalised output, float32) then goes to the workspace, and
//    the CTA that arrives last joins the parts in range order.
//  - The running maximum is raised only when a score exceeds it by 2^8 (in
//    the exponent's base 2): one vote a step instead of a reduction.
//
// float32 caches take the same road with multiply-adds on the FMA units in
// place of the matrix instructions, which have no float32 operands.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "kv_cache.cuh"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kMaxWorkers = 512;  // CTAs that may hold parts
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRaise = 8.f;
constexpr int kMinUnits = 2;  // fewer units are not worth a part of their own

struct AttnArgs {
  const void *q;
  long long q_stride;
  const uint8_t *kc, *vc;
  long long page_bytes;
  const int32_t *table, *lens;
  const float *kscale, *vscale;
  void *out;
  float *lse;
  int32_t *counters;  // one per (sequence, head group)
  float2 *part_ml;    // (2 kMaxWorkers, NH): maximum and sum of a part
  float *part_o;      // (2 kMaxWorkers, NH, D)
  int B, Hq, Hkv, G, VG, P, num_pages, max_pages, window;
  float scale_log2;
  int32_t *status;
};

__device__ __forceinline__ void cp_async16_zfill(uint32_t dst, const void *src, bool ok) {
  const int n = ok ? 16 : 0;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n)
               : "memory");
}
__device__ __forceinline__ void cp_async8_zfill(uint32_t dst, const void *src, bool ok) {
  const int n = ok ? 8 : 0;
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(n)
               : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a)
               : "memory");
  return v;
}
__device__ __forceinline__ uint32_t trans8x8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
template <bool F16>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (F16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// two e4m3 bytes (low half of x) as two halves
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t x) {
  const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)x, __NV_E4M3);
  return (uint32_t)r.x | ((uint32_t)r.y << 16);
}
__device__ __forceinline__ uint32_t word(const uint4 &v, int i) {
  return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}
__device__ __forceinline__ void store_out(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void store_out(float *p, float v) { *p = v; }

// One lane's piece of a raise of the running maxima: the reduction over the
// eight lanes that hold the same heads.
__device__ __forceinline__ float max_over_g(float v) {
  v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
  v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
  return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
}
__device__ __forceinline__ float sum_over_g(float v) {
  v += __shfl_xor_sync(0xffffffffu, v, 4);
  v += __shfl_xor_sync(0xffffffffu, v, 8);
  return v + __shfl_xor_sync(0xffffffffu, v, 16);
}
// exp2(a - b) of running maxima, 0 where the part is empty
__device__ __forceinline__ float rescale(float a, float b) {
  return a == -INFINITY ? 0.f : exp2f(a - b);
}

// ---------------------------------------------------------------------------
// bf16 and e4m3 caches: matrix instructions.  NT: groups of 8 query heads.
// ---------------------------------------------------------------------------
template <int D_, bool E4M3, int NT>
struct MmaPath {
  using Out = __nv_bfloat16;
  static constexpr int D = D_, KEYS = 16, NH = 8 * NT, EB = E4M3 ? 1 : 2;
  static constexpr int KE = 16 / EB;                    // values of a K piece
  static constexpr int KJ = D / KE / 4;                 // K pieces per lane and row
  static constexpr int VE = E4M3 && D >= 128 ? 16 : 8;  // values of a V piece
  static constexpr int MI = D / (8 * VE), MJ = VE / 2;
  static constexpr int LOADS = 2 * KJ + 4 * MI;
  static constexpr int STAGE_BYTES = LOADS * 512;
  static constexpr int CH = 8 * VE;  // output values of a merge chunk
  static constexpr int NCH = MI;
  static constexpr int Q_SMEM = 0;

  uint32_t qf[NT][KJ][E4M3 ? 8 : 4];
  float o[MI][MJ][NT][4];
  float m[NT][2], l[NT][2], mult[NT][2];

  __device__ __forceinline__ static void issue(uint32_t slot, const uint8_t *k, const uint8_t *v,
                                               int lo, int hi, int lane) {
    const int g = lane >> 2, t = lane & 3;
    uint32_t dst = slot + lane * 16;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int row = g + 8 * r;
      const bool ok = row >= lo && row < hi;
      const uint8_t *src = k + (size_t)row * (D * EB) + t * 16;
#pragma unroll
      for (int j = 0; j < KJ; ++j, dst += 512) cp_async16_zfill(dst, src + j * 64, ok);
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int row = 2 * t + (r & 1) + 8 * (r >> 1);
      const bool ok = row >= lo && row < hi;
      const uint8_t *src = v + (size_t)row * (D * EB) + g * (VE * EB);
#pragma unroll
      for (int i = 0; i < MI; ++i, dst += 512) {
        if constexpr (VE * EB == 16)
          cp_async16_zfill(dst, src + i * 128, ok);
        else
          cp_async8_zfill(dst, src + i * 64, ok);
      }
    }
  }

  // nh query heads from q (head rows contiguous); sc: scale (and k scale)
  __device__ __forceinline__ void begin(const Out *q, int nh, float sc, int lane, float *) {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const bool ok = 8 * n + g < nh;
      const uint4 *row = reinterpret_cast<const uint4 *>(q + (size_t)(ok ? 8 * n + g : 0) * D);
      if constexpr (!E4M3) {
#pragma unroll
        for (int j = 0; j < KJ; ++j) {
          const uint4 x = ok ? __ldg(row + t + 4 * j) : make_uint4(0, 0, 0, 0);
          qf[n][j][0] = x.x, qf[n][j][1] = x.y, qf[n][j][2] = x.z, qf[n][j][3] = x.w;
        }
        mult[n][0] = mult[n][1] = sc;
      } else {
        // e4m3 values are halves exactly; q as halves too, each head scaled by
        // a power of two so that its largest value is in [1, 2): bf16's 8
        // significant bits fit, and what falls under 2^-24 of the largest goes
        float f[KJ][16], top = 0.f;
#pragma unroll
        for (int j = 0; j < KJ; ++j)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint4 x = ok ? __ldg(row + 2 * (t + 4 * j) + i) : make_uint4(0, 0, 0, 0);
            const __nv_bfloat162 *h = reinterpret_cast<const __nv_bfloat162 *>(&x);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 y = __bfloat1622float2(h[e]);
              f[j][8 * i + 2 * e] = y.x, f[j][8 * i + 2 * e + 1] = y.y;
              top = fmaxf(top, fmaxf(fabsf(y.x), fabsf(y.y)));
            }
          }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        int ex = (int)(__float_as_uint(top) >> 23);
        ex = ex < 1 ? 1 : ex > 253 ? 253 : ex;
        const float down = __uint_as_float((uint32_t)(254 - ex) << 23);  // 2^(127 - ex)
        const float up = __uint_as_float((uint32_t)ex << 23) * sc;       // 2^(ex - 127)
#pragma unroll
        for (int j = 0; j < KJ; ++j)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const __half2 h = __floats2half2_rn(f[j][2 * e] * down, f[j][2 * e + 1] * down);
            qf[n][j][e] = *reinterpret_cast<const uint32_t *>(&h);
          }
        mult[n][0] = __shfl_sync(0xffffffffu, up, 8 * t);
        mult[n][1] = __shfl_sync(0xffffffffu, up, 8 * t + 4);
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) m[n][e] = -INFINITY, l[n][e] = 0.f;
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < MJ; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[i][j][n][e] = 0.f;
    }
  }

  // keys [lo, hi) of the 16 in the slot
  __device__ __forceinline__ void step(uint32_t slot, int lo, int hi, int nh, int lane,
                                       const float *) {
    const int g = lane >> 2;
    uint32_t src = slot + lane * 16;
    float s[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
#pragma unroll
    for (int j = 0; j < KJ; ++j) {
      const uint4 a = lds128(src + j * 512), b = lds128(src + (KJ + j) * 512);
      if constexpr (!E4M3) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          mma16816<false>(s[n], a.x, b.x, a.y, b.y, qf[n][j][0], qf[n][j][1]);
          mma16816<false>(s[n], a.z, b.z, a.w, b.w, qf[n][j][2], qf[n][j][3]);
        }
      } else {
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const uint32_t x = word(a, w), y = word(b, w);
          const uint32_t a0 = e4m3x2_to_f16x2(x & 0xffffu), a2 = e4m3x2_to_f16x2(x >> 16);
          const uint32_t a1 = e4m3x2_to_f16x2(y & 0xffffu), a3 = e4m3x2_to_f16x2(y >> 16);
#pragma unroll
          for (int n = 0; n < NT; ++n)
            mma16816<true>(s[n], a0, a1, a2, a3, qf[n][j][2 * w], qf[n][j][2 * w + 1]);
        }
      }
    }
    src += 2 * KJ * 512;
    // scores in base 2; masked keys are -inf
    const bool in0 = g >= lo && g < hi, in1 = g + 8 >= lo && g + 8 < hi;
    bool high = false;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        s[n][e] = in0 ? s[n][e] * mult[n][e] : -INFINITY;
        s[n][2 + e] = in1 ? s[n][2 + e] * mult[n][e] : -INFINITY;
        high |= fmaxf(s[n][e], s[n][2 + e]) > m[n][e] + kRaise;
      }
    }
    if (__any_sync(0xffffffffu, high)) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float top = fmaxf(m[n][e], max_over_g(fmaxf(s[n][e], s[n][2 + e])));
          const float f = rescale(m[n][e], top);
          m[n][e] = top;
          l[n][e] *= f;
#pragma unroll
          for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int j = 0; j < MJ; ++j) {
              o[i][j][n][e] *= f;
              o[i][j][n][2 + e] *= f;
            }
        }
    }
    uint32_t ph[NT][2], pl[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float p[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float mm = m[n][e & 1] == -INFINITY ? 0.f : m[n][e & 1];
        p[e] = exp2f(s[n][e] - mm);
      }
      l[n][0] += p[0] + p[2];
      l[n][1] += p[1] + p[3];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        if constexpr (E4M3) {
          // halves keep 11 significant bits of p next to e4m3's 4 of V
          const __half2 h = __floats2half2_rn(p[2 * r], p[2 * r + 1]);
          ph[n][r] = trans8x8(*reinterpret_cast<const uint32_t *>(&h));
        } else {
          // p in two bf16 parts: one alone would round the result as much as
          // its own rounding to bf16 does again
          const __nv_bfloat162 h = __floats2bfloat162_rn(p[2 * r], p[2 * r + 1]);
          const float2 hf = __bfloat1622float2(h);
          const __nv_bfloat162 w = __floats2bfloat162_rn(p[2 * r] - hf.x, p[2 * r + 1] - hf.y);
          ph[n][r] = trans8x8(*reinterpret_cast<const uint32_t *>(&h));
          pl[n][r] = trans8x8(*reinterpret_cast<const uint32_t *>(&w));
        }
      }
    }
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      uint4 v[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) v[r] = lds128(src + (r * MI + i) * 512);
#pragma unroll
      for (int j = 0; j < MJ; ++j) {
        uint32_t a0, a1, a2, a3;
        if constexpr (!E4M3) {
          const uint32_t x0 = word(v[0], j), x1 = word(v[1], j);
          const uint32_t x2 = word(v[2], j), x3 = word(v[3], j);
          a0 = __byte_perm(x0, x1, 0x5410), a1 = __byte_perm(x0, x1, 0x7632);
          a2 = __byte_perm(x2, x3, 0x5410), a3 = __byte_perm(x2, x3, 0x7632);
        } else {
          const int w = j >> 1;
          const uint32_t sel = j & 1 ? 0x7362 : 0x5140;
          const uint32_t x = __byte_perm(word(v[0], w), word(v[1], w), sel);
          const uint32_t y = __byte_perm(word(v[2], w), word(v[3], w), sel);
          a0 = e4m3x2_to_f16x2(x & 0xffffu), a1 = e4m3x2_to_f16x2(x >> 16);
          a2 = e4m3x2_to_f16x2(y & 0xffffu), a3 = e4m3x2_to_f16x2(y >> 16);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          mma16816<E4M3>(o[i][j][n], a0, a1, a2, a3, ph[n][0], ph[n][1]);
          if constexpr (!E4M3) mma16816<false>(o[i][j][n], a0, a1, a2, a3, pl[n][0], pl[n][1]);
        }
      }
    }
  }

  // this warp's maxima and sums, by head
  __device__ __forceinline__ void stats(float *sm, float *sl, int lane) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float sum = sum_over_g(l[n][e]);
        if (lane < 4) sm[8 * n + 2 * lane + e] = m[n][e], sl[8 * n + 2 * lane + e] = sum;
      }
  }

  // output chunk i times f[head] into buf (NH, CH)
  __device__ __forceinline__ void chunk(int i, const float *f, float *buf, int lane) {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int ii = 0; ii < MI; ++ii) {
      if (ii != i) continue;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int head = 8 * n + 2 * t + e;
          const float ff = f[head];
#pragma unroll
          for (int j = 0; j < MJ; ++j)
            *reinterpret_cast<float2 *>(buf + head * CH + VE * g + 2 * j) =
                make_float2(o[ii][j][n][e] * ff, o[ii][j][n][2 + e] * ff);
        }
    }
  }
};

// ---------------------------------------------------------------------------
// float32 caches: FMA units, up to 8 query heads, q in shared memory.
// ---------------------------------------------------------------------------
template <int D_>
struct FmaPath {
  using Out = float;
  static constexpr int D = D_, KEYS = 8, NH = 8, EB = 4;
  static constexpr int KJ = D / 16;            // K pieces per lane (row g, pieces t + 4j)
  static constexpr int VR = D >= 128 ? 1 : 2;  // rows of one V load of the warp
  static constexpr int VJ = D > 128 ? 2 : 1;   // V pieces per lane and row
  static constexpr int VL = KEYS / VR * VJ;
  static constexpr int LOADS = KJ + VL;
  static constexpr int STAGE_BYTES = LOADS * 512;
  static constexpr int CH = D > 128 ? 128 : D;
  static constexpr int NCH = D / CH;
  static constexpr int Q_SMEM = NH * D;

  float o[NH][VJ][4];
  float m[NH], l[NH];
  float mult;

  __device__ __forceinline__ static void issue(uint32_t slot, const uint8_t *k, const uint8_t *v,
                                               int lo, int hi, int lane) {
    const int g = lane >> 2, t = lane & 3;
    uint32_t dst = slot + lane * 16;
    const bool okk = g >= lo && g < hi;
    const uint8_t *ks = k + (size_t)g * (D * EB) + t * 16;
#pragma unroll
    for (int j = 0; j < KJ; ++j, dst += 512) cp_async16_zfill(dst, ks + j * 64, okk);
    const int sub = VR == 2 ? lane >> 4 : 0, piece = VR == 2 ? lane & 15 : lane;
#pragma unroll
    for (int r = 0; r < KEYS / VR; ++r) {
      const int row = r * VR + sub;
      const bool ok = row >= lo && row < hi;
      const uint8_t *src = v + (size_t)row * (D * EB) + piece * 16;
#pragma unroll
      for (int j = 0; j < VJ; ++j, dst += 512) cp_async16_zfill(dst, src + j * 512, ok);
    }
  }

  __device__ __forceinline__ void begin(const Out *q, int nh, float sc, int, float *qs) {
    mult = sc;
    for (int e = threadIdx.x; e < nh * D; e += blockDim.x) qs[e] = __ldg(q + e);
    __syncthreads();
#pragma unroll
    for (int h = 0; h < NH; ++h) {
      m[h] = -INFINITY, l[h] = 0.f;
#pragma unroll
      for (int j = 0; j < VJ; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[h][j][e] = 0.f;
    }
  }

  __device__ __forceinline__ void step(uint32_t slot, int lo, int hi, int nh, int lane,
                                       const float *qs) {
    const int g = lane >> 2, t = lane & 3;
    const uint32_t src = slot + lane * 16;
    float4 k[KJ];
#pragma unroll
    for (int j = 0; j < KJ; ++j) {
      const uint4 x = lds128(src + j * 512);
      k[j] = make_float4(__uint_as_float(x.x), __uint_as_float(x.y), __uint_as_float(x.z),
                         __uint_as_float(x.w));
    }
    const bool in = g >= lo && g < hi;
    float p[NH];
    bool high = false;
#pragma unroll
    for (int h = 0; h < NH; ++h) {
      if (h >= nh) break;
      const float4 *qr = reinterpret_cast<const float4 *>(qs + h * D) + t;
      float a = 0.f, b = 0.f, c = 0.f, d = 0.f;
#pragma unroll
      for (int j = 0; j < KJ; ++j) {
        const float4 x = qr[4 * j];
        a = fmaf(k[j].x, x.x, a), b = fmaf(k[j].y, x.y, b);
        c = fmaf(k[j].z, x.z, c), d = fmaf(k[j].w, x.w, d);
      }
      float s = (a + b) + (c + d);
      s += __shfl_xor_sync(0xffffffffu, s, 1);
      s += __shfl_xor_sync(0xffffffffu, s, 2);
      p[h] = in ? s * mult : -INFINITY;
      high |= p[h] > m[h] + kRaise;
    }
    if (__any_sync(0xffffffffu, high)) {
#pragma unroll
      for (int h = 0; h < NH; ++h) {
        if (h >= nh) break;
        const float top = fmaxf(m[h], max_over_g(p[h]));
        const float f = rescale(m[h], top);
        m[h] = top;
        l[h] *= f;
#pragma unroll
        for (int j = 0; j < VJ; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[h][j][e] *= f;
      }
    }
#pragma unroll
    for (int h = 0; h < NH; ++h) {
      if (h >= nh) break;
      p[h] = exp2f(p[h] - (m[h] == -INFINITY ? 0.f : m[h]));
      l[h] += p[h];  // the key's four lanes hold the same sum
    }
    const int sub = VR == 2 ? lane >> 4 : 0;
#pragma unroll
    for (int r = 0; r < KEYS / VR; ++r) {
      float4 v[VJ];
#pragma unroll
      for (int j = 0; j < VJ; ++j) {
        const uint4 x = lds128(src + (KJ + r * VJ + j) * 512);
        v[j] = make_float4(__uint_as_float(x.x), __uint_as_float(x.y), __uint_as_float(x.z),
                           __uint_as_float(x.w));
      }
#pragma unroll
      for (int h = 0; h < NH; ++h) {
        if (h >= nh) break;
        const float w = __shfl_sync(0xffffffffu, p[h], 4 * (r * VR + sub));
#pragma unroll
        for (int j = 0; j < VJ; ++j) {
          o[h][j][0] = fmaf(w, v[j].x, o[h][j][0]), o[h][j][1] = fmaf(w, v[j].y, o[h][j][1]);
          o[h][j][2] = fmaf(w, v[j].z, o[h][j][2]), o[h][j][3] = fmaf(w, v[j].w, o[h][j][3]);
        }
      }
    }
  }

  __device__ __forceinline__ void stats(float *sm, float *sl, int lane) {
#pragma unroll
    for (int h = 0; h < NH; ++h) {
      const float sum = sum_over_g(l[h]);
      if (lane == 0) sm[h] = m[h], sl[h] = sum;
    }
  }

  __device__ __forceinline__ void chunk(int i, const float *f, float *buf, int lane) {
#pragma unroll
    for (int j = 0; j < VJ; ++j) {
      if (j != i) continue;
#pragma unroll
      for (int h = 0; h < NH; ++h) {
        float x[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[e] = o[h][j][e];
          if (VR == 2) x[e] += __shfl_xor_sync(0xffffffffu, x[e], 16);
        }
        const float ff = f[h];
        if (VR == 1 || lane < 16)
          *reinterpret_cast<float4 *>(buf + h * CH + 4 * lane) =
              make_float4(x[0] * ff, x[1] * ff, x[2] * ff, x[3] * ff);
      }
    }
  }
};

// ---------------------------------------------------------------------------

// What a sequence asks for: tokens [first, len), read from the KEYS-aligned
// token `base` on, in `units` units.
struct Seq {
  int len, first, base, units;
};

template <class P, int NW>
__device__ __forceinline__ Seq seq_info(const AttnArgs &a, int b) {
  Seq s;
  s.len = __ldg(a.lens + b);
  if (s.len < 0 || (long long)s.len > (long long)a.max_pages * a.P) s.len = 0;  // flagged once
  s.first = a.window > 0 && s.len > a.window ? s.len - a.window : 0;
  s.base = s.first / P::KEYS * P::KEYS;
  s.units = (s.len - s.base + NW * P::KEYS - 1) / (NW * P::KEYS);
  return s;
}

// A place in the row of units: unit c of (sequence b, head group h).
template <class P, int NW>
struct Cursor {
  int b, h, c;
  Seq s;
  __device__ __forceinline__ void next(const AttnArgs &a) {
    if (++c < s.units) return;
    c = 0;
    if (++h < a.Hkv * a.VG) return;
    h = 0;
    do {
      if (++b >= a.B) return;
      s = seq_info<P, NW>(a, b);
    } while (s.units == 0);
  }
  __device__ __forceinline__ int key(int warp) const { return s.base + (c * NW + warp) * P::KEYS; }
};

template <class P, int NW>
constexpr int stages() {
  constexpr int want = (NW == 8 ? 24 : 26) * 1024 / P::STAGE_BYTES;
  return want < 2 ? 2 : want > 8 ? 8 : want;
}

template <class P, int NW>
constexpr size_t smem_bytes() {
  return (size_t)NW * stages<P, NW>() * P::STAGE_BYTES +
         sizeof(float) * (NW * P::NH * P::CH + 3 * NW * P::NH + P::Q_SMEM);
}

template <class P, int NW>
__global__ void __launch_bounds__(NW * 32, NW == 8 ? 1 : 2) paged_attention_kernel(
    const AttnArgs a) {
  pdl_enter();
  constexpr int NT = NW * 32, ST = stages<P, NW>();
  constexpr int D = P::D, NH = P::NH, CH = P::CH;
  using Out = typename P::Out;
  extern __shared__ __align__(128) uint8_t smem[];
  float *buf = reinterpret_cast<float *>(smem + (size_t)NW * ST * P::STAGE_BYTES);
  float *sm = buf + NW * NH * CH, *sl = sm + NW * NH, *sf = sl + NW * NH;
  float *qs = sf + NW * NH;
  __shared__ long long sh_sum[NW], sh_u;
  __shared__ int sh_b, sh_last;
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int HV = a.Hkv * a.VG;

  // ---- the row of units, and this CTA's range [u0, u1)
  const int per = (a.B + NT - 1) / NT;
  const int b0 = tid * per, b1 = min(b0 + per, a.B);
  long long mine = 0;
  for (int b = b0; b < b1; ++b) {
    mine += seq_info<P, NW>(a, b).units;
    const int len = __ldg(a.lens + b);
    if (blockIdx.x == 0 && (len < 0 || (long long)len > (long long)a.max_pages * a.P))
      flag_status(a.status, MOE_DEV_BAD_CACHE);
  }
  long long inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  if (lane == 31) sh_sum[w] = inc;
  __syncthreads();
  long long before = 0, total = 0;
#pragma unroll
  for (int i = 0; i < NW; ++i) {
    if (i < w) before += sh_sum[i];
    total += sh_sum[i];
  }
  const long long T = total * HV;
  // rows of empty sequences
  for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
    if (seq_info<P, NW>(a, b).units) continue;
    for (int e = tid; e < a.Hq * D; e += NT)
      store_out(reinterpret_cast<Out *>(a.out) + (size_t)b * a.Hq * D + e, 0.f);
    if (a.lse)
      for (int e = tid; e < a.Hq; e += NT) a.lse[(size_t)b * a.Hq + e] = -INFINITY;
  }
  long long want = (T + kMinUnits - 1) / kMinUnits;
  const long long W = want < (long long)gridDim.x ? want : (long long)gridDim.x;
  if ((long long)blockIdx.x >= W) return;
  const long long u0 = blockIdx.x * T / W, u1 = (blockIdx.x + 1) * T / W;
  if (u0 >= u1) return;
  const long long excl = (before + inc - mine) * HV;
  if (u0 >= excl && u0 < excl + mine * HV) {
    long long at = excl;
    for (int b = b0; b < b1; ++b) {
      const long long n = (long long)seq_info<P, NW>(a, b).units * HV;
      if (u0 < at + n) {
        sh_b = b;
        sh_u = u0 - at;
        break;
      }
      at += n;
    }
  }
  __syncthreads();

  Cursor<P, NW> in, cur;  // where copies are issued, where values are used
  cur.b = sh_b;
  cur.s = seq_info<P, NW>(a, cur.b);
  cur.h = (int)(sh_u / cur.s.units);
  cur.c = (int)(sh_u - (long long)cur.h * cur.s.units);
  in = cur;
  long long in_left = u1 - u0, left = u1 - u0, u = u0;
  const uint32_t ring = ptx::smem_u32(smem) + (uint32_t)w * (ST * P::STAGE_BYTES);
  const size_t head_bytes = (size_t)a.P * (D * P::EB);
  int slot_in = 0, slot = 0;

  // the page of the next copies is looked up one step ahead
  auto lookup = [&]() -> int {
    const int key = in.key(w);
    return key < in.s.len ? __ldg(a.table + (size_t)in.b * a.max_pages + key / a.P) : 0;
  };
  int page = lookup();
  auto issue = [&]() {
    if (in_left > 0) {
      const int key = in.key(w);
      if (key < in.s.len) {
        const bool ok = page >= 0 && page < a.num_pages;
        if (!ok && lane == 0) flag_status(a.status, MOE_DEV_BAD_CACHE);
        const size_t off = (size_t)(ok ? page : 0) * a.page_bytes +
                           (size_t)(in.h / a.VG) * head_bytes + (size_t)(key % a.P) * (D * P::EB);
        P::issue(ring + slot_in * P::STAGE_BYTES, a.kc + off, a.vc + off,
                 ok ? in.s.first - key : P::KEYS, in.s.len - key, lane);
      }
      slot_in = slot_in + 1 == ST ? 0 : slot_in + 1;
      if (--in_left > 0) {
        in.next(a);
        page = lookup();
      }
    }
    ptx::cp_async_commit();
  };
#pragma unroll 1
  for (int i = 0; i < ST - 1; ++i) issue();

  P st;
  bool fresh = true;
  int nh = 0, h0 = 0;
#pragma unroll 1
  while (left > 0) {
    if (fresh) {
      const int hk = cur.h / a.VG, vg = cur.h - hk * a.VG;
      h0 = hk * a.G + vg * NH;
      nh = min(NH, a.G - vg * NH);
      const float sc = a.scale_log2 * (a.kscale ? __ldg(a.kscale + hk) : 1.f);
      st.begin(reinterpret_cast<const Out *>(a.q) + cur.b * a.q_stride + (size_t)h0 * D, nh, sc,
               lane, qs);
      fresh = false;
    }
    issue();
    ptx::cp_async_wait<ST - 1>();
    const int key = cur.key(w);
    if (key < cur.s.len)
      st.step(ring + slot * P::STAGE_BYTES, cur.s.first - key, cur.s.len - key, nh, lane, qs);
    slot = slot + 1 == ST ? 0 : slot + 1;
    --left;
    const bool end = cur.c + 1 == cur.s.units;
    if (!end && left > 0) {
      cur.c++;
      ++u;
      continue;
    }
    // ---- the segment ends: join the warps, then store the rows or the part
    const long long F = u - cur.c, L = F + cur.s.units - 1;  // the item's units
    const int wf = (int)(((F + 1) * W - 1) / T), wl = (int)(((L + 1) * W - 1) / T);
    const bool whole = wf == wl;
    const int part = 2 * (int)blockIdx.x + (F < u0 ? 0 : 1);
    const int hk = cur.h / a.VG;
    const float vs = a.vscale ? __ldg(a.vscale + hk) : 1.f;
    Out *out = reinterpret_cast<Out *>(a.out) + ((size_t)cur.b * a.Hq + h0) * D;
    float *lse = a.lse ? a.lse + (size_t)cur.b * a.Hq + h0 : nullptr;
    st.stats(sm + w * NH, sl + w * NH, lane);
    __syncthreads();
    if (tid < nh) {  // warp factors; with them the sum, and the factor of a whole row
      float top = -INFINITY, sum = 0.f;
      for (int i = 0; i < NW; ++i) top = fmaxf(top, sm[i * NH + tid]);
      for (int i = 0; i < NW; ++i) {
        const float f = rescale(sm[i * NH + tid], top);
        sum += sl[i * NH + tid] * f;
        sf[i * NH + tid] = f;
      }
      if (whole) {
        for (int i = 0; i < NW; ++i) sf[i * NH + tid] *= vs / sum;
        if (lse) lse[tid] = (top + log2f(sum)) * kLn2;
      } else {
        __stcg(a.part_ml + (size_t)part * NH + tid, make_float2(top, sum));
      }
    }
    __syncthreads();
#pragma unroll 1
    for (int i = 0; i < P::NCH; ++i) {
      st.chunk(i, sf + w * NH, buf + w * NH * CH, lane);
      __syncthreads();
      for (int e = tid; e < nh * CH; e += NT) {
        float x = 0.f;
#pragma unroll
        for (int k = 0; k < NW; ++k) x += buf[k * NH * CH + e];
        const int at = (e / CH) * D + i * CH + e % CH;
        if (whole)
          store_out(out + at, x);
        else
          __stcg(a.part_o + (size_t)part * NH * D + at, x);
      }
      __syncthreads();
    }
    if (!whole) {
      __threadfence();
      __syncthreads();
      if (tid == 0) {
        int32_t *cnt = a.counters + (size_t)cur.b * HV + cur.h;
        const int n = atomicAdd(cnt, 1);
        sh_last = n == wl - wf;
        if (sh_last) *cnt = 0;  // ready for the next call
        __threadfence();
      }
      __syncthreads();
      if (sh_last) {  // every part is there: join them in range order
        auto part_of = [&](int k) { return 2 * k + (F < k * T / W ? 0 : 1); };
        for (int e = tid; e < nh * D; e += NT) {
          const int h = e / D;
          float top = -INFINITY, sum = 0.f, x = 0.f;
          for (int k0 = wf; k0 <= wl; k0 += 8) {
            float2 ml[8];
            float y[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              if (k0 + k > wl) continue;
              const size_t p = part_of(k0 + k);
              ml[k] = __ldcg(a.part_ml + p * NH + h);
              y[k] = __ldcg(a.part_o + p * NH * D + e);
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              if (k0 + k > wl) continue;
              const float t2 = fmaxf(top, ml[k].x);
              const float f = rescale(top, t2), f2 = rescale(ml[k].x, t2);
              sum = sum * f + ml[k].y * f2;
              x = x * f + y[k] * f2;
              top = t2;
            }
          }
          store_out(out + e, x * (vs / sum));
          if (lse && e % D == 0) lse[h] = (top + log2f(sum)) * kLn2;
        }
      }
    }
    fresh = true;
    ++u;
    if (left > 0) cur.next(a);
  }
  ptx::cp_async_wait<0>();
}

inline int head_groups(const KVCache &c, int nh) {
  return (c.q_heads / c.kv_heads + nh - 1) / nh;
}
// query heads that one read of a kv head serves
inline int item_heads(const KVCache &c) {
  return c.cache_dtype == MOE_F32 || c.q_heads / c.kv_heads <= 8 ? 8 : 16;
}
inline size_t align256(size_t v) { return (v + 255) & ~(size_t)255; }

template <class P, int NW>
cudaError_t launch(const AttnArgs &a, cudaStream_t s) {
  constexpr size_t bytes = smem_bytes<P, NW>();
  auto kernel = paged_attention_kernel<P, NW>;
  static int grid[64] = {0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  int &g = grid[dev >= 0 && dev < 64 ? dev : 0];
  if (g == 0) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    int per_sm = 0;
    if (e == cudaSuccess)
      e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, NW * 32, bytes);
    if (e != cudaSuccess) return e;
    const int n = (per_sm > 0 ? per_sm : 1) * device_sm_count();
    g = n < kMaxWorkers ? n : kMaxWorkers;
  }
  return launch_pdl(kernel, dim3(g), dim3(NW * 32), bytes, s, a);
}

template <class P>
cudaError_t launch_p(const AttnArgs &a, cudaStream_t s) {
  return launch<P, 4>(a, s);
}

template <bool E4M3, int NT>
cudaError_t launch_mma(const AttnArgs &a, int D, cudaStream_t s) {
  if (D == 64) return launch_p<MmaPath<64, E4M3, NT>>(a, s);
  if (D == 128) return launch_p<MmaPath<128, E4M3, NT>>(a, s);
  return launch_p<MmaPath<256, E4M3, NT>>(a, s);
}

}  // namespace

size_t paged_attention_ws_bytes(const KVCache &c) {
  const int nh = item_heads(c);
  const size_t items = (size_t)c.num_seqs * c.kv_heads * head_groups(c, nh);
  return align256(items * sizeof(int32_t)) + align256(2 * kMaxWorkers * nh * sizeof(float2)) +
         align256((size_t)2 * kMaxWorkers * nh * c.head_dim * sizeof(float));
}

cudaError_t launch_paged_attention(const KVCache &c, const void *q, long long q_stride,
                                   const int32_t *seq_lens, int window, float scale, void *out,
                                   float *lse, void *ws, int32_t *status, cudaStream_t s) {
  if (c.num_seqs == 0) return cudaSuccess;
  const int nh = item_heads(c);
  const int eb = c.cache_dtype == MOE_F32 ? 4 : c.cache_dtype == MOE_BF16 ? 2 : 1;
  AttnArgs a = {};
  a.q = q, a.q_stride = q_stride;
  a.kc = reinterpret_cast<const uint8_t *>(c.k_cache);
  a.vc = reinterpret_cast<const uint8_t *>(c.v_cache);
  a.page_bytes = c.page_stride * eb;
  a.table = c.page_table, a.lens = seq_lens;
  a.kscale = c.k_scale, a.vscale = c.v_scale;
  a.out = out, a.lse = lse;
  a.B = c.num_seqs, a.Hq = c.q_heads, a.Hkv = c.kv_heads, a.G = c.q_heads / c.kv_heads;
  a.VG = head_groups(c, nh);
  a.P = c.page_size, a.num_pages = c.num_pages, a.max_pages = c.max_pages, a.window = window;
  a.scale_log2 = scale * kLog2e;
  a.status = status;
  uint8_t *w = reinterpret_cast<uint8_t *>(ws);
  a.counters = reinterpret_cast<int32_t *>(w);
  w += align256((size_t)a.B * a.Hkv * a.VG * sizeof(int32_t));
  a.part_ml = reinterpret_cast<float2 *>(w);
  w += align256(2 * kMaxWorkers * nh * sizeof(float2));
  a.part_o = reinterpret_cast<float *>(w);
  if (c.cache_dtype == MOE_F32) {
    if (c.head_dim == 64) return launch_p<FmaPath<64>>(a, s);
    if (c.head_dim == 128) return launch_p<FmaPath<128>>(a, s);
    return launch_p<FmaPath<256>>(a, s);
  }
  if (c.cache_dtype == MOE_E4M3)
    return nh == 8 ? launch_mma<true, 1>(a, c.head_dim, s) : launch_mma<true, 2>(a, c.head_dim, s);
  return nh == 8 ? launch_mma<false, 1>(a, c.head_dim, s) : launch_mma<false, 2>(a, c.head_dim, s);
}

}  // namespace moe
