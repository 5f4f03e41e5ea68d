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
//  - The rows travel through shared memory in a queue of each warp's own
//    (asynchronous copies of whole lines, pieces permuted against bank
//    conflicts), which needs no barrier and runs on across the ends of
//    sequences and heads.
//  - The work of all sequences and kv heads is one row of units (a unit: the
//    tokens that the CTA's warps take in one step), cut into equal ranges for
//    one wave of CTAs.  A range may end inside a sequence: its part (maximum,
//    sum and unnormalised output, float32) then goes to the workspace.  When
//    its steps are done each CTA reports the parts it left; the one that
//    arrives last joins an item's parts in range order.
//  - The running maximum is raised only when a score exceeds it by 2^8 (in
//    the exponent's base 2): one vote a step instead of a reduction.
//
// float32 caches take the same road with multiply-adds on the FMA units in
// place of the matrix instructions, which have no float32 operands.
//
// Measured (cached bytes read once, of a copy rate of 6.7 TB/s): 62 sequences of
// 17 to 8191 tokens, 16/16 heads of 128, bf16: 111 us, 6.3 TB/s, 93 %; 128 of
// 500 to 12001, 64/8 heads, e4m3: 156 us, 6.1 TB/s (issue slots 57 % busy: the
// conversions of K and V and V's second product); one of 131071, 32/4 heads,
// bf16: 53 us, 5.0 TB/s, of which start and join take 11; one of 137 tokens: 7 us,
// the chain length, page, rows, exchange; a window of 2000 over 11 sequences,
// float32, 12/4 heads of 64: 15 us (bf16: 11).
#include <cuda_fp16.h>

#include "kv_cache.cuh"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kMaxWorkers = 512;  // CTAs that may hold parts
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRaise = 8.f;
constexpr int kItemCost = 2;  // a new item's overhead, in units
constexpr int kGroup = 12;    // parts joined at a time
constexpr int kSnap = 4;      // a range's end this near an item's edge moves to it (> kItemCost);
                              // ranges are no shorter unless there are more items than such ranges

struct AttnArgs {
  const void *q;
  long long q_stride;
  const uint8_t *kc, *vc;
  long long page_bytes;
  const int32_t *table, *lens;
  const float *kscale, *vscale;
  void *out;
  float *lse;
  int32_t *counters;        // of the item that begins in a range and goes on in the next: one per range
  int32_t *group_counters;  // one per part
  float2 *part_ml;    // (2 kMaxWorkers, NH): maximum and sum of a part
  float *part_o;      // (2 kMaxWorkers, NH, D)
  int B, Hq, Hkv, G, VG, P, num_pages, max_pages, window;
  float scale_log2;
  int32_t *status;
};

// 16 bytes global -> shared; EDGE: zeros unless ok (nothing is read then)
template <bool EDGE>
__device__ __forceinline__ void copy_piece(uint32_t dst, const uint8_t *src, bool ok) {
  if constexpr (EDGE) {
    const int n = ok ? 16 : 0;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n)
                 : "memory");
  } else {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  }
}
// 2^x by the hardware's approximation (relative error 2^-22, tiny results 0)
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a)
               : "memory");
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
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
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// four e4m3 bytes as two pairs of halves
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t x, uint32_t &lo, uint32_t &hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(x));
}
// a pair of halves that came from e4m3 as bf16, exactly: 4 significant bits, so
// the lower half of their float32 form is empty (NaN stays NaN)
__device__ __forceinline__ uint32_t f16_to_bf16(uint32_t x) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&x));
  return __byte_perm(__float_as_uint(f.x), __float_as_uint(f.y), 0x7632);
}
__device__ __forceinline__ uint32_t word(const uint4 &v, int i) {
  return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}
__device__ __forceinline__ void store_out(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void store_out(float *p, float v) { *p = v; }
__device__ __forceinline__ void store_out2(__nv_bfloat16 *p, float x, float y) {
  *reinterpret_cast<__nv_bfloat162 *>(p) = __floats2bfloat162_rn(x, y);
}
__device__ __forceinline__ void store_out2(float *p, float x, float y) {
  *reinterpret_cast<float2 *>(p) = make_float2(x, y);
}

// The rows of one step in the queue: KEYS rows of ROW bytes of K, then of V,
// each as it lies in the cache (a head's tokens are contiguous), except that
// the 16-byte pieces of a row are permuted: piece c of row r is in place
// c ^ spread(r).  Copies write whole 128-byte lines, and no two of the eight
// lanes that shared memory serves at a time read the same banks: for K those
// are pieces t + 4j of rows 2p and 2p + 1, for V pieces 2p and 2p + 1 of rows
// 0, 2, 4, 6 (or 1, 3, 5, 7).
__device__ __forceinline__ int spread(int r) { return (r & 2) | ((((r >> 2) ^ r) & 1) << 2); }

template <int KEYS, int ROW>
struct Rows {
  static constexpr int PIECES = ROW / 16;
  static constexpr int TILE = KEYS * ROW, LOADS = TILE / 512;
  static constexpr int MASK = PIECES < 8 ? PIECES - 1 : 7;  // of spread
  static_assert(TILE % 512 == 0, "whole warps of copies");

  // dst: the tile; lane: copies pieces lane, lane + 32, ...
  template <bool EDGE>
  __device__ __forceinline__ static void copy(uint32_t dst, const uint8_t *src, int lo, int hi,
                                              int lane) {
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
      const int x = i * 32 + lane, r = x / PIECES, c = x % PIECES;
      copy_piece<EDGE>(dst + r * ROW + ((c ^ (spread(r) & MASK)) * 16), src + x * 16,
                       r >= lo && r < hi);
    }
  }
};

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
  return a == -INFINITY ? 0.f : ex2(a - b);
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
  using Tile = Rows<KEYS, D * EB>;
  static constexpr int STAGE_BYTES = 2 * Tile::TILE;
  static constexpr int CH = 8 * VE;  // output values of a merge chunk
  static constexpr int NCH = MI;
  static constexpr int Q_SMEM = 0;

  static constexpr int QP = E4M3 ? 2 : 1;  // 16-byte pieces of q to a piece of K
  uint4 qr[NT][KJ][QP];  // the next item's queries, on their way
  uint32_t qf[NT][KJ][E4M3 ? 8 : 4];
  float o[MI][MJ][NT][4];
  float m[NT][2], l[NT][2], mult[NT][2];

  // asks for nh query heads (head rows contiguous)
  __device__ __forceinline__ void fetch(const Out *q, int nh, int lane) {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const bool ok = 8 * n + g < nh;
      const uint4 *row = reinterpret_cast<const uint4 *>(q + (size_t)(ok ? 8 * n + g : 0) * D);
#pragma unroll
      for (int j = 0; j < KJ; ++j)
#pragma unroll
        for (int i = 0; i < QP; ++i)
          qr[n][j][i] = ok ? __ldg(row + QP * (t + 4 * j) + i) : make_uint4(0, 0, 0, 0);
    }
  }

  // starts an item on the queries fetched; sc: scale (and k scale)
  __device__ __forceinline__ void begin(const Out *, int, float sc, int lane, float *) {
    const int t = lane & 3;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      if constexpr (!E4M3) {
#pragma unroll
        for (int j = 0; j < KJ; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) qf[n][j][e] = word(qr[n][j][0], e);
        mult[n][0] = mult[n][1] = sc;
      } else {
        // e4m3 values are halves exactly; q as halves too, each head scaled by
        // a power of two so that its largest value is in [2^14, 2^15) (its
        // products with 448 are far from float32's limit): all 8 bits of the
        // values down to 2^-31 of the largest are kept, less of smaller ones,
        // which is beyond what float32 sums keep beside the largest
        float top = 0.f;
#pragma unroll
        for (int j = 0; j < KJ; ++j)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const uint32_t x = word(qr[n][j][e >> 2], e & 3);
            const float2 y = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&x));
            top = fmaxf(top, fmaxf(fabsf(y.x), fabsf(y.y)));
          }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        int ex = (int)(__float_as_uint(top) >> 23);
        ex = ex < 15 ? 15 : ex > 253 ? 253 : ex;  // 2^127 is scaled to 2^15
        const float down = __uint_as_float((uint32_t)(268 - ex) << 23);  // 2^(141 - ex)
        const float up = __uint_as_float((uint32_t)(ex - 14) << 23) * sc;  // 2^(ex - 141)
#pragma unroll
        for (int j = 0; j < KJ; ++j)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const uint32_t x = word(qr[n][j][e >> 2], e & 3);
            const float2 y = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&x));
            const __half2 h = __floats2half2_rn(y.x * down, y.y * down);
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

  // the 16 keys of a slot; EDGE: only [lo, hi) count
  template <bool EDGE>
  __device__ __forceinline__ void step(uint32_t slot, int lo, int hi, int nh, int lane,
                                       const float *) {
    constexpr int ROW = D * EB, MASK = Tile::MASK;
    const int g = lane >> 2, t = lane & 3;
    const int sk = spread(g) & MASK;  // the same for rows g and g + 8
    // pieces t + 4j of row g: even j from k0, odd j from k1
    const uint32_t k0 = slot + g * ROW + ((t ^ sk) & 7) * 16;
    const uint32_t k1 = slot + g * ROW + (((t + 4) ^ sk) & 7) * 16;
    float s[NT][4], s2[NT][4];  // two chains of sums
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[n][e] = s2[n][e] = 0.f;
#pragma unroll
    for (int j = 0; j < KJ; ++j) {
      const uint32_t at = (j & 1 ? k1 : k0) + (j >> 1) * 128;
      const uint4 a = lds128(at), b = lds128(at + 8 * ROW);
      if constexpr (!E4M3) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          mma16816<false>(s[n], a.x, b.x, a.y, b.y, qf[n][j][0], qf[n][j][1]);
          mma16816<false>(s2[n], a.z, b.z, a.w, b.w, qf[n][j][2], qf[n][j][3]);
        }
      } else {
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          uint32_t a0, a1, a2, a3;
          e4m3x4_to_f16(word(a, w), a0, a2);
          e4m3x4_to_f16(word(b, w), a1, a3);
#pragma unroll
          for (int n = 0; n < NT; ++n)
            mma16816<true>(w & 1 ? s2[n] : s[n], a0, a1, a2, a3, qf[n][j][2 * w],
                           qf[n][j][2 * w + 1]);
        }
      }
    }
    // scores in base 2; masked keys are -inf
    const bool in0 = !EDGE || (g >= lo && g < hi), in1 = !EDGE || (g + 8 >= lo && g + 8 < hi);
    bool high = false;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        s[n][e] = in0 ? (s[n][e] + s2[n][e]) * mult[n][e] : -INFINITY;
        s[n][2 + e] = in1 ? (s[n][2 + e] + s2[n][2 + e]) * mult[n][e] : -INFINITY;
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
        p[e] = ex2(s[n][e] - mm);
      }
      l[n][0] += p[0] + p[2];
      l[n][1] += p[1] + p[3];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        // p in two bf16 parts: one alone would round the result as much as its
        // own rounding to bf16 does again, and halves end 2^-24 below the
        // largest p, which loses the tail of a steep softmax
        const __nv_bfloat162 h = __floats2bfloat162_rn(p[2 * r], p[2 * r + 1]);
        const float2 hf = __bfloat1622float2(h);
        const __nv_bfloat162 w = __floats2bfloat162_rn(p[2 * r] - hf.x, p[2 * r + 1] - hf.y);
        ph[n][r] = trans8x8(*reinterpret_cast<const uint32_t *>(&h));
        pl[n][r] = trans8x8(*reinterpret_cast<const uint32_t *>(&w));
      }
    }
    // rows 2t and 2t + 1 (+ 8): pieces g + 8i, or halves of piece g / 2
    uint32_t vrow[2];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int sv = spread(2 * t + c) & MASK;
      vrow[c] = slot + Tile::TILE + (2 * t + c) * ROW +
                (VE * EB == 16 ? (g ^ sv) * 16 : ((g >> 1) ^ sv) * 16 + (g & 1) * 8);
    }
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      uint4 v[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const uint32_t at = vrow[r & 1] + (r >> 1) * 8 * ROW + i * 128;
        if constexpr (VE * EB == 16) {
          v[r] = lds128(at);
        } else {
          const uint2 h = lds64(at);
          v[r].x = h.x, v[r].y = h.y;
        }
      }
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
          e4m3x4_to_f16(__byte_perm(word(v[0], w), word(v[1], w), sel), a0, a1);
          e4m3x4_to_f16(__byte_perm(word(v[2], w), word(v[3], w), sel), a2, a3);
          a0 = f16_to_bf16(a0), a1 = f16_to_bf16(a1), a2 = f16_to_bf16(a2), a3 = f16_to_bf16(a3);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) mma16816<false>(o[i][j][n], a0, a1, a2, a3, ph[n][0], ph[n][1]);
#pragma unroll
        for (int n = 0; n < NT; ++n) mma16816<false>(o[i][j][n], a0, a1, a2, a3, pl[n][0], pl[n][1]);
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

  // output chunks [i0, i0 + R) of heads < nh into buf (NH, R CH)
  template <int R>
  __device__ __forceinline__ void chunks(int i0, int nh, float *buf, int lane) {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      if (i < i0 || i >= i0 + R) continue;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int head = 8 * n + 2 * t + e;
          if (head >= nh) continue;
          float *to = buf + head * (R * CH) + (i - i0) * CH + VE * g;
#pragma unroll
          for (int j = 0; j < MJ; ++j)
            *reinterpret_cast<float2 *>(to + 2 * j) = make_float2(o[i][j][n][e], o[i][j][n][2 + e]);
        }
    }
  }
};

// ---------------------------------------------------------------------------
// float32 caches: FMA units, q in shared memory.  NH: 1, 4 or 8 query heads, all
// of them computed (those beyond the item's are of zeros), so that the heads'
// chains overlap and a call fetches no more code than its heads need (24
// sequences of 6500 tokens, 12/4 heads of 64: 46 us, against 65 with code for 8
// that left at the item's last head; 10/2 heads: 42 against 50; one set of inputs,
// part of which stays in L2: three sets in turn take 58 and 51).
// ---------------------------------------------------------------------------
template <int D_, int NH_>
struct FmaPath {
  using Out = float;
  static constexpr int D = D_, KEYS = 8, NH = NH_, EB = 4;
  static constexpr int KJ = D / 16;            // K pieces per lane (row g, pieces t + 4j)
  static constexpr int VR = D >= 128 ? 1 : 2;  // rows of one V load of the warp
  static constexpr int VJ = D > 128 ? 2 : 1;   // V pieces per lane and row
  using Tile = Rows<KEYS, D * EB>;
  static constexpr int STAGE_BYTES = 2 * Tile::TILE;
  static constexpr int CH = D > 128 ? 128 : D;
  static constexpr int NCH = D / CH;
  static constexpr int Q_SMEM = NH * D;

  static constexpr int QR = (NH * D / 4 + 127) / 128;
  float4 qr[QR];  // the next item's queries, on their way
  float o[NH][VJ][4];
  float m[NH], l[NH];
  float mult;

  // asks for nh query heads, shared out over the CTA's threads (128 of them)
  __device__ __forceinline__ void fetch(const Out *q, int nh, int) {
#pragma unroll
    for (int i = 0; i < QR; ++i) {
      const int e = threadIdx.x + i * 128;
      if (e < nh * D / 4) qr[i] = __ldg(reinterpret_cast<const float4 *>(q) + e);
    }
  }

  __device__ __forceinline__ void begin(const Out *, int nh, float sc, int, float *qs) {
    mult = sc;
    __syncthreads();  // qs is free
#pragma unroll
    for (int i = 0; i < QR; ++i) {
      const int e = threadIdx.x + i * 128;
      if (e < NH * D / 4)
        reinterpret_cast<float4 *>(qs)[e] =
            e < nh * D / 4 ? qr[i] : make_float4(0.f, 0.f, 0.f, 0.f);
    }
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

  template <bool EDGE>
  __device__ __forceinline__ void step(uint32_t slot, int lo, int hi, int nh, int lane,
                                       const float *qs) {
    constexpr int ROW = D * EB;
    const int g = lane >> 2, t = lane & 3;
    const uint32_t k0 = slot + g * ROW + (t ^ spread(g)) * 16;
    const uint32_t k1 = slot + g * ROW + ((t + 4) ^ spread(g)) * 16;
    float4 k[KJ];
#pragma unroll
    for (int j = 0; j < KJ; ++j) {
      const uint4 x = lds128((j & 1 ? k1 : k0) + (j >> 1) * 128);
      k[j] = make_float4(__uint_as_float(x.x), __uint_as_float(x.y), __uint_as_float(x.z),
                         __uint_as_float(x.w));
    }
    const bool in = !EDGE || (g >= lo && g < hi);
    float p[NH];
    bool high = false;
#pragma unroll
    for (int h = 0; h < NH; ++h) {
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
      p[h] = ex2(p[h] - (m[h] == -INFINITY ? 0.f : m[h]));
      l[h] += p[h];  // the key's four lanes hold the same sum
    }
    const int sub = VR == 2 ? lane >> 4 : 0, piece = VR == 2 ? lane & 15 : lane;
#pragma unroll
    for (int r = 0; r < KEYS / VR; ++r) {
      float4 v[VJ];
#pragma unroll
      for (int j = 0; j < VJ; ++j) {
        const int row = r * VR + sub;
        const uint4 x = lds128(slot + Tile::TILE + row * ROW + (piece ^ spread(row)) * 16 + j * 512);
        v[j] = make_float4(__uint_as_float(x.x), __uint_as_float(x.y), __uint_as_float(x.z),
                           __uint_as_float(x.w));
      }
#pragma unroll
      for (int h = 0; h < NH; ++h) {
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

  template <int R>
  __device__ __forceinline__ void chunks(int i0, int nh, float *buf, int lane) {
#pragma unroll
    for (int j = 0; j < VJ; ++j) {
      if (j < i0 || j >= i0 + R) continue;
#pragma unroll
      for (int h = 0; h < NH; ++h) {
        if (h >= nh) break;
        float x[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[e] = o[h][j][e];
          if (VR == 2) x[e] += __shfl_xor_sync(0xffffffffu, x[e], 16);
        }
        if (VR == 1 || lane < 16)
          *reinterpret_cast<float4 *>(buf + h * (R * CH) + (j - i0) * CH + 4 * lane) =
              make_float4(x[0], x[1], x[2], x[3]);
      }
    }
  }
};

// ---------------------------------------------------------------------------

// a / b for a >= 0, b > 0, in 32 bits where they fit
__device__ __forceinline__ long long quotient(long long a, long long b) {
  if (((unsigned long long)(a | b) >> 32) == 0) return (unsigned)a / (unsigned)b;
  return a / b;
}

// Tokens are counted in 32 bits, up to a few steps past a sequence's end.
constexpr int kMaxLen = 0x7fffffff - 1023;
__device__ __forceinline__ bool bad_length(const AttnArgs &a, int len) {
  return len < 0 || len > kMaxLen || (long long)len > (long long)a.max_pages * a.P;
}

// What a sequence asks for: tokens [first, len), read from the KEYS-aligned
// token `base` on, in `units` units.
struct Seq {
  int len, first, base, units;
};

template <class P, int NW>
__device__ __forceinline__ Seq seq_info(const AttnArgs &a, int b) {
  Seq s;
  s.len = __ldg(a.lens + b);
  if (bad_length(a, s.len)) s.len = 0;  // flagged once
  s.first = a.window > 0 && s.len > a.window ? s.len - a.window : 0;
  s.base = s.first / P::KEYS * P::KEYS;
  s.units = (s.len - s.base + NW * P::KEYS - 1) / (NW * P::KEYS);
  return s;
}

// CTAs of an SM, the output chunks that the warps exchange at a time, and the
// queue's depth: what the SM's shared memory and registers hold.
template <class P>
constexpr int ctas() {
  return P::STAGE_BYTES > 8192 ? 1 : P::NH * P::D <= (P::Q_SMEM ? 256 : 1024) ? 3 : 2;
}
template <class P>
constexpr int cta_bytes() {
  return (227 / ctas<P>() - 1) * 1024;
}
template <class P, int NW>
constexpr int round_chunks() {
  constexpr int fit = cta_bytes<P>() / 8 / (NW * P::NH * P::CH * 4);
  int n = P::NCH;  // a power of two; the rounds are whole
  while (n > 1 && n > fit) n /= 2;
  return n;
}
template <class P, int NW>
constexpr size_t merge_bytes() {
  return sizeof(float) *
         (NW * P::NH * P::CH * round_chunks<P, NW>() + 3 * NW * P::NH + P::Q_SMEM);
}
template <class P, int NW>
constexpr int stages() {
  constexpr int fit = (int)((cta_bytes<P>() - merge_bytes<P, NW>()) / (NW * P::STAGE_BYTES));
  static_assert(fit >= 2, "a queue of two steps");
  static_assert(P::NCH % round_chunks<P, NW>() == 0, "whole rounds");
  return fit > 8 ? 8 : fit;
}

template <class P, int NW>
constexpr size_t smem_bytes() {
  return (size_t)NW * stages<P, NW>() * P::STAGE_BYTES + merge_bytes<P, NW>();
}

// Counts this CTA's arrival; true in the CTA that arrives last of n, which then
// sees what the others stored.  Leaves the counter zero for the next call.
__device__ __forceinline__ bool arrive(int32_t *counter, int n, int *sh) {
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) {
    *sh = atomicAdd(counter, 1) == n - 1;
    if (*sh) *counter = 0;
    __threadfence();
  }
  __syncthreads();
  return *sh;
}

// Joins np parts in order, by the whole CTA: those of ranges first, first + step,
// ... of the item that begins in range wf; into the first one's part (out
// nullptr), or into the rows of nh heads at out.
template <class P, int NW>
__device__ __forceinline__ void join_parts(const AttnArgs &a, int first, int step, int wf, int np,
                                        int nh, float *sm, float *sl, float vs,
                                        typename P::Out *out, float *lse) {
  const bool to_part = out == nullptr;
  auto part_of = [=](int k) {
    return (size_t)(2 * (first + k * step) + (first + k * step == wf ? 1 : 0));
  };
  constexpr int D = P::D, NH = P::NH;
  // four outputs a thread and pass; each thread goes over the parts' maxima and
  // sums itself, in one round of loads with the outputs
  for (int e = threadIdx.x * 4; e < nh * D; e += NW * 32 * 4) {
    const int h = e / D;
    float top = -INFINITY, sum = 0.f;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k0 = 0; k0 < np; k0 += kGroup) {
      float2 ml[kGroup];
      float4 y[kGroup];
#pragma unroll
      for (int k = 0; k < kGroup; ++k) {
        ml[k] = make_float2(-INFINITY, 0.f);
        if (k0 + k < np) {
          const size_t p = part_of(k0 + k);
          ml[k] = __ldcg(a.part_ml + p * NH + h);
          y[k] = __ldcg(reinterpret_cast<const float4 *>(a.part_o + p * NH * D + e));
        }
      }
      float t2 = top;
#pragma unroll
      for (int k = 0; k < kGroup; ++k) t2 = fmaxf(t2, ml[k].x);
      const float f = rescale(top, t2);
      sum *= f, x.x *= f, x.y *= f, x.z *= f, x.w *= f;
      top = t2;
#pragma unroll
      for (int k = 0; k < kGroup; ++k)
        if (k0 + k < np) {
          const float r = rescale(ml[k].x, top);
          sum = fmaf(ml[k].y, r, sum);
          x.x = fmaf(y[k].x, r, x.x), x.y = fmaf(y[k].y, r, x.y);
          x.z = fmaf(y[k].z, r, x.z), x.w = fmaf(y[k].w, r, x.w);
        }
    }
    if (to_part) {
      // every thread of the head has to read part 0's maximum before it changes
      __stcg(reinterpret_cast<float4 *>(a.part_o + part_of(0) * NH * D + e), x);
      if (e % D == 0) sm[h] = top, sl[h] = sum;
    } else {
      const float f = vs / sum;
      store_out2(out + e, x.x * f, x.y * f);
      store_out2(out + e + 2, x.z * f, x.w * f);
      if (lse && e % D == 0) lse[h] = (top + log2f(sum)) * kLn2;
    }
  }
  if (to_part) {
    __syncthreads();
    if (threadIdx.x < nh)
      __stcg(a.part_ml + part_of(0) * NH + threadIdx.x, make_float2(sm[threadIdx.x], sl[threadIdx.x]));
  }
}

template <class P, int NW>
__global__ void __launch_bounds__(NW * 32, ctas<P>()) paged_attention_kernel(
    const __grid_constant__ AttnArgs a) {
  pdl_enter();
  constexpr int NT = NW * 32, ST = stages<P, NW>();
  constexpr int D = P::D, NH = P::NH, RC = round_chunks<P, NW>(), CH = P::CH * RC;
  using Out = typename P::Out;
  extern __shared__ __align__(128) uint8_t smem[];
  float *buf = reinterpret_cast<float *>(smem + (size_t)NW * ST * P::STAGE_BYTES);
  float *sm = buf + NW * NH * CH, *sl = sm + NW * NH, *sf = sl + NW * NH;
  float *qs = sf + NW * NH;
  __shared__ long long sh_sum[NW], sh_u[2], sh_S;
  __shared__ int sh_b, sh_h, sh_c, sh_last, sh_live[NW];
  __shared__ struct Part {
    int b, h, wf, wl;  // an item of which this range holds part 0 or 1
  } sh_part[2];
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int HV = a.Hkv * a.VG;

  // ---- the row of units, and this CTA's range [u0, u1)
  const int per = (a.B + NT - 1) / NT;
  const int b0 = tid * per, b1 = min(b0 + per, a.B);
  long long mine = 0;
  int live = 0;
  for (int b = b0; b < b1; ++b) {
    const int n = seq_info<P, NW>(a, b).units;
    mine += n ? n + kItemCost : 0;
    live += n != 0;
    if (blockIdx.x == 0 && bad_length(a, __ldg(a.lens + b)))
      flag_status(a.status, MOE_DEV_BAD_CACHE);
  }
  long long inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  live = __reduce_add_sync(0xffffffffu, live);
  if (lane == 31) sh_sum[w] = inc, sh_live[w] = live;
  __syncthreads();
  long long before = 0, total = 0, items = 0;
#pragma unroll
  for (int i = 0; i < NW; ++i) {
    items += sh_live[i];
    if (i < w) before += sh_sum[i];
    total += sh_sum[i];
  }
  // an item of n units stands for n + kItemCost in the row: what joining the
  // warps and starting over costs
  const long long T = total * HV;
  // rows of empty sequences
  for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
    if (seq_info<P, NW>(a, b).units) continue;
    for (int e = tid; e < a.Hq * D; e += NT)
      store_out(reinterpret_cast<Out *>(a.out) + (size_t)b * a.Hq * D + e, 0.f);
    if (a.lse)
      for (int e = tid; e < a.Hq; e += NT) a.lse[(size_t)b * a.Hq + e] = -INFINITY;
  }
  const long long want = max((T + kSnap - 1) / kSnap, items * HV);
  const long long W = min(want, (long long)gridDim.x);
  if ((long long)blockIdx.x >= W) return;
  // this CTA's range, its ends moved to the edges of items that they nearly meet
  const long long excl = (before + inc - mine) * HV;
  if (tid == 0) {
    sh_u[1] = T;
    sh_part[0].b = sh_part[1].b = -1;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const long long x = quotient((blockIdx.x + i) * T, W);
    if (x < excl || x >= excl + mine * HV) continue;
    long long at = excl;
    for (int b = b0; b < b1; ++b) {
      const int units = seq_info<P, NW>(a, b).units, n = units ? units + kItemCost : 0;
      if (x < at + (long long)n * HV) {
        const int h = (int)quotient(x - at, n);
        long long S = at + (long long)h * n;
        long long to = x - S < kSnap ? S : S + n - x < kSnap ? S + n : x;
        sh_u[i] = to;
        if (i == 0) {
          sh_b = b;
          sh_h = to == S + n ? h + 1 : h;  // HV: the next sequence
          sh_c = to == S || to == S + n ? 0 : (int)(to - S) - kItemCost;
          sh_S = to == S + n ? to : S;
        }
        break;
      }
      at += (long long)n * HV;
    }
  }
  __syncthreads();
  const long long u1 = sh_u[1];
  if (sh_u[0] >= u1) return;
  int b_first = sh_b, h_first = sh_h;
  const int c_first = sh_c;
  Seq s_first = seq_info<P, NW>(a, b_first);
  if (h_first == HV) {
    h_first = 0;
    do {
      s_first = seq_info<P, NW>(a, ++b_first);
    } while (s_first.units == 0);
  }
  long long S = sh_S;  // where the item begins in the row
  const uint32_t ring = ptx::smem_u32(smem) + (uint32_t)w * (ST * P::STAGE_BYTES);
  constexpr int ROW = D * P::EB, STRIDE = NW * P::KEYS;
  const size_t head_bytes = (size_t)a.P * ROW;
  const int page_step = STRIDE / a.P, off_step = STRIDE - page_step * a.P;

  // ---- the copying side: unit c of (sequence b, head group h), this warp's
  // first token `key` of it, in place `off` of its page; the page's number is
  // looked up one step ahead
  struct {
    int b, h, c, key, idx, off;
    Seq s;
  } in;
  in.b = b_first;
  in.s = s_first;
  in.h = h_first;
  in.c = c_first;
  long long in_S = S;
  // the units of the item that lie in the range
  auto units_of = [&](long long at, int units) {
    return (int)min((long long)units, u1 - at - kItemCost);
  };
  int in_end = units_of(in_S, in.s.units);
  bool more = true;
  int page = 0, slot_in = 0;
  size_t head_off = 0;
  auto lookup = [&]() {
    if (in.key < in.s.len) page = __ldg(a.table + (size_t)in.b * a.max_pages + in.idx);
  };
  auto enter = [&]() {  // the place of unit in.c
    in.key = in.s.base + (in.c * NW + w) * P::KEYS;
    in.idx = in.key / a.P;
    in.off = in.key - in.idx * a.P;
    head_off = (size_t)(a.VG == 1 ? in.h : in.h / a.VG) * head_bytes;
    lookup();
  };
  enter();
  auto issue = [&]() {
    if (more) {
      if (in.key < in.s.len) {
        const bool ok = (unsigned)page < (unsigned)a.num_pages;
        const size_t at = (size_t)(ok ? page : 0) * a.page_bytes + head_off + (size_t)in.off * ROW;
        const uint32_t dst = ring + slot_in * P::STAGE_BYTES;
        if (ok && in.key >= in.s.first && in.key + P::KEYS <= in.s.len) {
          P::Tile::template copy<false>(dst, a.kc + at, 0, 0, lane);
          P::Tile::template copy<false>(dst + P::Tile::TILE, a.vc + at, 0, 0, lane);
        } else {
          if (!ok && lane == 0) flag_status(a.status, MOE_DEV_BAD_CACHE);
          const int lo = ok ? in.s.first - in.key : P::KEYS, hi = in.s.len - in.key;
          P::Tile::template copy<true>(dst, a.kc + at, lo, hi, lane);
          P::Tile::template copy<true>(dst + P::Tile::TILE, a.vc + at, lo, hi, lane);
        }
      }
      slot_in = slot_in + 1 == ST ? 0 : slot_in + 1;
      if (++in.c < in_end) {
        in.key += STRIDE;
        in.idx += page_step;
        in.off += off_step;
        if (in.off >= a.P) in.off -= a.P, ++in.idx;
        lookup();
      } else {
        in_S += in.s.units + kItemCost;
        more = in_S < u1;
        if (more) {
          in.c = 0;
          if (++in.h == HV) {
            in.h = 0;
            do {
              in.s = seq_info<P, NW>(a, ++in.b);
            } while (in.s.units == 0);
          }
          in_end = units_of(in_S, in.s.units);
          enter();
        }
      }
    }
    ptx::cp_async_commit();
  };
#pragma unroll 1
  for (int i = 0; i < ST - 1; ++i) issue();

  // ---- the computing side, a segment (what the range holds of one item) at a time
  P st;
  int b = b_first, h = h_first, c = c_first, slot = 0;
  Seq sq = s_first;
  int hk = 0, h0 = 0, nh = 0;
  const Out *qrow = nullptr;
  auto ask = [&]() {  // the item's queries
    hk = a.VG == 1 ? h : h / a.VG;
    h0 = hk * a.G + (h - hk * a.VG) * NH;
    nh = min(NH, (hk + 1) * a.G - h0);
    qrow = reinterpret_cast<const Out *>(a.q) + b * a.q_stride + (size_t)h0 * D;
    st.fetch(qrow, nh, lane);
  };
  ask();
#pragma unroll 1
  while (true) {
    const float sc = a.scale_log2 * (a.kscale ? __ldg(a.kscale + hk) : 1.f);
    const float vs = a.vscale ? __ldg(a.vscale + hk) : 1.f;
    st.begin(qrow, nh, sc, lane, qs);
    const int n = units_of(S, sq.units) - c;
    int key = sq.base + (c * NW + w) * P::KEYS;
#pragma unroll 1
    for (int i = 0; i < n; ++i, key += STRIDE) {
      __syncwarp();  // the slot that is filled next has been read
      issue();
      ptx::cp_async_wait<ST - 1>();
      __syncwarp();  // the other lanes' pieces have arrived too
      const uint32_t src = ring + slot * P::STAGE_BYTES;
      if (key >= sq.first && key + P::KEYS <= sq.len)
        st.template step<false>(src, 0, 0, nh, lane, qs);
      else if (key < sq.len)
        st.template step<true>(src, sq.first - key, sq.len - key, nh, lane, qs);
      slot = slot + 1 == ST ? 0 : slot + 1;
    }
    // ---- the segment ends: join the warps, then store the rows or the part.
    // Ranges k_lo - 1 .. k_hi hold parts of it: k_lo is the first whose
    // beginning, floor(k T / W), is not moved to S or lies before it; those
    // that begin in [S + kSnap, E - kSnap] begin inside.
    const long long E = S + sq.units + kItemCost;
    const int k_lo = (int)quotient(min(S + kSnap, E) * W + T - 1, T);
    const int k_hi = (int)quotient((E - kSnap + 1) * W + T - 1, T) - 1;
    const int wf = k_lo - 1, wl = k_hi < k_lo ? wf : k_hi;
    const bool whole = wf == wl;
    const int me = (int)blockIdx.x;
    const size_t part = 2 * me + (me == wf ? 1 : 0);  // the item begins in range wf
    Out *out = reinterpret_cast<Out *>(a.out) + ((size_t)b * a.Hq + h0) * D;
    float *lse = a.lse ? a.lse + (size_t)b * a.Hq + h0 : nullptr;
    const int b_done = b, h_done = h, nh_done = nh;
    S = E;
    const bool last_item = S >= u1;
    c = 0;
    if (!last_item) {  // the next item's queries travel meanwhile
      if (++h == HV) {
        h = 0;
        do {
          sq = seq_info<P, NW>(a, ++b);
        } while (sq.units == 0);
      }
      ask();
    }
#pragma unroll 1
    for (int i = 0; i < P::NCH; i += RC) {
      __syncthreads();  // the exchange is free
      if (i == 0) st.stats(sm + w * NH, sl + w * NH, lane);
      st.template chunks<RC>(i, nh_done, buf + w * NH * CH, lane);
      __syncthreads();
      if (i == 0) {
        if (tid < nh_done) {  // warp factors; with them the sum, and the factor of a whole row
          float top = -INFINITY, sum = 0.f;
          for (int k = 0; k < NW; ++k) top = fmaxf(top, sm[k * NH + tid]);
          for (int k = 0; k < NW; ++k) {
            const float f = rescale(sm[k * NH + tid], top);
            sum += sl[k * NH + tid] * f;
            sf[k * NH + tid] = f;
          }
          if (whole) {
            for (int k = 0; k < NW; ++k) sf[k * NH + tid] *= vs / sum;
            if (lse) lse[tid] = (top + log2f(sum)) * kLn2;
          } else {
            __stcg(a.part_ml + part * NH + tid, make_float2(top, sum));
          }
        }
        __syncthreads();
      }
      for (int e = tid * 2; e < nh_done * CH; e += NT * 2) {
        const int head = e / CH, at = head * D + i * P::CH + e % CH;
        float x = 0.f, y = 0.f;
#pragma unroll
        for (int k = 0; k < NW; ++k) {
          const float2 v = *reinterpret_cast<const float2 *>(buf + k * NH * CH + e);
          const float f = sf[k * NH + head];
          x = fmaf(v.x, f, x), y = fmaf(v.y, f, y);
        }
        if (whole)
          store_out2(out + at, x, y);
        else
          __stcg(reinterpret_cast<float2 *>(a.part_o + part * NH * D + at), make_float2(x, y));
      }
    }
    if (!whole && tid == 0) {
      Part &p = sh_part[me == wf ? 1 : 0];
      p.b = b_done, p.h = h_done, p.wf = wf, p.wl = wl;
    }
    if (last_item) break;
  }
  ptx::cp_async_wait<0>();

  // ---- the join of the items that the range shares with others (kept until
  // the end: it would take registers from the steps).  Parts of more than
  // kGroup ranges are joined in two levels, so that no CTA reads them all: the
  // last of kGroup neighbouring ranges to arrive joins theirs into the first
  // one's part, the last group joins the groups.
  __threadfence();
  __syncthreads();
#pragma unroll 1
  for (int i = 0; i < 2; ++i) {
    const Part p = sh_part[i];
    if (p.b < 0) continue;
    const int me = (int)blockIdx.x, np = p.wl - p.wf + 1;
    const int hk = p.h / a.VG, h0 = hk * a.G + (p.h - hk * a.VG) * NH;
    const int nh = min(NH, (hk + 1) * a.G - h0);
    const float vs = a.vscale ? __ldg(a.vscale + hk) : 1.f;
    Out *out = reinterpret_cast<Out *>(a.out) + ((size_t)p.b * a.Hq + h0) * D;
    float *lse = a.lse ? a.lse + (size_t)p.b * a.Hq + h0 : nullptr;
    const int step = np > kGroup ? kGroup : 1, groups = (np + step - 1) / step;
    bool last = true;
    if (step > 1) {
      const int first = p.wf + (me - p.wf) / kGroup * kGroup, n = min(kGroup, p.wl - first + 1);
      last = arrive(a.group_counters + 2 * first + (first == p.wf ? 1 : 0), n, &sh_last);
      if (last) join_parts<P, NW>(a, first, 1, p.wf, n, nh, sm, sl, vs, nullptr, nullptr);
    }
    if (last && arrive(a.counters + p.wf, groups, &sh_last))
      join_parts<P, NW>(a, p.wf, step, p.wf, groups, nh, sm, sl, vs, out, lse);
  }
}

inline int head_groups(const KVCache &c, int nh) {
  return (c.q_heads / c.kv_heads + nh - 1) / nh;
}
// query heads that one read of a kv head serves
inline int item_heads(const KVCache &c) {
  const int G = c.q_heads / c.kv_heads;
  if (c.cache_dtype == MOE_F32) return G == 1 ? 1 : G <= 4 ? 4 : 8;
  return G <= 8 ? 8 : 16;
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

template <int NH>
cudaError_t launch_fma(const AttnArgs &a, int D, cudaStream_t s) {
  if (D == 64) return launch_p<FmaPath<64, NH>>(a, s);
  if (D == 128) return launch_p<FmaPath<128, NH>>(a, s);
  return launch_p<FmaPath<256, NH>>(a, s);
}

}  // namespace

// The counters come first and in the same place whatever the call, so that
// calls of any sizes may follow one another on one workspace.
constexpr size_t kCounterBytes = kMaxWorkers * sizeof(int32_t);
constexpr size_t kGroupCounterBytes = 2 * kMaxWorkers * sizeof(int32_t);
static_assert(kCounterBytes % 256 == 0 && kGroupCounterBytes % 256 == 0, "alignment");

size_t paged_attention_ws_bytes(const KVCache &c) {
  const int nh = item_heads(c);
  return kCounterBytes + kGroupCounterBytes + align256(2 * kMaxWorkers * nh * sizeof(float2)) +
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
  w += kCounterBytes;
  a.group_counters = reinterpret_cast<int32_t *>(w);
  w += kGroupCounterBytes;
  a.part_ml = reinterpret_cast<float2 *>(w);
  w += align256(2 * kMaxWorkers * nh * sizeof(float2));
  a.part_o = reinterpret_cast<float *>(w);
  if (c.cache_dtype == MOE_F32) {
    if (nh == 1) return launch_fma<1>(a, c.head_dim, s);
    return nh == 4 ? launch_fma<4>(a, c.head_dim, s) : launch_fma<8>(a, c.head_dim, s);
  }
  if (c.cache_dtype == MOE_E4M3)
    return nh == 8 ? launch_mma<true, 1>(a, c.head_dim, s) : launch_mma<true, 2>(a, c.head_dim, s);
  return nh == 8 ? launch_mma<false, 1>(a, c.head_dim, s) : launch_mma<false, 2>(a, c.head_dim, s);
}

}  // namespace moe
