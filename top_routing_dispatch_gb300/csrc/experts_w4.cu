// The routed SwiGLU experts of a few tokens on 4-bit weights with group
// scales (Algorithm 2 steps 4-11 of "MoE 分布式推理基础（基于 vLLM）" §1.2):
//   h[f] = SiLU(x[t] Wg[e]) * (x[t] Wu[e]),  y[t] = sum_k w[f] (h[f] W2[e]),
//   f = t*K + k, e = topk_idx[f], W = (code - 8) * scale(group).
//
// Bound: HBM, by the hit experts' weights (a weight meets the expert's one to
// a few tens of tokens).  What the kernels do about it:
//  - A warp owns 16 weight rows (output columns) over the whole reduction, so
//    no sum crosses warps and no barrier is needed after the routing lists.
//    Its weights stream through a shared-memory queue of its own, 1 KB (16
//    rows x 128 codes) a step, which runs on across units.
//  - The weights are the 16-row operand of m16n8k16, tokens the 8 columns
//    (1-4 column groups a pass).  A pair of codes becomes two bf16 (code - 8)
//    / 4, exactly, by one and(-or) and one multiply-add (see quarter_codes);
//    the group's scale multiplies the float32 partial sums of its group, so
//    weights are never rounded.
//  - h is carried in two bf16 parts, which stand in neighbouring columns of
//    the second product: one bf16 alone would round the result as much as its
//    own rounding to bf16 does again.
//  - Words are handed to lanes so that one instruction's 16 indices lie in one
//    group; x is read in the same order, 16 bytes a lane, as it lies.
#include <type_traits>

#include "kv_cache.cuh"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int WT = 256, WW = WT / 32;  // threads and warps per CTA
constexpr int TILE_BYTES = 1024 + 128;  // codes of 16 rows; their scales (8 bytes a row)
template <int MT>
constexpr int queue_steps() {  // of a warp
  return MT == 1 ? 8 : 5;
}
constexpr int kMaxEntries = kMaxE + kW4MaxPairs / 16;

struct W4Args {
  const int32_t *q;          // (E, C, R/8)
  const __nv_bfloat16 *s;    // (E, C, R/group)
  const int32_t *idx;        // (n K)
  const float *w;            // (n K)
  const __nv_bfloat16 *x;    // (n, H)
  __nv_bfloat16 *hhi, *hlo;  // (n K, I): h = hhi + hlo
  float *yslot;              // (n K, H), weighted
  int nK, K, E, C, R, I;
  int32_t *status;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_small(uint32_t dst, const void *src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(N)
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
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// the same from zero sums
__device__ __forceinline__ void mma_bf16_first(float (&c)[4], uint32_t a0, uint32_t a1,
                                               uint32_t a2, uint32_t a3, uint32_t b0,
                                               uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
// Codes 0,1 (even) or 2,3 of a word (4..7: of the word shifted right by 8) as
// a pair of bf16 (code - 8) / 4.  Bits 0-3 of a half under 0x43 are 128 + code;
// bits 4-7 alone are code * 2^-129, subnormal or of the smallest exponent,
// which a multiply-add takes as it is.
template <bool SECOND>
__device__ __forceinline__ uint32_t quarter_codes(uint32_t w) {
  const uint32_t v = SECOND ? w & 0x00f000f0u : (w & 0x000f000fu) | 0x43004300u;
  const uint32_t mul = SECOND ? 0x7f007f00u : 0x3e803e80u;  // 2^127, 1/4
  const uint32_t add = SECOND ? 0xc000c000u : 0xc208c208u;  // -2, -34
  uint32_t r;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(v), "r"(mul), "r"(add));
  return r;
}

// The routing lists of the call, built by every CTA for itself: pairs sorted
// by expert, in ascending order inside an expert (so that every CTA cuts an
// expert's pairs into the same entries), and the entries (expert, first pair,
// pairs <= ROWS) to compute.
struct Lists {
  int start[kMaxE];
  int entry_expert[kMaxEntries];
  int entry_first[kMaxEntries];
  int entry_n[kMaxEntries];
  int entries;
  uint16_t pair[kW4MaxPairs];
};

// hist: (WW, kMaxE) scratch.  Each warp takes a contiguous slice of the pairs.
template <int ROWS>
__device__ __forceinline__ void build_lists(Lists &L, int (*hist)[kMaxE], const W4Args &a) {
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int slice = (a.nK + 32 * WW - 1) / (32 * WW) * 32;
  const int f0 = w * slice, f1 = min(f0 + slice, a.nK);
  for (int e = lane; e < a.E; e += 32) hist[w][e] = 0;
  __syncwarp();
  bool bad = false;
  for (int f = f0 + lane; f < f1; f += 32) {
    const int e = __ldg(a.idx + f);
    if ((unsigned)e < (unsigned)a.E)
      atomicAdd(&hist[w][e], 1);
    else
      bad = true;
  }
  if (__syncthreads_or(bad) && tid == 0 && blockIdx.x == 0)
    flag_status(a.status, MOE_DEV_BAD_ROUTING);
  for (int e = tid; e < a.E; e += WT) {  // counts; each warp's first rank
    int run = 0;
#pragma unroll
    for (int i = 0; i < WW; ++i) {
      const int h = hist[i][e];
      hist[i][e] = run;
      run += h;
    }
    L.start[e] = run;
  }
  __syncthreads();
  if (w == 0) {  // starts, and the entries in expert order
    int pairs = 0, entries = 0;
    for (int e0 = 0; e0 < a.E; e0 += 32) {
      const int c = e0 + lane < a.E ? L.start[e0 + lane] : 0;
      const int m = (c + ROWS - 1) / ROWS;
      int ic = c, im = m;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, ic, o), z = __shfl_up_sync(0xffffffffu, im, o);
        if (lane >= o) ic += y, im += z;
      }
      const int first = pairs + ic - c;
      if (e0 + lane < a.E) L.start[e0 + lane] = first;
      for (int i = 0; i < m; ++i) {
        const int at = entries + im - m + i;
        L.entry_expert[at] = e0 + lane;
        L.entry_first[at] = first + ROWS * i;
        L.entry_n[at] = min(ROWS, c - ROWS * i);
      }
      pairs += __shfl_sync(0xffffffffu, ic, 31);
      entries += __shfl_sync(0xffffffffu, im, 31);
    }
    if (lane == 0) L.entries = entries;
  }
  __syncthreads();
  for (int fb = f0; fb < f1; fb += 32) {
    const int f = fb + lane;
    int e = f < f1 ? __ldg(a.idx + f) : -1;
    const bool ok = (unsigned)e < (unsigned)a.E;
    if (!ok) e = -1;
    const unsigned peers = __match_any_sync(0xffffffffu, e);
    const int rank = __popc(peers & ((1u << lane) - 1u));
    if (ok) L.pair[L.start[e] + hist[w][e] + rank] = (uint16_t)f;
    __syncwarp();
    if (ok && rank == 0) hist[w][e] += __popc(peers);
    __syncwarp();
  }
  __syncthreads();
}

// DOWN false: gate and up rows of 8 MT columns of h, DOWN true: 16 MT columns
// of y, a unit's MT tiles of 16 rows sharing each operand piece of x or h.
// GROUP: reduction indices per scale.
template <bool DOWN, int GROUP, int MT>
__global__ void __launch_bounds__(WT, 2) w4_kernel(const W4Args a) {
  constexpr int NS = 128 / GROUP;  // scales of a row in a step
  constexpr int WPL = 4 / NS;      // a lane's words of a group: WPL t .. of the group's 4 WPL
  constexpr int CR = DOWN ? 4 : 8;         // pairs of a column group
  constexpr int ROWS = DOWN ? 16 : 32;     // pairs of an entry
  constexpr int ST = queue_steps<MT>(), STEP_BYTES = MT * TILE_BYTES;
  extern __shared__ __align__(128) uint8_t smem[];
  Lists &L = *reinterpret_cast<Lists *>(smem + WW * ST * STEP_BYTES);
  pdl_enter();
  build_lists<ROWS>(L, reinterpret_cast<int(*)[kMaxE]>(smem), a);  // the queue starts after it
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int tiles = (DOWN ? a.C / 16 : a.I / 8) / MT;
  const int NB = a.R / 128;
  const int units = L.entries * tiles;
  const int step = gridDim.x * WW;
  const int u0 = w * gridDim.x + blockIdx.x;  // the first units go to different CTAs
  const uint32_t ring = ptx::smem_u32(smem) + w * (ST * STEP_BYTES);
  // a row's four 16-byte pieces are permuted so that the reads below meet no
  // bank twice
  const int swz = GROUP == 32 ? (g >> 1) & 3 : GROUP == 64 ? g & 2 : 0;
  const uint32_t put = ring + (uint32_t)(g * 4 + (t ^ swz)) * 16;

  // this lane's row of a unit: tile m, lower or upper eight rows
  auto row_of = [&](int tile, int m, int half) {
    return DOWN ? (tile * MT + m) * 16 + 8 * half + g : half * a.I + (tile * MT + m) * 8 + g;
  };
  int pu = u0, pb = 0, pslot = 0;
  const int32_t *src[MT][2];
  // t < 2: the first scale of the rows (lower, upper) whose scales this lane copies
  const __nv_bfloat16 *scale[MT];
  bool odd[MT] = {};  // NS == 1: that scale is the upper half of its 4 bytes
  auto locate = [&]() {
    if (pu >= units) return;
    const int ent = pu / tiles, tile = pu - ent * tiles;
    const size_t e = L.entry_expert[ent];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const size_t ra = e * a.C + row_of(tile, m, 0), rb = e * a.C + row_of(tile, m, 1);
      src[m][0] = a.q + ra * (a.R / 8) + t * 4;
      src[m][1] = a.q + rb * (a.R / 8) + t * 4;
      const size_t at = ((t & 1) ? rb : ra) * (a.R / GROUP);
      scale[m] = a.s + at;
      odd[m] = at & 1;
    }
  };
  auto issue = [&]() {
    if (pu < units) {
      const uint32_t dst = pslot * STEP_BYTES;
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        cp_async16(put + dst + m * TILE_BYTES, src[m][0]);
        cp_async16(put + dst + m * TILE_BYTES + 512, src[m][1]);
        src[m][0] += 16, src[m][1] += 16;
        if (t < 2) {
          const uint32_t to = ring + dst + m * TILE_BYTES + 1024 + (t * 8 + g) * 8;
          // a lone scale comes with its neighbour, from the 4-byte boundary
          if constexpr (NS == 1)
            cp_async_small<4>(to, scale[m] + pb - (odd[m] ^ (pb & 1)));
          else
            cp_async_small<2 * NS>(to, scale[m] + pb * NS);
        }
      }
      pslot = pslot + 1 == ST ? 0 : pslot + 1;
      if (++pb == NB) {
        pb = 0;
        pu += step;
        locate();
      }
    }
    ptx::cp_async_commit();
  };
  locate();
#pragma unroll 1
  for (int i = 0; i < ST - 1; ++i) issue();

  int slot = 0;
#pragma unroll 1
  for (int u = u0; u < units; u += step) {
    const int ent = u / tiles, tile = u - ent * tiles;
    const int rows = L.entry_n[ent], first = L.entry_first[ent];
    auto pass = [&](auto nt_c) {
      constexpr int NT = decltype(nt_c)::value;
      constexpr bool AHEAD = NT <= 2;
      // the operand row of this lane's column in each group: a pair's x, or in
      // even columns the first, in odd the second part of its h (columns past
      // the last pair repeat it; their sums are not stored)
      const uint4 *xr[NT];
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        const int f = L.pair[first + min(CR * i + (DOWN ? g >> 1 : g), rows - 1)];
        const __nv_bfloat16 *p = DOWN ? (g & 1 ? a.hlo : a.hhi) + (size_t)f * a.R
                                      : a.x + (size_t)(f / a.K) * a.R;
        xr[i] = reinterpret_cast<const uint4 *>(p) + t * WPL;
      }
      float acc[MT][NT][4], part[MT][NT][4];
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < NT; ++i)
          acc[m][i][0] = acc[m][i][1] = acc[m][i][2] = acc[m][i][3] = 0.f;
      [[maybe_unused]] bool up[MT][2];
      if constexpr (NS == 1)
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            up[m][h] = ((size_t)L.entry_expert[ent] * a.C + row_of(tile, m, h)) * NB & 1;
      uint4 xv[NT][4];  // the operand pieces of a step
      auto load_x = [&](int b, int j) {
#pragma unroll
        for (int i = 0; i < NT; ++i)
          xv[i][j] = __ldg(xr[i] + b * 16 + (j / WPL) * 4 * WPL + j % WPL);
      };
      if constexpr (AHEAD)
#pragma unroll
        for (int j = 0; j < 4; ++j) load_x(0, j);
#pragma unroll 1
      for (int b = 0; b < NB; ++b) {
        ptx::cp_async_wait<ST - 2>();
        __syncwarp();
        issue();
        const uint32_t from = ring + slot * STEP_BYTES + g * 64;
        const uint32_t sfrom = ring + slot * STEP_BYTES + 1024 + g * 8;
        slot = slot + 1 == ST ? 0 : slot + 1;
        uint2 sc[MT][2];
        uint32_t wd[MT][2][4];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t at = from + m * TILE_BYTES + h * 512;
            if constexpr (GROUP == 128) {
              const uint4 v = lds128(at + t * 16);
              wd[m][h][0] = v.x, wd[m][h][1] = v.y, wd[m][h][2] = v.z, wd[m][h][3] = v.w;
            } else if constexpr (GROUP == 64) {
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const uint2 v = lds64(at + ((2 * k + (t >> 1)) ^ swz) * 16 + (t & 1) * 8);
                wd[m][h][2 * k] = v.x, wd[m][h][2 * k + 1] = v.y;
              }
            } else {
#pragma unroll
              for (int k = 0; k < 4; ++k) wd[m][h][k] = lds32(at + (k ^ swz) * 16 + t * 4);
            }
            if constexpr (NS == 4)
              sc[m][h] = lds64(sfrom + m * TILE_BYTES + h * 64);
            else
              sc[m][h].x = lds32(sfrom + m * TILE_BYTES + h * 64);
            if constexpr (NS == 1) {
              if (!(up[m][h] ^ (b & 1))) sc[m][h].x <<= 16;
            }
          }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if constexpr (!AHEAD) load_x(b, j);
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            const uint32_t wa = wd[m][0][j], wb = wd[m][1][j];
            {
              const uint32_t a0 = quarter_codes<false>(wa), a1 = quarter_codes<false>(wb);
              const uint32_t a2 = quarter_codes<true>(wa), a3 = quarter_codes<true>(wb);
#pragma unroll
              for (int i = 0; i < NT; ++i) {
                if (j % WPL == 0)
                  mma_bf16_first(part[m][i], a0, a1, a2, a3, xv[i][j].x, xv[i][j].y);
                else
                  mma_bf16(part[m][i], a0, a1, a2, a3, xv[i][j].x, xv[i][j].y);
              }
            }
            {
              const uint32_t a0 = quarter_codes<false>(wa >> 8), a1 = quarter_codes<false>(wb >> 8);
              const uint32_t a2 = quarter_codes<true>(wa >> 8), a3 = quarter_codes<true>(wb >> 8);
#pragma unroll
              for (int i = 0; i < NT; ++i)
                mma_bf16(part[m][i], a0, a1, a2, a3, xv[i][j].z, xv[i][j].w);
            }
            if (j % WPL == WPL - 1) {
              const int k = j / WPL;  // this group's scale
              float s[2];
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const uint32_t p = k < 2 ? sc[m][h].x : sc[m][h].y;
                s[h] = __uint_as_float(NS == 1 || (k & 1) ? p & 0xffff0000u : p << 16);
              }
#pragma unroll
              for (int i = 0; i < NT; ++i) {
                acc[m][i][0] = fmaf(part[m][i][0], s[0], acc[m][i][0]);
                acc[m][i][1] = fmaf(part[m][i][1], s[0], acc[m][i][1]);
                acc[m][i][2] = fmaf(part[m][i][2], s[1], acc[m][i][2]);
                acc[m][i][3] = fmaf(part[m][i][3], s[1], acc[m][i][3]);
              }
            }
          }
          if constexpr (AHEAD) load_x(b + 1 < NB ? b + 1 : b, j);
        }
      }
      // the sums are of quarter codes
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        if constexpr (DOWN) {
          const int r = CR * i + t;  // columns 2t and 2t+1: h's two parts
          if (r >= rows) continue;
          const int f = L.pair[first + r];
          const float wt = 4.f * __ldg(a.w + f);
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            float *y = a.yslot + (size_t)f * a.C + (tile * MT + m) * 16 + g;
            y[0] = (acc[m][i][0] + acc[m][i][1]) * wt;
            y[8] = (acc[m][i][2] + acc[m][i][3]) * wt;
          }
        } else {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int r = CR * i + 2 * t + c;
            if (r >= rows) continue;
            const int f = L.pair[first + r];
#pragma unroll
            for (int m = 0; m < MT; ++m) {
              const float gate = 4.f * acc[m][i][c], up_ = 4.f * acc[m][i][2 + c];
              const float h = gate / (1.f + __expf(-gate)) * up_;
              const __nv_bfloat16 hi = __float2bfloat16_rn(h);
              const size_t at = (size_t)f * a.I + (tile * MT + m) * 8 + g;
              a.hhi[at] = hi;
              a.hlo[at] = __float2bfloat16_rn(h - __bfloat162float(hi));
            }
          }
        }
      }
    };
    if (rows <= CR)
      pass(std::integral_constant<int, 1>());
    else if (rows <= 2 * CR)
      pass(std::integral_constant<int, 2>());
    else
      pass(std::integral_constant<int, 4>());
  }
  ptx::cp_async_wait<0>();
}

// y[t] = sum over k of the weighted rows of its valid experts, in slot order
__global__ void __launch_bounds__(256) w4_combine_kernel(const float4 *__restrict__ yslot,
                                                         const int32_t *__restrict__ idx,
                                                         uint2 *__restrict__ y, int n, int K,
                                                         int E, int V) {
  pdl_enter();
  const long long total = (long long)n * V;
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < total;
       i += (long long)gridDim.x * 256) {
    const int t = (int)(i / V), v = (int)(i - (long long)t * V);
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k = 0; k < K; ++k) {
      if ((unsigned)__ldg(idx + t * K + k) >= (unsigned)E) continue;
      const float4 r = __ldg(yslot + (size_t)(t * K + k) * V + v);
      s.x += r.x, s.y += r.y, s.z += r.z, s.w += r.w;
    }
    uint2 o;
    __nv_bfloat162 *h = reinterpret_cast<__nv_bfloat162 *>(&o);
    h[0] = __floats2bfloat162_rn(s.x, s.y);
    h[1] = __floats2bfloat162_rn(s.z, s.w);
    y[i] = o;
  }
}

// One warp quantises the groups of 32 neighbouring columns c of one expert:
// lane = column, so the row-major weights are read along rows.
template <int GROUP>
__global__ void __launch_bounds__(256) quantize_w4_kernel(const __nv_bfloat16 *__restrict__ w,
                                                          uint32_t *__restrict__ q,
                                                          __nv_bfloat16 *__restrict__ s,
                                                          long long tasks, int R, int C) {
  pdl_enter();
  const int lane = threadIdx.x & 31;
  const int groups = R / GROUP, cb = C / 32;
  for (long long i = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); i < tasks;
       i += (long long)gridDim.x * 8) {
    const int c = (int)(i % cb) * 32 + lane;
    const long long rest = i / cb;
    const int gr = (int)(rest % groups);
    const long long e = rest / groups;
    const __nv_bfloat16 *src = w + ((size_t)e * R + (size_t)gr * GROUP) * C + c;
    float top = 0.f;
#pragma unroll 8
    for (int r = 0; r < GROUP; ++r) top = fmaxf(top, fabsf(__bfloat162float(src[(size_t)r * C])));
    const __nv_bfloat16 sb = __float2bfloat16_rn(top / 7.f);
    const float sc = __bfloat162float(sb);
    s[((size_t)e * C + c) * groups + gr] = sb;
    uint32_t *dst = q + ((size_t)e * C + c) * (R / 8) + (size_t)gr * (GROUP / 8);
    for (int o = 0; o < GROUP / 8; ++o) {
      uint32_t word = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float v = __bfloat162float(src[(size_t)(8 * o + j) * C]);
        const float k = sc > 0.f ? rintf(v / sc) + 8.f : 8.f;
        word |= (uint32_t)fminf(fmaxf(k, 0.f), 15.f) << (4 * (j / 2) + 16 * (j % 2));
      }
      dst[o] = word;
    }
  }
}

inline size_t align256(size_t v) { return (v + 255) & ~(size_t)255; }

template <bool DOWN, int GROUP, int MT>
cudaError_t launch_mt(const W4Args &a, cudaStream_t s) {
  constexpr size_t smem = (size_t)WW * queue_steps<MT>() * MT * TILE_BYTES + sizeof(Lists);
  auto kernel = w4_kernel<DOWN, GROUP, MT>;
  static bool ready[64] = {false};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  bool &r = ready[dev >= 0 && dev < 64 ? dev : 0];
  if (!r) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    r = true;
  }
  // no more warps than the call can have units
  const long long tiles = (DOWN ? a.C / 16 : a.I / 8) / MT;
  const long long hit = a.nK < a.E ? a.nK : a.E + a.nK / 16;
  const long long full = 2ll * device_sm_count(), most = hit * tiles;
  const int grid = (int)(most < full ? most : full);
  return launch_pdl(kernel, dim3(grid), dim3(WT), smem, s, a);
}

template <bool DOWN, int GROUP>
cudaError_t launch_stage(const W4Args &a, cudaStream_t s) {
  // two tiles a unit halve the operand loads; one tile while that leaves
  // warps without work
  const long long tiles = DOWN ? a.C / 16 : a.I / 8;
  const long long hit = a.nK < a.E ? a.nK : a.E;
  if (hit * tiles <= 4ll * WW * device_sm_count()) return launch_mt<DOWN, GROUP, 1>(a, s);
  return launch_mt<DOWN, GROUP, 2>(a, s);
}

template <int GROUP>
cudaError_t run(const Desc &d, W4Args a, const int32_t *w13_q, const void *w13_s,
                const int32_t *w2_q, const void *w2_s, void *y, cudaStream_t s) {
  a.q = w13_q, a.s = reinterpret_cast<const __nv_bfloat16 *>(w13_s);
  a.C = 2 * d.I, a.R = d.H;
  cudaError_t e = launch_stage<false, GROUP>(a, s);
  if (e != cudaSuccess) return e;
  a.q = w2_q, a.s = reinterpret_cast<const __nv_bfloat16 *>(w2_s);
  a.C = d.H, a.R = d.I;
  e = launch_stage<true, GROUP>(a, s);
  if (e != cudaSuccess) return e;
  const int V = d.H / 4;
  const long long want = ((long long)d.n * V + 255) / 256, cap = 8ll * device_sm_count();
  return launch_pdl(w4_combine_kernel, dim3((int)(want < cap ? want : cap)), dim3(256), 0, s,
                    reinterpret_cast<const float4 *>(a.yslot), a.idx,
                    reinterpret_cast<uint2 *>(y), d.n, d.K, d.E, V);
}

}  // namespace

size_t experts_w4_ws_bytes(const Desc &d) {
  const size_t nK = (size_t)d.nK();
  return 2 * align256(nK * d.I * 2) + align256(nK * d.H * 4);
}

cudaError_t launch_experts_w4(const Desc &d, int group, const void *x, const int32_t *topk_idx,
                              const float *topk_w, const int32_t *w13_q, const void *w13_s,
                              const int32_t *w2_q, const void *w2_s, void *y, void *ws,
                              int32_t *status, cudaStream_t s) {
  if (d.n == 0) return cudaSuccess;
  W4Args a = {};
  a.idx = topk_idx, a.w = topk_w;
  a.x = reinterpret_cast<const __nv_bfloat16 *>(x);
  uint8_t *p = reinterpret_cast<uint8_t *>(ws);
  const size_t hb = align256((size_t)d.nK() * d.I * 2);
  a.hhi = reinterpret_cast<__nv_bfloat16 *>(p);
  a.hlo = reinterpret_cast<__nv_bfloat16 *>(p + hb);
  a.yslot = reinterpret_cast<float *>(p + 2 * hb);
  a.nK = (int)d.nK(), a.K = d.K, a.E = d.E, a.I = d.I;
  a.status = status;
  if (group == 32) return run<32>(d, a, w13_q, w13_s, w2_q, w2_s, y, s);
  if (group == 64) return run<64>(d, a, w13_q, w13_s, w2_q, w2_s, y, s);
  return run<128>(d, a, w13_q, w13_s, w2_q, w2_s, y, s);
}

cudaError_t launch_quantize_w4(int E, int rows, int cols, int group, const void *w, int32_t *q,
                               void *scales, cudaStream_t s) {
  const long long tasks = (long long)E * (rows / group) * (cols / 32);
  const long long want = (tasks + 7) / 8, cap = 16ll * device_sm_count();
  const dim3 grid((int)(want < cap ? want : cap));
  auto kernel = group == 32 ? quantize_w4_kernel<32>
                : group == 64 ? quantize_w4_kernel<64> : quantize_w4_kernel<128>;
  return launch_pdl(kernel, grid, dim3(256), 0, s, reinterpret_cast<const __nv_bfloat16 *>(w),
                    reinterpret_cast<uint32_t *>(q), reinterpret_cast<__nv_bfloat16 *>(scales),
                    tasks, rows, cols);
}

}  // namespace moe
