// The routed SwiGLU experts of a few tokens on 4-bit weights with group
// scales (Algorithm 2 steps 4-11 of "MoE 分布式推理基础（基于 vLLM）" §1.2):
//   h[f] = SiLU(x[t] Wg[e]) * (x[t] Wu[e]),  y[t] = sum_k w[f] (h[f] W2[e]),
//   f = t*K + k, e = topk_idx[f], W = (code - 8) * scale(group).
//
// Bound: HBM, by the hit experts' weights (a weight meets the expert's one to
// a few tens of tokens).  What the kernels do about it:
//  - The weights lie in records (moe_prepare_weights_w4): 16 rows x 128
//    codes, 1 KB in the order in which a warp's lanes use them, and the
//    records' scales.  A warp owns one or two tiles of 16 rows (output columns)
//    over the whole reduction, so no sum crosses warps and no barrier is
//    needed after the routing lists; its records stream through a
//    shared-memory queue of its own, which runs on across units, and every
//    lane reads back what it copied.
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

#include "experts_w4.cuh"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int WT = 256, WW = WT / 32;  // threads and warps per CTA
template <int GROUP>
constexpr int record_bytes() {  // codes; 128 / GROUP bf16 scales a row
  return 1024 + 16 * (128 / GROUP) * 2;
}
constexpr int kMaxEntries = kMaxE + kW4MaxPairs / 4;


struct W4Args {
  const uint8_t *rec;        // records (E, C/16, R/128)
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
__device__ __forceinline__ uint32_t word(const uint4 &v, int i) {
  return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// the same from zero sums
__device__ __forceinline__ void mma_bf16_first(float (&c)[4], uint32_t a0, uint32_t a1,
                                               uint32_t a2, uint32_t a3, uint32_t b0,
                                               uint32_t b1) {
  asm(
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
  uint8_t entry_expert[kMaxEntries];
  uint8_t entry_n[kMaxEntries];
  uint16_t entry_first[kMaxEntries];
  int entries;
  uint16_t pair[kW4MaxPairs];
};

// Queue steps of a warp: what two CTAs of an SM can hold.
template <int GROUP, int MT>
constexpr int queue_steps() {
  constexpr int fit = (int)((112 * 1024 - sizeof(Lists)) / (WW * MT * record_bytes<GROUP>()));
  return fit > 8 ? 8 : fit;
}

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

// DOWN false: tiles of 8 gate and 8 up rows (8 columns of h), DOWN true: tiles
// of 16 columns of y; a unit's MT tiles share each operand piece of x or h.
// GROUP: reduction indices per scale.  NTM: column groups of an entry at most.
template <bool DOWN, int GROUP, int MT, int NTM>
__global__ void __launch_bounds__(WT, 2) w4_kernel(const W4Args a) {
  constexpr int NS = 128 / GROUP;   // scales of a row in a record
  constexpr int WPL = 4 / NS;       // a lane's words of a group: WPL t .. of the group's 4 WPL
  constexpr int CR = DOWN ? 4 : 8;  // pairs of a column group
  constexpr int REC = record_bytes<GROUP>();
  constexpr int ST = queue_steps<GROUP, MT>(), STEP_BYTES = MT * REC;
  extern __shared__ __align__(128) uint8_t smem[];
  Lists &L = *reinterpret_cast<Lists *>(smem + WW * ST * STEP_BYTES);
  pdl_enter();
  // the queue's memory is scratch until the lists are ready
  build_lists<CR * NTM>(L, reinterpret_cast<int(*)[kMaxE]>(smem), a);
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int tiles = a.C / 16 / MT;  // units of an entry
  const int NB = a.R / 128;
  const int units = L.entries * tiles;
  const int step = gridDim.x * WW;
  const int u0 = w * gridDim.x + blockIdx.x;  // the first units go to different CTAs
  const uint32_t ring = ptx::smem_u32(smem) + w * (ST * STEP_BYTES);
  const size_t tile_bytes = (size_t)NB * REC;

  // the copying side
  int pu = u0, pb = 0;
  uint32_t put = ring + lane * 16;
  const uint8_t *src = nullptr;
  auto locate = [&]() {
    if (pu >= units) return;
    const int ent = pu / tiles, tile = pu - ent * tiles;
    src = a.rec + ((size_t)L.entry_expert[ent] * (a.C / 16) + tile * MT) * tile_bytes + lane * 16;
  };
  auto issue = [&]() {
    if (pu < units) {
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const uint8_t *from = src + m * tile_bytes;
        cp_async16(put + m * REC, from);
        cp_async16(put + m * REC + 512, from + 512);
        if (lane < 2 * NS) cp_async16(put + m * REC + 1024, from + 1024);
      }
      src += REC;
      put += STEP_BYTES;
      if (put >= ring + ST * STEP_BYTES) put -= ST * STEP_BYTES;
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

  uint32_t get = ring + lane * 16;
#pragma unroll 1
  for (int u = u0; u < units; u += step) {
    const int ent = u / tiles, tile = (u - ent * tiles) * MT;
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
      uint4 xv[NT][4];  // the operand pieces of a step
      auto load_x = [&](int j) {
#pragma unroll
        for (int i = 0; i < NT; ++i) xv[i][j] = __ldg(xr[i] + (j / WPL) * 4 * WPL + j % WPL);
      };
      if constexpr (AHEAD)
#pragma unroll
        for (int j = 0; j < 4; ++j) load_x(j);
#pragma unroll 1
      for (int b = 0; b < NB; ++b) {
        ptx::cp_async_wait<ST - 2>();
        __syncwarp();  // scales are read by lanes that did not copy them
        issue();
        if (!AHEAD || b + 1 < NB) {  // the next pieces, or (not AHEAD) this step's
          if (AHEAD || b > 0)
#pragma unroll
            for (int i = 0; i < NT; ++i) xr[i] += 16;
        }
        uint4 wd[MT][2], sc[MT];
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          wd[m][0] = lds128(get + m * REC);
          wd[m][1] = lds128(get + m * REC + 512);
          const uint32_t at = get - lane * 16 + m * REC + 1024 + g * (4 * NS);
          if constexpr (NS == 4) sc[m] = lds128(at);
          if constexpr (NS == 2) {
            const uint2 v = lds64(at);
            sc[m].x = v.x, sc[m].y = v.y;
          }
          if constexpr (NS == 1) sc[m].x = lds32(at);
        }
        get += STEP_BYTES;
        if (get >= ring + ST * STEP_BYTES) get -= ST * STEP_BYTES;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if constexpr (!AHEAD) load_x(j);
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            const uint32_t wa = word(wd[m][0], j), wb = word(wd[m][1], j);
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
              // this group's scales: rows g and g + 8 are NS scales apart
              constexpr int K1 = NS;
              const int k = j / WPL;
              const uint32_t p0 = word(sc[m], k >> 1), p1 = word(sc[m], (K1 + k) >> 1);
              const float s0 = __uint_as_float(k & 1 ? p0 & 0xffff0000u : p0 << 16);
              const float s1 = __uint_as_float((K1 + k) & 1 ? p1 & 0xffff0000u : p1 << 16);
#pragma unroll
              for (int i = 0; i < NT; ++i) {
                acc[m][i][0] = fmaf(part[m][i][0], s0, acc[m][i][0]);
                acc[m][i][1] = fmaf(part[m][i][1], s0, acc[m][i][1]);
                acc[m][i][2] = fmaf(part[m][i][2], s1, acc[m][i][2]);
                acc[m][i][3] = fmaf(part[m][i][3], s1, acc[m][i][3]);
              }
            }
          }
          if constexpr (AHEAD) load_x(j);
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
            float *y = a.yslot + (size_t)f * a.C + (tile + m) * 16 + g;
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
              const float gate = 4.f * acc[m][i][c], up = 4.f * acc[m][i][2 + c];
              const float h = gate / (1.f + __expf(-gate)) * up;
              const __nv_bfloat16 hi = __float2bfloat16_rn(h);
              const size_t at = (size_t)f * a.I + (tile + m) * 8 + g;
              a.hhi[at] = hi;
              a.hlo[at] = __float2bfloat16_rn(h - __bfloat162float(hi));
            }
          }
        }
      }
    };
    if (NTM == 1 || rows <= CR) {
      pass(std::integral_constant<int, 1>());
    } else if constexpr (NTM >= 2) {
      if (NTM == 2 || rows <= 2 * CR)
        pass(std::integral_constant<int, 2>());
      else if constexpr (NTM == 4)
        pass(std::integral_constant<int, 4>());
    }
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

// Records of w13 (DOWN false) or w2: one thread writes 16 bytes.
template <bool DOWN, int GROUP>
__global__ void __launch_bounds__(256) prepare_w4_kernel(const uint32_t *__restrict__ q,
                                                         const __nv_bfloat16 *__restrict__ s,
                                                         uint8_t *__restrict__ rec,
                                                         long long records, int C, int R) {
  pdl_enter();
  constexpr int NS = 128 / GROUP, WPL = 4 / NS, REC = record_bytes<GROUP>(), PIECES = REC / 16;
  const int NB = R / 128, tiles = C / 16;
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < records * PIECES;
       i += (long long)gridDim.x * 256) {
    const long long r = i / PIECES;
    const int p = (int)(i - r * PIECES);
    const int b = (int)(r % NB), tile = (int)(r / NB % tiles);
    const size_t e = (size_t)(r / NB / tiles);
    auto row = [&](int g, int half) {
      return e * C + (DOWN ? tile * 16 + 8 * half + g : half * (C / 2) + tile * 8 + g);
    };
    uint4 v;
    uint32_t *o = reinterpret_cast<uint32_t *>(&v);
    if (p < 64) {  // plane p / 32, lane p % 32: the lane's four words of its row
      const int g = (p & 31) >> 2, t = p & 3;
      const uint32_t *from = q + row(g, p >> 5) * (R / 8) + b * 16 + t * WPL;
#pragma unroll
      for (int j = 0; j < 4; ++j) o[j] = __ldg(from + (j / WPL) * 4 * WPL + j % WPL);
    } else {  // scales (g, half, NS), eight of them
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int k = (p - 64) * 8 + j, g = k / (2 * NS), half = k / NS % 2;
        reinterpret_cast<__nv_bfloat16 *>(o)[j] = s[row(g, half) * (R / GROUP) + b * NS + k % NS];
      }
    }
    reinterpret_cast<uint4 *>(rec + r * REC)[p] = v;
  }
}

inline size_t align256(size_t v) { return (v + 255) & ~(size_t)255; }

template <bool DOWN, int GROUP, int MT, int NTM>
cudaError_t launch_mt(const W4Args &a, cudaStream_t s) {
  constexpr size_t smem =
      (size_t)WW * queue_steps<GROUP, MT>() * MT * record_bytes<GROUP>() + sizeof(Lists);
  auto kernel = w4_kernel<DOWN, GROUP, MT, NTM>;
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
  const long long tiles = a.C / 16 / MT;
  const long long hit = a.nK < a.E ? a.nK : a.E + a.nK / ((DOWN ? 4 : 8) * NTM);
  const long long full = 2ll * device_sm_count(), most = hit * tiles;
  const int grid = (int)(most < full ? most : full);
  return launch_pdl(kernel, dim3(grid), dim3(WT), smem, s, a);
}

template <bool DOWN, int GROUP>
cudaError_t launch_stage(const W4Args &a, cudaStream_t s) {
  // two tiles a unit halve the operand loads; one tile while that leaves
  // warps without work
  const long long tiles = a.C / 16;
  const long long hit = a.nK < a.E ? a.nK : a.E;
  if (hit * tiles <= 4ll * WW * device_sm_count()) return launch_mt<DOWN, GROUP, 1, 1>(a, s);
  // column groups for nearly every expert's tokens at once (the mean and four
  // deviations of their number); what exceeds them reads the weights again
  const float mean = (float)a.nK / a.E, want = (mean + 4.f * sqrtf(mean)) / (DOWN ? 4 : 8);
  if (want <= 1.f) return launch_mt<DOWN, GROUP, 2, 1>(a, s);
  if (want <= 2.f) return launch_mt<DOWN, GROUP, 2, 2>(a, s);
  return launch_mt<DOWN, GROUP, 2, 4>(a, s);
}

template <int GROUP>
cudaError_t run(const Desc &d, W4Args a, const void *w13_t, const void *w2_t, void *y,
                cudaStream_t s) {
  a.rec = reinterpret_cast<const uint8_t *>(w13_t);
  a.C = 2 * d.I, a.R = d.H;
  cudaError_t e = launch_stage<false, GROUP>(a, s);
  if (e != cudaSuccess) return e;
  a.rec = reinterpret_cast<const uint8_t *>(w2_t);
  a.C = d.H, a.R = d.I;
  e = launch_stage<true, GROUP>(a, s);
  if (e != cudaSuccess) return e;
  const int V = d.H / 4;
  const long long want = ((long long)d.n * V + 255) / 256, cap = 8ll * device_sm_count();
  return launch_pdl(w4_combine_kernel, dim3((int)(want < cap ? want : cap)), dim3(256), 0, s,
                    reinterpret_cast<const float4 *>(a.yslot), a.idx,
                    reinterpret_cast<uint2 *>(y), d.n, d.K, d.E, V);
}

template <int GROUP>
cudaError_t prepare(const Desc &d, int which, const int32_t *q, const void *scales, void *tiled,
                    cudaStream_t s) {
  const int C = which ? d.H : 2 * d.I, R = which ? d.I : d.H;
  const long long records = (long long)d.E * (C / 16) * (R / 128);
  const long long want = (records * (record_bytes<GROUP>() / 16) + 255) / 256;
  const long long cap = 64ll * device_sm_count();
  return launch_pdl(which ? prepare_w4_kernel<true, GROUP> : prepare_w4_kernel<false, GROUP>,
                    dim3((unsigned)(want < cap ? want : cap)), dim3(256), 0, s,
                    reinterpret_cast<const uint32_t *>(q),
                    reinterpret_cast<const __nv_bfloat16 *>(scales),
                    reinterpret_cast<uint8_t *>(tiled), records, C, R);
}

}  // namespace

size_t experts_w4_ws_bytes(const Desc &d) {
  const size_t nK = (size_t)d.nK();
  return 2 * align256(nK * d.I * 2) + align256(nK * d.H * 4);
}

size_t w4_tiled_bytes(const Desc &d, int group, int which) {
  const size_t C = which ? d.H : 2 * d.I, R = which ? d.I : d.H;
  return (size_t)d.E * (C / 16) * (R / 128) * (1024 + 32 * (128 / group));
}

cudaError_t launch_prepare_w4(const Desc &d, int group, int which, const int32_t *q,
                              const void *scales, void *tiled, cudaStream_t s) {
  if (group == 32) return prepare<32>(d, which, q, scales, tiled, s);
  if (group == 64) return prepare<64>(d, which, q, scales, tiled, s);
  return prepare<128>(d, which, q, scales, tiled, s);
}

cudaError_t launch_experts_w4(const Desc &d, int group, const void *x, const int32_t *topk_idx,
                              const float *topk_w, const void *w13_t, const void *w2_t, void *y,
                              void *ws, int32_t *status, cudaStream_t s) {
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
  if (group == 32) return run<32>(d, a, w13_t, w2_t, y, s);
  if (group == 64) return run<64>(d, a, w13_t, w2_t, y, s);
  return run<128>(d, a, w13_t, w2_t, y, s);
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
