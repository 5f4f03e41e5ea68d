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
//    (1-4 column groups a pass).  A code becomes bf16 128 + code by one
//    and-or, minus 136 exactly; the group's scale multiplies the float32
//    partial sums of its group, so weights are never rounded.
//  - Words are handed to lanes so that one instruction's 16 indices lie in
//    one group of 32: step (word 4j + t of a row) takes indices 32j + 8t...;
//    x is read in the same order, 16 bytes a lane, without rearrangement.
#include <type_traits>

#include "kv_cache.cuh"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int WT = 256, WW = WT / 32;  // threads and warps per CTA
constexpr int ST = 8;                  // queue steps per warp
constexpr int STEP_BYTES = 1024 + 128; // codes; scales (8 bytes a row)
constexpr int kMaxEntries = kMaxE + kW4MaxPairs / 32;

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
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
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
// codes 2i and 2i+1 of a word as bf16 (code - 8)
__device__ __forceinline__ uint32_t codes(uint32_t w, int i) {
  const uint32_t v = ((w >> (4 * i)) & 0x000f000fu) | 0x43004300u;  // 128 + code
  const __nv_bfloat162 c = __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&v),
                                   __floats2bfloat162_rn(136.f, 136.f));
  return *reinterpret_cast<const uint32_t *>(&c);
}
__device__ __forceinline__ float bf16_bits(uint32_t b) { return __uint_as_float(b << 16); }

// The routing lists of the call, built by every CTA for itself: pairs sorted
// by expert, in ascending order inside an expert (so that every CTA cuts an
// expert's pairs into the same entries), and the entries (expert, first pair,
// pairs <= 32) to compute.
struct Lists {
  int start[kMaxE];
  int entry_expert[kMaxEntries];
  int entry_first[kMaxEntries];
  int entry_n[kMaxEntries];
  int entries;
  uint16_t pair[kW4MaxPairs];
};

// hist: (WW, kMaxE) scratch.  Each warp takes a contiguous slice of the pairs.
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
      const int m = (c + 31) / 32;
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
        L.entry_first[at] = first + 32 * i;
        L.entry_n[at] = min(32, c - 32 * i);
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

// DOWN false: gate and up rows of 8 columns of h (16 rows), DOWN true: 16
// columns of y.  GROUP: reduction indices per scale.
template <bool DOWN, int GROUP>
__global__ void __launch_bounds__(WT, 2) w4_kernel(const W4Args a) {
  constexpr int NS = 128 / GROUP;  // scales of a row in a step
  extern __shared__ __align__(128) uint8_t smem[];
  Lists &L = *reinterpret_cast<Lists *>(smem + WW * ST * STEP_BYTES);
  pdl_enter();
  build_lists(L, reinterpret_cast<int(*)[kMaxE]>(smem), a);  // the queue starts after it
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int tiles = DOWN ? a.C / 16 : a.I / 8;
  const int NB = a.R / 128;
  const int units = L.entries * tiles;
  const int step = gridDim.x * WW;
  const int u0 = w * gridDim.x + blockIdx.x;  // the first units go to different CTAs
  const uint32_t ring = ptx::smem_u32(smem) + w * (ST * STEP_BYTES);
  const int swz = (g >> 1) & 3;
  const uint32_t put = (uint32_t)(g * 4 + (t ^ swz)) * 16;

  // this lane's rows (g and g + 8) of a unit
  auto row_of = [&](int tile, int half) {
    return DOWN ? tile * 16 + 8 * half + g : half * a.I + tile * 8 + g;
  };
  int pu = u0, pb = 0, pslot = 0;
  const int32_t *qa = nullptr, *qb = nullptr;
  size_t sc = 0;  // first scale of the row whose scales this lane copies
  auto locate = [&]() {
    if (pu >= units) return;
    const int ent = pu / tiles, tile = pu - ent * tiles;
    const size_t e = L.entry_expert[ent];
    const size_t ra = e * a.C + row_of(tile, 0), rb = e * a.C + row_of(tile, 1);
    qa = a.q + ra * (a.R / 8) + t * 4;
    qb = a.q + rb * (a.R / 8) + t * 4;
    sc = (t == 0 ? ra : rb) * (a.R / GROUP);
  };
  auto issue = [&]() {
    if (pu < units) {
      const uint32_t dst = ring + pslot * STEP_BYTES;
      cp_async16(dst + put, qa + pb * 16);
      cp_async16(dst + 512 + put, qb + pb * 16);
      if (t < 2) {
        const uint32_t to = dst + 1024 + (t * 8 + g) * 8;
        // a lone scale comes with its neighbour, from the 4-byte boundary
        if constexpr (NS == 1)
          cp_async_small<4>(to, a.s + ((sc + pb) & ~(size_t)1));
        else
          cp_async_small<2 * NS>(to, a.s + sc + pb * NS);
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
    const size_t e = L.entry_expert[ent];
    const size_t srow[2] = {(e * a.C + row_of(tile, 0)) * (size_t)(a.R / GROUP),
                            (e * a.C + row_of(tile, 1)) * (size_t)(a.R / GROUP)};
    auto pass = [&](auto nt_c) {
      constexpr int NT = decltype(nt_c)::value;
      // the operand row of this lane's column in each group (columns past the
      // last row repeat it; their sums are not stored)
      const uint4 *xr[NT];
      size_t lo_step = 0;
      if (DOWN) lo_step = (a.hlo - a.hhi) / 8;
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        const int f = L.pair[first + min(8 * i + g, rows - 1)];
        const __nv_bfloat16 *p = DOWN ? a.hhi + (size_t)f * a.R : a.x + (size_t)(f / a.K) * a.R;
        xr[i] = reinterpret_cast<const uint4 *>(p) + t;
      }
      float acc[NT][4];
#pragma unroll
      for (int i = 0; i < NT; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
#pragma unroll 1
      for (int b = 0; b < NB; ++b) {
        ptx::cp_async_wait<ST - 2>();
        __syncwarp();
        issue();
        const uint32_t src = ring + slot * STEP_BYTES;
        slot = slot + 1 == ST ? 0 : slot + 1;
        float part[NT][4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (j % (GROUP / 32) == 0)
#pragma unroll
            for (int i = 0; i < NT; ++i)
              part[i][0] = part[i][1] = part[i][2] = part[i][3] = 0.f;
          const uint32_t from = src + (g * 4 + (j ^ swz)) * 16 + t * 4;
          const uint32_t wa = lds32(from), wb = lds32(from + 512);
          const uint32_t a0 = codes(wa, 0), a1 = codes(wb, 0), a2 = codes(wa, 1),
                         a3 = codes(wb, 1);
          const uint32_t c0 = codes(wa, 2), c1 = codes(wb, 2), c2 = codes(wa, 3),
                         c3 = codes(wb, 3);
#pragma unroll
          for (int i = 0; i < NT; ++i) {
            const uint4 v = __ldg(xr[i] + b * 16 + j * 4);
            mma_bf16(part[i], a0, a1, a2, a3, v.x, v.y);
            mma_bf16(part[i], c0, c1, c2, c3, v.z, v.w);
            if (DOWN) {
              const uint4 z = __ldg(xr[i] + lo_step + b * 16 + j * 4);
              mma_bf16(part[i], a0, a1, a2, a3, z.x, z.y);
              mma_bf16(part[i], c0, c1, c2, c3, z.z, z.w);
            }
          }
          if ((j + 1) % (GROUP / 32) == 0) {
            float s0, s1;
            const uint32_t at = src + 1024 + g * 8;
            if constexpr (NS == 1) {
              const uint32_t p0 = lds32(at), p1 = lds32(at + 64);
              s0 = (srow[0] + b) & 1 ? __uint_as_float(p0 & 0xffff0000u) : bf16_bits(p0);
              s1 = (srow[1] + b) & 1 ? __uint_as_float(p1 & 0xffff0000u) : bf16_bits(p1);
            } else {
              const int k = j / (GROUP / 32);  // this group's scale
              const uint32_t p0 = lds32(at + (k >> 1) * 4), p1 = lds32(at + 64 + (k >> 1) * 4);
              s0 = k & 1 ? __uint_as_float(p0 & 0xffff0000u) : bf16_bits(p0);
              s1 = k & 1 ? __uint_as_float(p1 & 0xffff0000u) : bf16_bits(p1);
            }
#pragma unroll
            for (int i = 0; i < NT; ++i) {
              acc[i][0] = fmaf(part[i][0], s0, acc[i][0]);
              acc[i][1] = fmaf(part[i][1], s0, acc[i][1]);
              acc[i][2] = fmaf(part[i][2], s1, acc[i][2]);
              acc[i][3] = fmaf(part[i][3], s1, acc[i][3]);
            }
          }
        }
      }
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int col = 8 * i + 2 * t + c;
          if (col >= rows) continue;
          const int f = L.pair[first + col];
          if (DOWN) {
            const float wt = __ldg(a.w + f);
            float *y = a.yslot + (size_t)f * a.C + tile * 16 + g;
            y[0] = acc[i][c] * wt;
            y[8] = acc[i][2 + c] * wt;
          } else {
            const float gate = acc[i][c], up = acc[i][2 + c];
            const float h = gate / (1.f + expf(-gate)) * up;
            const __nv_bfloat16 hi = __float2bfloat16_rn(h);
            const size_t at = (size_t)f * a.I + tile * 8 + g;
            a.hhi[at] = hi;
            a.hlo[at] = __float2bfloat16_rn(h - __bfloat162float(hi));
          }
        }
    };
    if (rows <= 8)
      pass(std::integral_constant<int, 1>());
    else if (rows <= 16)
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

constexpr size_t kSmem = (size_t)WW * ST * STEP_BYTES + sizeof(Lists);
inline size_t align256(size_t v) { return (v + 255) & ~(size_t)255; }

template <bool DOWN, int GROUP>
cudaError_t launch_stage(const W4Args &a, cudaStream_t s) {
  auto kernel = w4_kernel<DOWN, GROUP>;
  static bool ready[64] = {false};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  bool &r = ready[dev >= 0 && dev < 64 ? dev : 0];
  if (!r) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
    if (e != cudaSuccess) return e;
    r = true;
  }
  // no more warps than the call can have units
  const long long tiles = DOWN ? a.C / 16 : a.I / 8;
  const long long hit = a.nK < a.E ? a.nK : a.E + a.nK / 32;
  const long long full = 2ll * device_sm_count(), most = hit * tiles;
  const int grid = (int)(most < full ? most : full);
  return launch_pdl(kernel, dim3(grid), dim3(WT), kSmem, s, a);
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
