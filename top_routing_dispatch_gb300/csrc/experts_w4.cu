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
//    over the whole reduction, so no sum crosses warps (except where two share
//    a reduction for want of work); its records stream through a queue in
//    shared memory, which runs on across units, and every lane reads back the
//    codes that it copied.
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
//
// Measured, both products and the sum over experts (hit experts' weights read
// once, of a copy rate of 6.7 TB/s): H = 7168, I = 2048, E = 256, K = 8: 1 token
// 47 us (57 %), 3 tokens 110 us (72 %), 61 tokens in groups of 32 885 us (91 %);
// H = 2048, I = 1024, E = 64, K = 8: 1 token 14 us (28 %), 120 tokens 90 us (35 %).
// The conversion of codes holds the kernels at few tokens an expert (3 tokens
// without it: 97 of then 124 us), at 15 tokens matrix instructions and operand
// reads (matrix pipe 40 % and issue 50 % busy, 12 warps an SM).
#include <cmath>
#include <type_traits>

#include "experts_w4.cuh"
#include "ptx.cuh"

namespace moe {
namespace {

template <int GROUP>
constexpr int record_bytes() {  // codes; 128 / GROUP bf16 scales a row
  return 1024 + 16 * (128 / GROUP) * 2;
}


struct W4Args {
  const uint8_t *rec;        // records (E, C/16, R/128)
  const int32_t *idx;        // (n K)
  const float *w;            // (n K)
  const __nv_bfloat16 *x;    // (n, H)
  __nv_bfloat16 *hhi, *hlo;  // (n K, I): h = hhi + hlo
  float *yslot;              // (n K, H), weighted
  __nv_bfloat16 *y;          // (n, H)
  int nK, K, E, C, R, H, I;
  unsigned k_inv;            // f / K = f * k_inv >> 16 (f < 4096, K <= 16: checked for all)
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

// The routing lists of the call, built by every CTA for itself in shared
// memory: pairs sorted by expert, in ascending order inside an expert (so that
// every CTA cuts an expert's pairs into the same entries), and the entries
// (expert, first pair, pairs <= ROWS) to compute.
struct Lists {
  uint32_t *entry;    // expert | pairs - 1 << 8 | first << 16
  uint16_t *pair;     // (nK)
  int entries;
  __device__ __forceinline__ int expert(int i) const { return entry[i] & 0xff; }
  __device__ __forceinline__ int count(int i) const { return (entry[i] >> 8 & 0xff) + 1; }
  __device__ __forceinline__ int first(int i) const { return entry[i] >> 16; }
};

__host__ __device__ inline int max_entries(int nK, int E, int rows) {
  return (nK < E ? nK : E) + nK / rows;
}
__host__ __device__ inline int lists_bytes(int nK, int E, int rows) {
  return (4 * max_entries(nK, E, rows) + 2 * nK + 15) & ~15;
}

// mem: lists_bytes; scratch: build_bytes.  Each warp ranks a contiguous slice of
// the pairs, 32 at a time; a thread then sums up the warps' counts of two
// neighbouring experts and one scan gives their places.  The chain of
// barriers and loads is what this costs, and every CTA waits for it: about 7500
// cycles at 120 tokens, E = 64, K = 8 and 3000 at 3 tokens, E = 256 (a pass of
// counts, a scan by one warp and a second pass for the ranks took 11000 and
// 7700).
constexpr int MW = 4;  // warps of a CTA
static_assert(kMaxE <= 256 && kMaxE <= 2 * MW * 32, "8 bits, two experts a thread");
constexpr int build_bytes(int nK) { return 4 * (MW * kMaxE + nK); }

template <int ROWS>
__device__ __forceinline__ Lists build_lists(uint8_t *mem, uint8_t *scratch, const W4Args &a) {
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  __shared__ uint32_t sh_warp[MW];
  Lists L;
  L.entry = reinterpret_cast<uint32_t *>(mem);
  L.pair = reinterpret_cast<uint16_t *>(L.entry + max_entries(a.nK, a.E, ROWS));
  // (warps, kMaxE): pairs of an expert in a warp's slice, then the slice's place
  int *hist = reinterpret_cast<int *>(scratch);
  int *mine = hist + w * kMaxE;
  uint32_t *rank = reinterpret_cast<uint32_t *>(hist + MW * kMaxE);  // (nK): expert | rank << 16
  const int slice = (a.nK + MW * 32 - 1) / (MW * 32) * 32;
  const int f0 = w * slice, f1 = min(f0 + slice, a.nK);
#pragma unroll
  for (int e = 0; e < kMaxE; e += 128)
    *reinterpret_cast<int4 *>(mine + e + 4 * lane) = make_int4(0, 0, 0, 0);
  bool bad = false;
#pragma unroll 8
  for (int f = f0 + lane; f < f1; f += 32) {
    const uint32_t e = (uint32_t)__ldg(a.idx + f);
    bad |= e >= (uint32_t)a.E;
    rank[f] = e < (uint32_t)a.E ? e : 0xffffu;
  }
  __syncwarp();
#pragma unroll 2
  for (int f = f0 + lane; f - lane < f1; f += 32) {
    const uint32_t e = f < f1 ? rank[f] : 0xffffu;
    const bool ok = e != 0xffffu;
    // the lanes with the same expert, by the bits of its number: a ballot a
    // bit, independent of each other (the instruction that compares all lanes
    // at once takes several hundred cycles when most differ)
    unsigned peers = __ballot_sync(0xffffffffu, ok);
#pragma unroll
    for (int b = 0; b < 8; ++b) {
      const unsigned m = __ballot_sync(0xffffffffu, e >> b & 1u);
      peers &= e >> b & 1u ? m : ~m;
    }
    const unsigned below = peers & ((1u << lane) - 1u);
    const int at = ok ? mine[e] : 0;
    if (ok) rank[f] = e | (uint32_t)(at + __popc(below)) << 16;
    __syncwarp();  // every peer has read the count
    if (ok && below == 0) mine[e] = at + __popc(peers);
    __syncwarp();
  }
  if (__syncthreads_or(bad) && tid == 0 && blockIdx.x == 0)
    flag_status(a.status, MOE_DEV_BAD_ROUTING);
  // experts 2 tid and 2 tid + 1
  int2 run = make_int2(0, 0), at[MW];
#pragma unroll
  for (int i = 0; i < MW; ++i) {
    at[i] = run;
    const int2 h = *reinterpret_cast<const int2 *>(hist + i * kMaxE + 2 * tid);
    run.x += h.x, run.y += h.y;
  }
  // pairs and, above them, entries
  const uint32_t m0 = (run.x + ROWS - 1) / ROWS, m1 = (run.y + ROWS - 1) / ROWS;
  const uint32_t own = (uint32_t)(run.x + run.y) | (m0 + m1) << 16;
  uint32_t inc = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  if (lane == 31) sh_warp[w] = inc;
  __syncthreads();
  uint32_t before = inc - own, total = 0;
#pragma unroll
  for (int i = 0; i < MW; ++i) {
    if (i < w) before += sh_warp[i];
    total += sh_warp[i];
  }
  const uint32_t first = before & 0xffffu;
#pragma unroll
  for (int i = 0; i < MW; ++i)
    *reinterpret_cast<int2 *>(hist + i * kMaxE + 2 * tid) =
        make_int2(first + at[i].x, first + run.x + at[i].y);
  uint32_t *entry = L.entry + (before >> 16);
#pragma unroll 1
  for (uint32_t i = 0; i < m0 + m1; ++i) {
    const uint32_t second = i >= m0, k = (second ? i - m0 : i) * ROWS;
    entry[i] = (2 * tid + second) | (min((uint32_t)ROWS, (second ? run.y : run.x) - k) - 1) << 8 |
               (first + (second ? run.x : 0) + k) << 16;
  }
  __syncthreads();
#pragma unroll 4
  for (int f = f0 + lane; f < f1; f += 32) {
    const uint32_t r = rank[f], e = r & 0xffffu;
    if (e != 0xffffu) L.pair[mine[e] + (r >> 16)] = (uint16_t)f;
  }
  L.entries = total >> 16;
  __syncthreads();
  return L;
}

// acc += one step (128 indices) of MT tiles: codes wd (two planes), scales sc;
// x(i, j): the operand piece of column group i for words j.
template <int GROUP, int MT, int NT, class X>
__device__ __forceinline__ void step_product(const uint4 (&wd)[MT][2], const uint4 (&sc)[MT], X x,
                                             float (&acc)[MT][NT][4]) {
  constexpr int NS = 128 / GROUP, WPL = 4 / NS;
  float part[MT][NT][4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint4 xv[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) xv[i] = x(i, j);
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const uint32_t wa = word(wd[m][0], j), wb = word(wd[m][1], j);
      {
        const uint32_t a0 = quarter_codes<false>(wa), a1 = quarter_codes<false>(wb);
        const uint32_t a2 = quarter_codes<true>(wa), a3 = quarter_codes<true>(wb);
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          if (j % WPL == 0)
            mma_bf16_first(part[m][i], a0, a1, a2, a3, xv[i].x, xv[i].y);
          else
            mma_bf16(part[m][i], a0, a1, a2, a3, xv[i].x, xv[i].y);
        }
      }
      {
        const uint32_t a0 = quarter_codes<false>(wa >> 8), a1 = quarter_codes<false>(wb >> 8);
        const uint32_t a2 = quarter_codes<true>(wa >> 8), a3 = quarter_codes<true>(wb >> 8);
#pragma unroll
        for (int i = 0; i < NT; ++i)
          mma_bf16(part[m][i], a0, a1, a2, a3, xv[i].z, xv[i].w);
      }
      if (j % WPL == WPL - 1) {
        // this group's scales: rows g and g + 8 are NS scales apart
        const int k = j / WPL;
        const uint32_t p0 = word(sc[m], k >> 1), p1 = word(sc[m], (NS + k) >> 1);
        const float s0 = __uint_as_float(k & 1 ? p0 & 0xffff0000u : p0 << 16);
        const float s1 = __uint_as_float((NS + k) & 1 ? p1 & 0xffff0000u : p1 << 16);
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          acc[m][i][0] = fmaf(part[m][i][0], s0, acc[m][i][0]);
          acc[m][i][1] = fmaf(part[m][i][1], s0, acc[m][i][1]);
          acc[m][i][2] = fmaf(part[m][i][2], s1, acc[m][i][2]);
          acc[m][i][3] = fmaf(part[m][i][3], s1, acc[m][i][3]);
        }
      }
    }
  }
}

// The scales of a record for a lane's two rows.
template <int GROUP>
__device__ __forceinline__ uint4 load_scales(uint32_t at) {
  constexpr int NS = 128 / GROUP;
  uint4 sc = make_uint4(0, 0, 0, 0);
  if constexpr (NS == 4) sc = lds128(at);
  if constexpr (NS == 2) {
    const uint2 v = lds64(at);
    sc.x = v.x, sc.y = v.y;
  }
  if constexpr (NS == 1) sc.x = lds32(at);
  return sc;
}

__device__ __forceinline__ size_t wide(unsigned a, unsigned b) {
  return (unsigned long long)a * b;
}

// h of pair f in column c from the sums (of quarter codes) of gate and up
__device__ __forceinline__ void store_h(const W4Args &a, int f, int c, float gate, float up) {
  gate *= 4.f, up *= 4.f;
  // SiLU by the full-precision exp of a number that is not positive: the fast
  // one's error grows with the gate, and the fast division (2 ulp) wants a
  // divisor below 2^126, here 1 to 2
  const float e = expf(-fabsf(gate));
  const float h = __fdividef(gate < 0.f ? gate * e : gate, 1.f + e) * up;
  // a finite h beyond bf16's largest value has that as its first part; an
  // infinite one or NaN has no second part (inf - inf is NaN)
  constexpr float kTop = 0x1.fep127f;
  const bool finite = fabsf(h) < INFINITY;
  const __nv_bfloat16 hi = __float2bfloat16_rn(finite ? fminf(fmaxf(h, -kTop), kTop) : h);
  const size_t at = wide((unsigned)f, (unsigned)a.I) + c;
  a.hhi[at] = hi;
  a.hlo[at] = __float2bfloat16_rn(finite ? h - __bfloat162float(hi) : 0.f);
}

// Stores the sums (of quarter codes) of tile `tile` for an entry's pairs.
template <bool DOWN, int NT>
__device__ __forceinline__ void store_tile(const W4Args &a, const Lists &L, const float (&acc)[NT][4],
                                           int tile, int rows, int first, int lane) {
  constexpr int CR = DOWN ? 4 : 8;
  const int g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    if constexpr (DOWN) {
      const int r = CR * i + t;  // columns 2t and 2t+1: h's two parts
      if (r >= rows) continue;
      const int f = L.pair[first + r];
      const float wt = 4.f * __ldg(a.w + f);
      float *y = a.yslot + wide((unsigned)f, (unsigned)a.C) + tile * 16 + g;
      y[0] = (acc[i][0] + acc[i][1]) * wt;
      y[8] = (acc[i][2] + acc[i][3]) * wt;
    } else {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int r = CR * i + 2 * t + c;
        if (r >= rows) continue;
        store_h(a, L.pair[first + r], tile * 8 + g, acc[i][c], acc[i][2 + c]);
      }
    }
  }
}

// Queue steps: what `ctas` CTAs of an SM can hold of `step` bytes beside 4 KB
// of lists each (a call with longer lists gets fewer CTAs).
constexpr int queue_steps(int ctas, int step) {
  const int fit = ((227 / ctas - 1) * 1024 - 4 * 1024) / step;
  return fit > 8 ? 8 : fit;
}

// Few tokens: at most 32 pairs, each an entry of its own (an expert that two of
// them share is read twice, mostly from L2); every warp works by itself on
// (tile, pair) units.  DOWN false: the units of all pairs are dealt out over
// the warps of the grid.  DOWN true: a CTA's warps share out the pairs of a
// tile and the CTA then adds each token's rows in slot order, so that no
// separate combine is needed.  KS = 2: two warps share a unit's reduction, the
// first half's sum plus the second's, for calls that would leave most
// warps without work (the codes' conversion keeps an SM's few warps busier
// than the memory).
constexpr int kFewPairs = 32;
__device__ __forceinline__ void team_sync(int team) {  // the two warps of a team
  asm volatile("bar.sync %0, 64;" ::"r"(team + 1) : "memory");
}
template <bool DOWN, int GROUP, int KS>
struct Few {
  static constexpr int WW = DOWN ? 8 * KS : 8, WT = WW * 32;  // warps and threads of a CTA
  static constexpr int CTAS = 16 / WW;                        // of an SM
  static constexpr int REC = record_bytes<GROUP>(), ST = 8 / KS;
  static constexpr int STEP = REC + 512;  // and 128 values of x, or of h's two parts
  static constexpr int QUEUE = WW * ST * STEP;
};

template <bool DOWN, int GROUP, int KS>
__global__ void __launch_bounds__(Few<DOWN, GROUP, KS>::WT, Few<DOWN, GROUP, KS>::CTAS)
    w4_few_kernel(const W4Args a) {
  using F = Few<DOWN, GROUP, KS>;
  constexpr int WW = F::WW, WT = F::WT;
  constexpr int WPL = GROUP / 32;   // a lane's words of a group: WPL t .. of the group's 4 WPL
  constexpr int REC = F::REC, STEP = F::STEP, ST = F::ST, NS = 128 / GROUP;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint8_t sh_pair[WW][kFewPairs];    // the valid pairs, each warp's own copy
  __shared__ uint8_t sh_expert[WW][kFewPairs];
  __shared__ float sh_y[KS][DOWN ? kFewPairs : WW / KS][16];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  if constexpr (!DOWN) pdl_enter();
  const int e = lane < a.nK ? __ldg(a.idx + lane) : -1;
  const bool ok = (unsigned)e < (unsigned)a.E;
  const unsigned valid = __ballot_sync(0xffffffffu, ok);
  if (ok) {
    const int at = __popc(valid & ((1u << lane) - 1u));
    sh_pair[w][at] = (uint8_t)lane;
    sh_expert[w][at] = (uint8_t)e;
  }
  if (!DOWN && lane < a.nK && !ok && w == 0 && blockIdx.x == 0)
    flag_status(a.status, MOE_DEV_BAD_ROUTING);
  __syncwarp();
  const int pairs = __popc(valid);
  const int tiles = a.C / 16, NB = a.R / 128;
  const uint32_t ring = ptx::smem_u32(smem) + w * (ST * STEP), ring_end = ring + ST * STEP;
  const size_t tile_bytes = (size_t)NB * REC;

  // blocks [b_first, b_first + b_count) of the reduction are this warp's
  const int half = w % KS, team = w / KS;
  constexpr int TEAMS = WW / KS;
  const int b_first = half * NB / KS, b_count = (half + 1) * NB / KS - b_first;

  // a team's units in order: DOWN: pairs team, team + TEAMS, ... of the CTA's
  // tiles; else: every (teams of the grid)-th unit, a pair's tiles next to each
  // other
  struct Unit {
    int tile, pair;  // pair: place in sh_pair
  };
  const int step = gridDim.x * TEAMS;
  auto first_unit = [&]() {
    if constexpr (DOWN) return Unit{(int)blockIdx.x, team};
    const int u = team * gridDim.x + blockIdx.x;
    return Unit{u % tiles, u / tiles};
  };
  auto next_unit = [&](Unit &u) {
    if constexpr (DOWN) {
      u.pair += TEAMS;
      if (u.pair >= pairs) u.pair = team, u.tile += gridDim.x;
    } else {
      u.tile += step;
      if (u.tile >= tiles) u.pair += u.tile / tiles, u.tile %= tiles;
    }
  };
  auto more = [&](const Unit &u) { return u.pair < pairs && u.tile < tiles; };

  // the copying side: a record, and its 128 operand values (lanes 0-15: x or
  // h's first part, lanes 16-31: h's second part)
  Unit in = first_unit();
  int pb = b_count;  // steps of it to go
  uint32_t put = ring + lane * 16;
  const uint8_t *src = nullptr;
  const uint4 *xsrc = nullptr;
  auto locate = [&]() {
    if (!more(in)) return;
    src = a.rec + ((size_t)sh_expert[w][in.pair] * tiles + in.tile) * tile_bytes +
          (size_t)b_first * REC + lane * 16;
    const unsigned f = sh_pair[w][in.pair];
    const __nv_bfloat16 *p = DOWN ? (lane & 16 ? a.hlo : a.hhi) + wide(f, (unsigned)a.R)
                                  : a.x + wide(f * a.k_inv >> 16, (unsigned)a.R);
    xsrc = reinterpret_cast<const uint4 *>(p) + b_first * 16 + (lane & 15);
  };
  auto copy_weights = [&]() {
    cp_async16(put, src);
    cp_async16(put + 512, src + 512);
    if (lane < 2 * NS) cp_async16(put + 1024, src + 1024);
    src += REC;
  };
  auto copy_operand = [&]() {
    if (DOWN || lane < 16) cp_async16(put + REC, xsrc);
    xsrc += 16;
  };
  auto advance = [&]() {
    put += STEP;
    if (put >= ring_end) put -= ST * STEP;
    if (--pb == 0) {
      pb = b_count;
      next_unit(in);
      locate();
    }
  };
  locate();
  if constexpr (DOWN) {  // weights are on their way before h is there
#pragma unroll 1
    for (int i = 0; i < ST - 1; ++i)
      if (more(in)) {
        copy_weights();
        advance();
      }
    pdl_wait();
    pdl_launch();
    in = first_unit(), pb = b_count, put = ring + lane * 16;
    locate();
  }
#pragma unroll 1
  for (int i = 0; i < ST - 1; ++i) {
    if (more(in)) {
      if constexpr (DOWN)
        src += REC;
      else
        copy_weights();
      copy_operand();
      advance();
    }
    ptx::cp_async_commit();
  }

  uint32_t get = ring;
  // every column is the pair's x, or in turn the first and second part of h
  const uint32_t xget = REC + (DOWN ? (g & 1) * 256 : 0) + t * WPL * 16;
  auto product = [&](float (&acc)[1][1][4]) {
    acc[0][0][0] = acc[0][0][1] = acc[0][0][2] = acc[0][0][3] = 0.f;
#pragma unroll 1
    for (int b = b_count; b > 0; --b) {
      ptx::cp_async_wait<ST - 2>();
      __syncwarp();  // lanes read what others copied
      if (more(in)) {
        copy_weights();
        copy_operand();
        advance();
      }
      ptx::cp_async_commit();
      const uint4 wd[1][2] = {{lds128(get + lane * 16), lds128(get + 512 + lane * 16)}};
      const uint4 sc[1] = {load_scales<GROUP>(get + 1024 + g * (4 * NS))};
      const uint32_t x = get + xget;
      get += STEP;
      if (get == ring_end) get = ring;
      step_product<GROUP, 1, 1>(
          wd, sc,
          [&](int, int j) { return lds128(x + ((j / WPL) * 4 * WPL + j % WPL) * 16); }, acc);
    }
  };
  float acc[1][1][4];
  if constexpr (DOWN) {
    const int V = a.nK / a.K;  // tokens
    for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
      if (lane < 16)
        for (int f = w; f < a.nK; f += WW)
          if (!(valid >> f & 1u))
#pragma unroll
            for (int k = 0; k < KS; ++k) sh_y[k][f][lane] = 0.f;
      for (int p = team; p < pairs; p += TEAMS) {
        product(acc);
        if (t == 0) {
          const int f = sh_pair[w][p];
          sh_y[half][f][g] = acc[0][0][0] + acc[0][0][1];
          sh_y[half][f][g + 8] = acc[0][0][2] + acc[0][0][3];
        }
      }
      __syncthreads();
      for (int i = threadIdx.x; i < V * 16; i += WT) {
        const int tok = i >> 4, c = i & 15;
        float y = 0.f;
        for (int k = 0; k < a.K; ++k) {
          const int f = tok * a.K + k;
          float z = sh_y[0][f][c];
          if constexpr (KS == 2) z += sh_y[1][f][c];
          if (valid >> f & 1u) y += z * (4.f * __ldg(a.w + f));  // the sums are of quarter codes
        }
        a.y[(size_t)tok * a.C + tile * 16 + c] = __float2bfloat16_rn(y);
      }
      __syncthreads();
    }
  } else {
    for (Unit u = first_unit(); more(u); next_unit(u)) {
      product(acc);
      if constexpr (KS == 2) {  // the second half's sums to the first half's warp
        if (half == 1 && t == 0)
          *reinterpret_cast<float2 *>(&sh_y[0][team][2 * g]) =
              make_float2(acc[0][0][0], acc[0][0][2]);
        team_sync(team);
        if (half == 0 && t == 0) {
          const float2 v = *reinterpret_cast<const float2 *>(&sh_y[0][team][2 * g]);
          acc[0][0][0] += v.x, acc[0][0][2] += v.y;
        }
        team_sync(team);
      }
      if (half == 0 && t == 0)
        store_h(a, sh_pair[w][u.pair], u.tile * 8 + g, acc[0][0][0], acc[0][0][2]);
    }
  }
  ptx::cp_async_wait<0>();
}

// More tokens: up to NTM column groups an entry.  The four warps of a CTA work
// on eight tiles of one entry and share its operand rows, which travel in the
// same queue as the weights: each step holds the 8 KB of codes of the eight
// tiles and 128 indices of up to 8 NTM operand rows, pieces permuted so that
// the reads meet no bank twice.
constexpr int MT_MANY = 2;
// CT: CTAs of an SM.
template <bool DOWN, int GROUP, int NTM, int CT>
struct Many {
  static constexpr int WEIGHTS = MW * MT_MANY * record_bytes<GROUP>();
  static constexpr int STEP = WEIGHTS + NTM * 8 * 256;
  static constexpr int ST = queue_steps(CT, STEP);
  static constexpr int QUEUE = ST * STEP;
  static_assert(ST >= 3, "a queue of three steps");
  static_assert(QUEUE >= build_bytes(kW4MaxPairs), "the lists' scratch lies in the queue");
};

// place of 16-byte piece c of operand row r
template <int WPL>
__device__ __forceinline__ int operand_place(int r, int c) {
  return WPL == 1 ? c ^ ((r & 1) << 2) : WPL == 2 ? c ^ (r & 1) : c ^ ((c >> 3) & 1) ^ ((r & 1) << 1);
}

template <bool DOWN, int GROUP, int NTM, int CT>
__global__ void __launch_bounds__(MW * 32, CT) w4_many_kernel(const W4Args a) {
  using Q = Many<DOWN, GROUP, NTM, CT>;
  constexpr int WPL = GROUP / 32, MT = MT_MANY;
  constexpr int CR = DOWN ? 4 : 8;  // pairs of a column group
  constexpr int REC = record_bytes<GROUP>(), ST = Q::ST, STEP = Q::STEP, NS = 128 / GROUP;
  extern __shared__ __align__(128) uint8_t smem[];
  if constexpr (!DOWN) pdl_enter();
  const Lists L = build_lists<CR * NTM>(smem + Q::QUEUE, smem, a);
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int tiles = a.C / 16 / (MW * MT);  // units of an entry
  const int NB = a.R / 128;
  // unit = (entry, tile group); a CTA's units are gridDim.x apart
  struct Unit {
    int ent, grp;
  };
  const Unit stride{(int)gridDim.x / tiles, (int)gridDim.x % tiles};
  auto next_unit = [&](Unit &u) {
    u.ent += stride.ent, u.grp += stride.grp;
    if (u.grp >= tiles) u.grp -= tiles, ++u.ent;
  };
  const Unit first_unit{(int)blockIdx.x / tiles, (int)blockIdx.x % tiles};
  const uint32_t ring = ptx::smem_u32(smem), ring_end = ring + ST * STEP;
  const size_t tile_bytes = (size_t)NB * REC;

  // the copying side: this warp's tiles, and one 16-byte piece of every
  // eighth operand row
  const uint32_t wput = w * MT * REC + lane * 16;
  const uint32_t xput = Q::WEIGHTS + (tid >> 4) * 256 + operand_place<WPL>(tid >> 4, tid & 15) * 16;
  Unit pu = first_unit;
  int pb = NB;  // steps of it to go
  uint32_t put = ring;
  const uint8_t *src[MT];
  const uint4 *xsrc[NTM];
  int groups = 0;  // column groups in use
  auto locate = [&]() {
    if (pu.ent >= L.entries) return;
    const int tile = pu.grp * (MW * MT) + w * MT;
    src[0] = a.rec + (size_t)(L.expert(pu.ent) * (a.C / 16) + tile) * tile_bytes + lane * 16;
#pragma unroll
    for (int m = 1; m < MT; ++m) src[m] = src[m - 1] + tile_bytes;
    const int rows = L.count(pu.ent), first = L.first(pu.ent);
    groups = (rows + CR - 1) / CR;
#pragma unroll
    for (int i = 0; i < NTM; ++i) {
      const int r = i * 8 + (tid >> 4);
      const unsigned f = L.pair[first + min(DOWN ? r >> 1 : r, rows - 1)];
      const __nv_bfloat16 *p = DOWN ? (r & 1 ? a.hlo : a.hhi) + wide(f, (unsigned)a.R)
                                    : a.x + wide(f * a.k_inv >> 16, (unsigned)a.R);
      xsrc[i] = reinterpret_cast<const uint4 *>(p) + (tid & 15);
    }
  };
  auto copy_weights = [&]() {
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const uint32_t to = put + wput;
      cp_async16(to + m * REC, src[m]);
      cp_async16(to + m * REC + 512, src[m] + 512);
      if (lane < 2 * NS) cp_async16(to + m * REC + 1024, src[m] + 1024);
      src[m] += REC;
    }
  };
  auto copy_operand = [&]() {
    const uint32_t to = put + xput;
#pragma unroll
    for (int i = 0; i < NTM; ++i) {
      if (i == 0 || i < groups) cp_async16(to + i * 8 * 256, xsrc[i]);
      xsrc[i] += 16;
    }
  };
  auto advance = [&]() {
    put += STEP;
    if (put == ring_end) put = ring;
    if (--pb == 0) {
      pb = NB;
      next_unit(pu);
      locate();
    }
  };
  locate();
  if constexpr (DOWN) {  // weights are on their way before h is there
#pragma unroll 1
    for (int i = 0; i < ST - 1; ++i)
      if (pu.ent < L.entries) {
        copy_weights();
        advance();
      }
    pdl_wait();
    pdl_launch();
    pu = first_unit, pb = NB, put = ring;
    locate();
  }
#pragma unroll 1
  for (int i = 0; i < ST - 1; ++i) {
    if (pu.ent < L.entries) {
      if constexpr (!DOWN) copy_weights();
      if constexpr (DOWN)
#pragma unroll
        for (int m = 0; m < MT; ++m) src[m] += REC;
      copy_operand();
      advance();
    }
    ptx::cp_async_commit();
  }

  uint32_t get = ring;
  const uint32_t sget = w * MT * REC + 1024 + g * (4 * NS);
  uint32_t xget[4];  // this lane's operand pieces of a step, column group 0
#pragma unroll
  for (int j = 0; j < 4; ++j)
    xget[j] = Q::WEIGHTS + g * 256 +
              operand_place<WPL>(g, (j / WPL) * 4 * WPL + t * WPL + j % WPL) * 16;
#pragma unroll 1
  for (Unit u = first_unit; u.ent < L.entries; next_unit(u)) {
    const int tile = u.grp * (MW * MT) + w * MT;
    const int rows = L.count(u.ent), first = L.first(u.ent);
    auto pass = [&](auto nt_c) {
      constexpr int NT = decltype(nt_c)::value;
      float acc[MT][NT][4];
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < NT; ++i)
          acc[m][i][0] = acc[m][i][1] = acc[m][i][2] = acc[m][i][3] = 0.f;
#pragma unroll 1
      for (int b = NB; b > 0; --b) {
        ptx::cp_async_wait<ST - 2>();
        __syncthreads();  // the step has arrived; the one before it has been used
        if (pu.ent < L.entries) {
          copy_weights();
          copy_operand();
          advance();
        }
        ptx::cp_async_commit();
        const uint32_t rec = get + wput;
        uint4 wd[MT][2], sc[MT];
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          wd[m][0] = lds128(rec + m * REC);
          wd[m][1] = lds128(rec + m * REC + 512);
          sc[m] = load_scales<GROUP>(get + sget + m * REC);
        }
        const uint32_t x = get;
        get += STEP;
        if (get == ring_end) get = ring;
        step_product<GROUP, MT, NT>(
            wd, sc, [&](int i, int j) { return lds128(x + xget[j] + i * 8 * 256); }, acc);
      }
#pragma unroll
      for (int m = 0; m < MT; ++m)
        store_tile<DOWN, NT>(a, L, acc[m], tile + m, rows, first, lane);
    };
    if (NTM == 1 || rows <= CR) {
      pass(std::integral_constant<int, 1>());
    } else if constexpr (NTM >= 2) {
      if (NTM == 2 || rows <= 2 * CR) {
        pass(std::integral_constant<int, 2>());
      } else if constexpr (NTM == 4) {
        if (rows <= 3 * CR)
          pass(std::integral_constant<int, 3>());
        else
          pass(std::integral_constant<int, 4>());
      }
    }
  }
  ptx::cp_async_wait<0>();
}

// y[t] = sum over k of the weighted rows of its valid experts, in slot order.
// Bound: the L2, where the rows still are, and its own launch: 120 tokens of
// H = 2048, K = 8 (7.9 MB) 7.6 us alone.
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
// lane = column, so the row-major weights are read along rows, once for the
// group's largest magnitude and once, from the cache, for the codes.  Done once
// for a layer's weights: 537 MB of bf16 in 460 us (1.2 TB/s).
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
    // magnitudes compare as their bits do, infinity and NaN above all others
    unsigned bits = 0;
#pragma unroll 8
    for (int r = 0; r < GROUP; ++r)
      bits = max(bits, __bfloat16_as_ushort(src[(size_t)r * C]) & 0x7fffu);
    const float top = bits < 0x7f80u ? __uint_as_float(bits << 16) : NAN;
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

// Records of w13 (DOWN false) or w2: a warp writes a record, 16 bytes a lane and
// turn.  Done once for a layer's weights: 67 MB of codes in 117 us, 34 MB in 32 us
// (the reads are pieces of 64 bytes).
template <bool DOWN, int GROUP>
__global__ void __launch_bounds__(256) prepare_w4_kernel(const uint32_t *__restrict__ q,
                                                         const __nv_bfloat16 *__restrict__ s,
                                                         uint8_t *__restrict__ rec,
                                                         long long records, int C, int R) {
  pdl_enter();
  constexpr int NS = 128 / GROUP, WPL = 4 / NS, REC = record_bytes<GROUP>();
  const int NB = R / 128, tiles = C / 16, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  for (long long r = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); r < records;
       r += (long long)gridDim.x * 8) {
    const long long rt = r / NB;
    const int b = (int)(r - rt * NB);
    const size_t e = (size_t)(rt / tiles);
    const int tile = (int)(rt - (long long)e * tiles);
    auto row = [&](int gg, int half) {
      return e * C + (DOWN ? tile * 16 + 8 * half + gg : half * (C / 2) + tile * 8 + gg);
    };
    uint4 v[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {  // plane h: the lane's four words of its row
      const uint32_t *from = q + row(g, h) * (R / 8) + b * 16 + t * WPL;
      uint32_t *o = reinterpret_cast<uint32_t *>(&v[h]);
#pragma unroll
      for (int j = 0; j < 4; ++j) o[j] = __ldg(from + (j / WPL) * 4 * WPL + j % WPL);
    }
    uint4 *to = reinterpret_cast<uint4 *>(rec + r * REC);
    to[lane] = v[0];
    to[32 + lane] = v[1];
    if (lane < 2 * NS) {  // scales (g, half, NS), eight of them
      __align__(16) __nv_bfloat16 o[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int k = lane * 8 + j, gg = k / (2 * NS), half = k / NS % 2;
        o[j] = s[row(gg, half) * (R / GROUP) + b * NS + k % NS];
      }
      to[64 + lane] = *reinterpret_cast<const uint4 *>(o);
    }
  }
}

inline size_t align256(size_t v) { return (v + 255) & ~(size_t)255; }

// smem: the queue's bytes; the lists follow.  units: of the whole call at most.
template <auto Kernel>
cudaError_t launch_w4(const W4Args &a, int queue, int rows, int threads, int ctas,
                      long long units, cudaStream_t s) {
  const int smem = queue + (rows ? lists_bytes(a.nK, a.E, rows) : 0);
  static bool ready[64] = {false};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  bool &r = ready[dev >= 0 && dev < 64 ? dev : 0];
  if (!r) {
    e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             queue + (rows ? lists_bytes(kW4MaxPairs, kMaxE, rows) : 0));
    if (e != cudaSuccess) return e;
    r = true;
  }
  const long long fit = 227 * 1024 / (smem + 1024);
  const long long full = (fit < ctas ? fit : ctas) * device_sm_count();
  return launch_pdl(Kernel, dim3((unsigned)(units < full ? units : full)), dim3(threads), smem, s,
                    a);
}

template <bool DOWN, int GROUP, int NTM, int CT>
cudaError_t launch_many(const W4Args &a, cudaStream_t s) {
  constexpr int rows = (DOWN ? 4 : 8) * NTM;
  return launch_w4<w4_many_kernel<DOWN, GROUP, NTM, CT>>(
      a, Many<DOWN, GROUP, NTM, CT>::QUEUE, rows, MW * 32, CT,
      (long long)max_entries(a.nK, a.E, rows) * (a.C / 16 / (MW * MT_MANY)), s);
}

// CTAs of an SM for `units` equal units: as few as hold them all at once (the
// queues are deeper), else those whose last round is fullest; 4 are a little
// faster in the long run (61 tokens at H = 7168, I = 2048, E = 256: 919, 901 and
// 936 us with 3, 4 and 5), 5 where they make one round of two (3 tokens there:
// 124, 132 and 112 us).
inline int ctas_for(double units) {
  const double sms = device_sm_count();
  const double weight[] = {0.97, 1.0, 0.985};
  int best = 3;
  double top = 0.0;
  for (int c = 3; c <= 5; ++c) {
    const double rounds = units / (c * sms);
    if (rounds <= 1.0) return c;
    const double score = weight[c - 3] * rounds / ceil(rounds);
    if (score > top) top = score, best = c;
  }
  return best;
}

// Few pairs, in units of the first product (tiles over all pairs): up to one to
// four warps of the grid, two warps share a unit's reduction; up to one to two,
// a warp takes a unit while its reduction is short.  Beyond that the other
// kernel's larger steps pay.  One token, I = 1024, group 128, the kernel taken
// and the next best: 512 units of H = 2048 8.5 us (other kernel 13.8), of 4096
// 13.3 (20.4), of 7168 20.6 (28.5); 1024 units of H = 2048 13.8 (two warps a unit
// 14.5, other kernel 16.3), of 4096 24.1 (two warps 24.6, one 30.5), of 7168 32.4
// (37, 47.7); two tokens of H = 2048 22 (26).
inline long long few_units(const W4Args &a) { return (long long)a.nK * (a.I / 8); }
inline bool few_shared(const W4Args &a) { return few_units(a) <= 4 * device_sm_count(); }
inline bool few_pairs(const W4Args &a) {
  return a.nK <= kFewPairs &&
         (few_shared(a) || (a.H <= 2048 && few_units(a) <= 8 * device_sm_count()));
}

// The first product's CTAs with shared reductions are no more than the SMs, and ask
// for half of an SM's shared memory so that no two share one: beside the CTAs of
// a call before and of the second product they else settle in pairs, in some
// runs for good (one token, I = 512, eight experts of H = 4096: 12 us against 19;
// four of H = 2048, I = 1024: 8.5 against 9.8; not where a warp has a unit to
// itself: eight of H = 2048 16.5 against 14).
constexpr int kHalfSm = 114 * 1024;

template <bool DOWN, int GROUP, int KS>
cudaError_t launch_few(const W4Args &a, cudaStream_t s) {
  using F = Few<DOWN, GROUP, KS>;
  constexpr int teams = F::WW / KS;
  constexpr int smem = !DOWN && KS == 2 ? kHalfSm : F::QUEUE;
  static_assert(smem >= F::QUEUE, "the queue");
  return launch_w4<w4_few_kernel<DOWN, GROUP, KS>>(
      a, smem, 0, F::WT, F::CTAS,
      DOWN ? a.C / 16 : (few_units(a) + teams - 1) / teams, s);
}

template <bool DOWN, int GROUP>
cudaError_t launch_stage(const W4Args &a, cudaStream_t s) {
  if (few_pairs(a))
    // (a reduction of less than eight steps is too short to share)
    return few_shared(a) && a.R >= 1024 ? launch_few<DOWN, GROUP, 2>(a, s)
                                        : launch_few<DOWN, GROUP, 1>(a, s);
  // column groups for most experts' tokens at once (the mean and one deviation
  // of their number); what exceeds them reads the weights again, mostly from
  // L2.  With four deviations, 30 and 45 tokens at H = 2048, I = 1024, E = 64
  // take 60 and 65 us against 54 and 59, 128 at H = 7168, E = 256 1173 against
  // 1127.
  const float mean = (float)a.nK / a.E, want = (mean + sqrtf(mean)) / (DOWN ? 4 : 8);
  if (want <= 1.f) {
    // experts hit by tokens that choose theirs independently
    const double hit = a.E * (1.0 - pow(1.0 - (double)a.K / a.E, (double)a.nK / a.K));
    const int c = ctas_for(hit * (a.C / 16 / (MW * MT_MANY)));
    return c == 3   ? launch_many<DOWN, GROUP, 1, 3>(a, s)
           : c == 4 ? launch_many<DOWN, GROUP, 1, 4>(a, s)
                    : launch_many<DOWN, GROUP, 1, 5>(a, s);
  }
  if (want <= 2.f) return launch_many<DOWN, GROUP, 2, 3>(a, s);
  return launch_many<DOWN, GROUP, 4, 3>(a, s);
}

template <int GROUP>
cudaError_t run(const Desc &d, W4Args a, const void *w13_t, const void *w2_t, cudaStream_t s) {
  a.rec = reinterpret_cast<const uint8_t *>(w13_t);
  a.C = 2 * d.I, a.R = d.H;
  cudaError_t e = launch_stage<false, GROUP>(a, s);
  if (e != cudaSuccess) return e;
  a.rec = reinterpret_cast<const uint8_t *>(w2_t);
  a.C = d.H, a.R = d.I;
  e = launch_stage<true, GROUP>(a, s);
  if (e != cudaSuccess || few_pairs(a)) return e;
  const int V = d.H / 4;
  const long long want = ((long long)d.n * V + 255) / 256, cap = 8ll * device_sm_count();
  return launch_pdl(w4_combine_kernel, dim3((int)(want < cap ? want : cap)), dim3(256), 0, s,
                    reinterpret_cast<const float4 *>(a.yslot), a.idx,
                    reinterpret_cast<uint2 *>(a.y), d.n, d.K, d.E, V);
}

template <int GROUP>
cudaError_t prepare(const Desc &d, int which, const int32_t *q, const void *scales, void *tiled,
                    cudaStream_t s) {
  const int C = which ? d.H : 2 * d.I, R = which ? d.I : d.H;
  const long long records = (long long)d.E * (C / 16) * (R / 128);
  const long long want = (records + 7) / 8, cap = 64ll * device_sm_count();
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
  a.y = reinterpret_cast<__nv_bfloat16 *>(y);
  uint8_t *p = reinterpret_cast<uint8_t *>(ws);
  const size_t hb = align256((size_t)d.nK() * d.I * 2);
  a.hhi = reinterpret_cast<__nv_bfloat16 *>(p);
  a.hlo = reinterpret_cast<__nv_bfloat16 *>(p + hb);
  a.yslot = reinterpret_cast<float *>(p + 2 * hb);
  a.nK = (int)d.nK(), a.K = d.K, a.E = d.E, a.H = d.H, a.I = d.I;
  a.k_inv = (65536u + d.K - 1) / d.K;
  a.status = status;
  if (group == 32) return run<32>(d, a, w13_t, w2_t, s);
  if (group == 64) return run<64>(d, a, w13_t, w2_t, s);
  return run<128>(d, a, w13_t, w2_t, s);
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
