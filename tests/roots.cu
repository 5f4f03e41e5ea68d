// Every float32 of a range through the functions of roots.cuh, for test_gpu_roots.py.
#include <cuda_runtime.h>
#include <math.h>

#include "roots.cuh"

using namespace moe;

namespace {

constexpr double kU = 0x1p-24;

// what: 0 root2 (both halves), 1 reciprocal: counts[0] results that are not the
// correctly rounded ones; 2 approx_rcp, 3 rsqrt_of: results further than 2 u.
// counts[1]: values looked at.
__global__ void roots_kernel(int what, unsigned first, unsigned last, unsigned long long *counts) {
  const unsigned long long step = (unsigned long long)gridDim.x * blockDim.x;
  unsigned long long wrong = 0, seen = 0;
  for (unsigned long long i = first + (unsigned long long)blockIdx.x * blockDim.x + threadIdx.x;
       i <= last; i += step) {
    const float x = __uint_as_float((unsigned)i);
    bool ok;
    if (what == 0) {
      const float other = __uint_as_float(first + (last - (unsigned)i));
      const float2 r = root2(make_float2(x, other));
      ok = r.x == __fsqrt_rn(x) && r.y == __fsqrt_rn(other);
    } else if (what == 1) {
      ok = reciprocal(x) == __frcp_rn(x);
    } else if (what == 2) {
      ok = fabs((double)x * approx_rcp(x) - 1.0) <= 2 * kU;
    } else {
      // (1 + e)^2 - 1 = 2 e + e^2
      const double r = rsqrt_of(x);
      ok = fabs(r * r * x - 1.0) <= 4 * kU * (1 + 1e-6);
    }
    wrong += !ok, ++seen;
  }
  atomicAdd(counts, wrong);
  atomicAdd(counts + 1, seen);
}

}  // namespace

extern "C" int roots_check(int what, unsigned first, unsigned last, unsigned long long *counts) {
  roots_kernel<<<1216, 256>>>(what, first, last, counts);
  return (int)cudaGetLastError();
}
