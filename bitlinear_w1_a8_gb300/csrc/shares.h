// shares.h -- the arithmetic by which attention.cu shares rows out over CTAs in proportion
// to their steps.  Plain functions of whole numbers, for the host, the device and tests.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define BITLINEAR_BOTH __host__ __device__ __forceinline__
#else
#define BITLINEAR_BOTH inline
#endif

namespace bitlinear {

// Whether the steps of `rows` rows, `steps` each at most, are counted in 31 bits.
BITLINEAR_BOTH bool steps_fit(int64_t rows, int64_t steps) { return steps <= 0x7fffffff / rows; }

// Steps that a CTA has at most, so that rows of ceil(steps / share) CTAs each, `total` steps
// in all, fit `spare` CTAs beside one a row.  total may be 2^31 - 1, and total + spare more.
BITLINEAR_BOTH int share_of_steps(int total, int spare, int least) {
  const int share = (int)(((uint32_t)total + (uint32_t)spare - 1u) / (uint32_t)spare);
  return share > least ? share : least;
}

}  // namespace bitlinear
