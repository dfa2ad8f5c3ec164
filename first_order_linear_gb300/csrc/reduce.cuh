// reduce.cuh -- sums over warps and CTAs, in a fixed order, for the
// policy-update operators.
#pragma once

#include "scan_core.cuh"

namespace rlca {

template <class T>
__device__ __forceinline__ T warp_sum(T v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sum over a CTA of at most 1024 threads (whole warps), returned to all of
// them; `scratch` holds one value per warp and is free again on return.
template <class T>
__device__ __forceinline__ T cta_sum(T v, T* scratch) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, n = blockDim.x >> 5;
  v = warp_sum(v);
  if (lane == 0) scratch[warp] = v;
  __syncthreads();
  T t = lane < n ? scratch[lane] : T(0);
  t = warp_sum(t);
  __syncthreads();
  return t;
}

// reads and (with clear) zeroes this translation unit's status word
static inline cudaError_t unit_status(unsigned int* word, bool clear) {
  unsigned int w = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&w, g_tu_status, sizeof(w));
  if (e != cudaSuccess) return e;
  *word |= w;
  if (clear && w != 0) {
    const unsigned int zero = 0;
    e = cudaMemcpyToSymbol(g_tu_status, &zero, sizeof(zero));
  }
  return e;
}

}  // namespace rlca
