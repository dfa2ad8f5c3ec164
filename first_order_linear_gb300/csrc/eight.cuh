// eight.cuh -- rows in 8 bits: e4m3 values with a float32 scale for each group
// of consecutive columns.
#pragma once

#include <cuda_fp16.h>

#include "scan_core.cuh"

namespace rlca {

constexpr int kGroup = 128;  // RLCA_GROUP
// The exponent keeps what is small beside a few large columns (a stream's
// usual outliers), which whole numbers under the same scale would lose; the
// groups keep a large column from setting the scale of a whole row.
constexpr float kE4m3Max = 448.f;

__host__ __device__ constexpr int64_t groups_of(int64_t D) { return (D + kGroup - 1) / kGroup; }

// Products with reciprocals: quotients rounded as divisions round them would
// only move values that lie on a border of two steps already, and the norm's
// issue slots are its next bound behind HBM (65536 x 4096 bfloat16 with two
// 8-bit outputs: 318 us; with divisions 513 us, with a paired remainder step in
// their place 340 us; unaligned 300000 x 201 163, 276 and 193 us).
// (A group of zeros gets the smallest normal scale, whose reciprocal is finite.)
__device__ __forceinline__ float group_scale(float amax) { return fmaxf(amax * (1.f / kE4m3Max), 1.17549435e-38f); }

// two values, the first at the lower address; saturating, NaN kept
__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float2 from_e4m3x2(uint32_t v) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)v));
  return __half22float2(*reinterpret_cast<const __half2*>(&r));
}

}  // namespace rlca
