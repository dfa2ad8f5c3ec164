// trunk.h -- host-side calls of the operators of a recurrent policy's trunk
// (RMS norm, gated scan), between the C entry points and the kernels.
// Arguments are checked by the entry points.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

namespace rlca {

// ---- RMS norm (k_rms.cu) -----------------------------------------------------
struct RmsArgs {
  const float *x, *residual, *weight;  // element type by `bf16_io`
  float *total, *y;                    // total: null without a residual
  uint8_t *y8, *total8;
  float *y8_scale, *total8_scale, *rstd;
  int64_t N, D, x_stride, residual_stride;
  float eps;
  bool bf16_io;
};
cudaError_t run_rms_norm(const RmsArgs& a, int sm_count, cudaStream_t s);

struct RmsGradArgs {
  const float *dy, *d_total, *total, *weight, *rstd;
  const uint8_t* total8;  // read (with its scales) where total is null
  const float* total8_scale;
  float *dx, *dweight;
  int64_t N, D, dy_stride, d_total_stride, total_stride;
  bool bf16_io;
  float* ws;
};
cudaError_t run_rms_norm_backward(const RmsGradArgs& a, int sm_count, cudaStream_t s);

// ---- gated scan (k_gated.cu) ---------------------------------------------------
// Element (e, t, c) of a matrix with row stride r lies at (e step_e + t step_t) r + c.
struct GatedArgs {
  const float *x, *gate;  // element type by `bf16_io`
  const uint8_t *terminated, *truncated;
  const float* state;
  const int32_t* lengths;
  float *h, *last;
  // backward
  const float *dh, *in_h, *d_last;
  float *dx, *dgate, *d_state;
  int64_t E, T, D, step_e, step_t;
  int64_t x_stride, gate_stride, h_stride, dh_stride, dx_stride, dgate_stride;
  bool bf16_io;
  void* ws;
  int nseg, seg_len;  // segments of a row, and their steps (set by the calls)
};
cudaError_t run_gated_scan(const GatedArgs& a, int sm_count, cudaStream_t s);
cudaError_t run_gated_scan_backward(const GatedArgs& a, int sm_count, cudaStream_t s);

}  // namespace rlca
