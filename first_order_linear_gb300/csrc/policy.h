// policy.h -- host-side calls of the policy-update operators (layer norm,
// token log-probabilities, gradient clipping), between the C entry points
// and the kernels.  Arguments are checked by the entry points.
#pragma once

#include <atomic>
#include <cstddef>
#include <cstdint>
#include <cuda.h>  // CUtensorMap
#include <cuda_runtime.h>

namespace rlca {

// one kernel on `s`, allowed to be scheduled while its predecessor drains
// (every kernel here waits for the predecessor before it touches memory)
template <class... P, class... A>
cudaError_t launch_pdl(void (*kernel)(P...), int64_t grid, int block, size_t smem, cudaStream_t s, const A&... args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Opts a kernel in to `bytes` of dynamic shared memory on the current device,
// the first time it is launched there.
template <class K>
cudaError_t allow_smem(K* kernel, size_t bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

constexpr int64_t div_up(int64_t a, int64_t b) { return (a + b - 1) / b; }

// ---- layer norm (k_norm.cu) ------------------------------------------------
struct NormArgs {
  const float *x, *weight, *bias;  // element type by `bf16_io`
  float *y, *mean, *rstd;
  int64_t N, D, x_stride;
  float eps;
  bool bf16_io;
};
cudaError_t run_layer_norm(const NormArgs& a, int sm_count, cudaStream_t s);

struct NormGradArgs {
  const float *dy, *x, *weight, *mean, *rstd;
  float *dx, *dweight, *dbias;
  int64_t N, D, dy_stride, x_stride;
  bool bf16_io;
  float* ws;
};
size_t layer_norm_backward_workspace(int64_t N, int64_t D, int sm_count);
cudaError_t run_layer_norm_backward(const NormGradArgs& a, int sm_count, cudaStream_t s);

// ---- token log-probabilities (k_head.cu) -------------------------------------
struct HeadArgs {
  const float *hidden, *weight;  // element type by `bf16_io`
  const int32_t* tokens;
  float *logp, *lse, *entropy;  // forward outputs
  // backward
  const float *in_lse, *in_entropy, *d_logp, *d_entropy;
  float *d_hidden, *d_weight;
  int64_t N, D, V, hidden_stride, weight_stride;
  float inv_temperature;
  bool bf16_io;
  void* ws;
};
size_t head_workspace(int64_t N, int64_t D, int64_t V, bool bf16_io, bool backward, int sm_count);
cudaError_t run_token_logprob(const HeadArgs& a, int sm_count, cudaStream_t s);
cudaError_t run_token_logprob_backward(const HeadArgs& a, int sm_count, cudaStream_t s);

// ---- gradient clipping (k_clip.cu) -------------------------------------------
struct ClipArgs {
  const void* const* grads;
  void* const* outs;
  const int64_t* sizes;
  const uint32_t* dtypes;
  int64_t count;
  float max_norm, eps;
  float* norm;
  double* ws;
};
size_t clip_workspace(int64_t count, int sm_count);
cudaError_t run_clip_grads(const ClipArgs& a, int sm_count, cudaStream_t s);

// the device status words of these translation units, ORed into *word
cudaError_t status_norm(unsigned int* word, bool clear);
cudaError_t status_head(unsigned int* word, bool clear);
cudaError_t status_clip(unsigned int* word, bool clear);

int checked_build_status(cudaStream_t s);

// Map of `planes` bfloat16 matrices [rows, width] (strides in elements, both
// multiples of 8; base 16-byte aligned) for copies of 64 x box_rows boxes in
// the 128-byte swizzle; what lies outside reads as zero.  False when the
// encoder is unavailable or refuses.
bool encode_matrix_map(CUtensorMap* m, const void* base, int64_t width, int64_t rows, int64_t planes,
                       int64_t row_stride, int64_t plane_stride, int box_rows);

}  // namespace rlca
