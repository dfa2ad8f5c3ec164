// Layer norm and its gradient.
#include "policy.h"
#include "reduce.cuh"

namespace rlca {

namespace {

constexpr int kNormThreads = 256;

// y = (x - mean) * rstd * w + b.  The variance is the mean square of the
// centred row (two passes over the row): sum(x^2) - mean^2 would cancel for
// rows whose mean is large against their spread.
template <class ST>
__global__ void __launch_bounds__(kNormThreads) norm_rows_kernel(NormArgs a) {
  pdl_trigger();
  pdl_wait();
  __shared__ float scratch[32];
  const int64_t i = blockIdx.x;
  const float inv_d = 1.f / (float)a.D;
  const int64_t at = i * a.x_stride;
  float s = 0.f;
  for (int64_t c = threadIdx.x; c < a.D; c += blockDim.x) s += Stor<ST>::ld(a.x, at + c);
  const float mean = cta_sum(s, scratch) * inv_d;
  float q = 0.f;
  for (int64_t c = threadIdx.x; c < a.D; c += blockDim.x) {
    const float d = Stor<ST>::ld(a.x, at + c) - mean;
    q += d * d;
  }
  const float rstd = rsqrtf(cta_sum(q, scratch) * inv_d + a.eps);
  for (int64_t c = threadIdx.x; c < a.D; c += blockDim.x) {
    const float xh = (Stor<ST>::ld(a.x, at + c) - mean) * rstd;
    const float b = a.bias ? Stor<ST>::ld(a.bias, c) : 0.f;
    Stor<ST>::st(a.y, i * a.D + c, xh * Stor<ST>::ld(a.weight, c) + b);
  }
  if (threadIdx.x == 0) {
    if (a.mean) a.mean[i] = mean;
    if (a.rstd) a.rstd[i] = rstd;
  }
}

template <class ST>
__global__ void __launch_bounds__(kNormThreads) norm_grad_rows_kernel(NormGradArgs a) {
  pdl_trigger();
  pdl_wait();
  __shared__ float scratch[32];
  const int64_t i = blockIdx.x;
  const float inv_d = 1.f / (float)a.D;
  const float mean = a.mean[i], rstd = a.rstd[i];
  float s1 = 0.f, s2 = 0.f;
  for (int64_t c = threadIdx.x; c < a.D; c += blockDim.x) {
    const float g = Stor<ST>::ld(a.dy, i * a.dy_stride + c) * Stor<ST>::ld(a.weight, c);
    const float xh = (Stor<ST>::ld(a.x, i * a.x_stride + c) - mean) * rstd;
    s1 += g;
    s2 += g * xh;
  }
  s1 = cta_sum(s1, scratch) * inv_d;
  s2 = cta_sum(s2, scratch) * inv_d;
  for (int64_t c = threadIdx.x; c < a.D; c += blockDim.x) {
    const float g = Stor<ST>::ld(a.dy, i * a.dy_stride + c) * Stor<ST>::ld(a.weight, c);
    const float xh = (Stor<ST>::ld(a.x, i * a.x_stride + c) - mean) * rstd;
    Stor<ST>::st(a.dx, i * a.D + c, rstd * (g - s1 - xh * s2));
  }
}

// rows a slice of the weight gradient's first sum covers
constexpr int64_t kSliceRows = 64;

// ws[slice][0][c] = sum over the slice's rows of dy * xh, ws[slice][1][c] = of dy
template <class ST>
__global__ void __launch_bounds__(kNormThreads) norm_grad_slices_kernel(NormGradArgs a, int64_t col_blocks) {
  pdl_trigger();
  pdl_wait();
  const int64_t slice = blockIdx.x / col_blocks;
  const int64_t c = (blockIdx.x % col_blocks) * kNormThreads + threadIdx.x;
  if (c >= a.D) return;
  const int64_t i1 = min(a.N, (slice + 1) * kSliceRows);
  float dw = 0.f, db = 0.f;
  for (int64_t i = slice * kSliceRows; i < i1; ++i) {
    const float dy = Stor<ST>::ld(a.dy, i * a.dy_stride + c);
    dw += dy * ((Stor<ST>::ld(a.x, i * a.x_stride + c) - a.mean[i]) * a.rstd[i]);
    db += dy;
  }
  a.ws[(2 * slice) * a.D + c] = dw;
  a.ws[(2 * slice + 1) * a.D + c] = db;
}

// the slices' sums, in order
template <class ST>
__global__ void __launch_bounds__(kNormThreads) norm_grad_join_kernel(NormGradArgs a, int64_t slices) {
  pdl_trigger();
  pdl_wait();
  const int64_t c = (int64_t)blockIdx.x * kNormThreads + threadIdx.x;
  if (c >= a.D) return;
  float dw = 0.f, db = 0.f;
  for (int64_t k = 0; k < slices; ++k) {
    dw += a.ws[(2 * k) * a.D + c];
    db += a.ws[(2 * k + 1) * a.D + c];
  }
  if (a.dweight) Stor<ST>::st(a.dweight, c, dw);
  if (a.dbias) Stor<ST>::st(a.dbias, c, db);
}

template <class ST>
cudaError_t grad_typed(const NormGradArgs& a, cudaStream_t s) {
  if (a.dx != nullptr && a.N > 0) {
    cudaError_t e = launch_pdl(norm_grad_rows_kernel<ST>, a.N, kNormThreads, 0, s, a);
    if (e != cudaSuccess) return e;
  }
  if (a.dweight == nullptr && a.dbias == nullptr) return cudaSuccess;
  const int64_t slices = div_up(a.N, kSliceRows), col_blocks = div_up(a.D, kNormThreads);
  if (slices > 0) {
    cudaError_t e = launch_pdl(norm_grad_slices_kernel<ST>, slices * col_blocks, kNormThreads, 0, s, a, col_blocks);
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(norm_grad_join_kernel<ST>, col_blocks, kNormThreads, 0, s, a, slices);
}

}  // namespace

cudaError_t run_layer_norm(const NormArgs& a, int, cudaStream_t s) {
  return a.bf16_io ? launch_pdl(norm_rows_kernel<bf16>, a.N, kNormThreads, 0, s, a)
                   : launch_pdl(norm_rows_kernel<float>, a.N, kNormThreads, 0, s, a);
}

size_t layer_norm_backward_workspace(int64_t N, int64_t D, int) {
  return (size_t)div_up(N, kSliceRows) * 2 * (size_t)D * sizeof(float);
}

cudaError_t run_layer_norm_backward(const NormGradArgs& a, int, cudaStream_t s) {
  return a.bf16_io ? grad_typed<bf16>(a, s) : grad_typed<float>(a, s);
}

cudaError_t status_norm(unsigned int* word, bool clear) { return unit_status(word, clear); }

}  // namespace rlca
