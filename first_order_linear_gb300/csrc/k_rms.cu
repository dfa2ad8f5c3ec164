// Root-mean-square norm with the residual's addition, its result and its
// input in 8 bits, and its gradient.
//
//   total = x + residual,  y = total rstd w,  rstd = 1 / sqrt(mean(total^2) + eps)
//   dx = d_total + rstd (g - s mean(g s)),  g = dy w,  s = total rstd
//   dw = sum over rows of dy s
#include <algorithm>

#include "eight.cuh"
#include "policy.h"
#include "reduce.cuh"
#include "trunk.h"

namespace rlca {

namespace {

// Plain loads: total may be the residual's buffer, and rows too long for
// registers are read again from it.
template <class ST>
__device__ __forceinline__ float load1(const float* p, int64_t i, int64_t n) {
  if (!in_range(i, n)) return 0.f;
  if constexpr (Stor<ST>::kBytes == 4) return p[i];
  else return Stor<ST>::from_bits(reinterpret_cast<const uint16_t*>(p)[i]);
}
template <class ST>
__device__ __forceinline__ void store1(float* p, int64_t i, int64_t n, float v) {
  if (in_range(i, n)) Stor<ST>::st(p, i, v);
}
// v as it reads back from its storage
template <class ST>
__device__ __forceinline__ float stored(float v) {
  if constexpr (Stor<ST>::kBytes == 4) return v;
  else return Stor<ST>::from_bits(Stor<ST>::to_bits(v));
}
__device__ __forceinline__ int64_t extent(int64_t rows, int64_t width, int64_t stride) { return (rows - 1) * stride + width; }

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFullMask, v, o));
  return v;
}

// ---------------------------------------------------------------------------
// A CTA a row, two passes over it: a warp takes a group of columns at a time,
// a lane four of them, 32 apart.
// ---------------------------------------------------------------------------
constexpr int kLongThreads = 512;
constexpr int kPart = kGroup / 32;

// one group of a row in 8 bits
__device__ __forceinline__ void store_group(uint8_t* q, float* scale, const RmsArgs& a, int64_t row, int64_t group, int lane,
                                            const float* v) {
  const int64_t groups = groups_of(a.D);
  float m = 0.f;
#pragma unroll
  for (int k = 0; k < kPart; ++k) m = fmaxf(m, fabsf(v[k]));
  const float sc = group_scale(warp_max(m)), inv = __frcp_rn(sc);
  if (lane == 0 && in_range(row * groups + group, a.N * groups)) scale[row * groups + group] = sc;
#pragma unroll
  for (int k = 0; k < kPart; ++k) {
    const int64_t c = group * kGroup + lane + 32 * k;
    if (c < a.D && in_range(row * a.D + c, a.N * a.D)) q[row * a.D + c] = (uint8_t)to_e4m3x2(v[k] * inv, 0.f);
  }
}

template <class ST>
__global__ void __launch_bounds__(kLongThreads) rms_long_kernel(RmsArgs a) {
  pdl_trigger();
  pdl_wait();
  __shared__ float scratch[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t groups = groups_of(a.D), nd = a.N * a.D;
  for (int64_t row = blockIdx.x; row < a.N; row += gridDim.x) {
    float ss = 0.f;
    for (int64_t g = warp; g < groups; g += kLongThreads / 32) {
#pragma unroll
      for (int k = 0; k < kPart; ++k) {
        const int64_t c = g * kGroup + lane + 32 * k;
        if (c >= a.D) continue;
        float v = load1<ST>(a.x, row * a.x_stride + c, extent(a.N, a.D, a.x_stride));
        if (a.residual != nullptr) {
          v = stored<ST>(v + load1<ST>(a.residual, row * a.residual_stride + c, extent(a.N, a.D, a.residual_stride)));
          store1<ST>(a.total, row * a.D + c, nd, v);
        }
        ss = fmaf(v, v, ss);
      }
    }
    const float rstd = rsqrtf(cta_sum(ss, scratch) / (float)a.D + a.eps);
    if (threadIdx.x == 0 && a.rstd != nullptr) a.rstd[row] = rstd;
    if (a.y == nullptr && a.y8 == nullptr && a.total8 == nullptr) continue;
    for (int64_t g = warp; g < groups; g += kLongThreads / 32) {
      float v[kPart], y[kPart];
#pragma unroll
      for (int k = 0; k < kPart; ++k) {
        const int64_t c = g * kGroup + lane + 32 * k;
        v[k] = y[k] = 0.f;
        if (c >= a.D) continue;
        // (this thread's own stores of the first pass)
        v[k] = a.residual != nullptr ? load1<ST>(a.total, row * a.D + c, nd)
                                     : load1<ST>(a.x, row * a.x_stride + c, extent(a.N, a.D, a.x_stride));
        y[k] = v[k] * rstd * load1<ST>(a.weight, c, a.D);
        if (a.y != nullptr) store1<ST>(a.y, row * a.D + c, nd, y[k]);
      }
      if (a.y8 != nullptr) store_group(a.y8, a.y8_scale, a, row, g, lane, y);
      if (a.total8 != nullptr) store_group(a.total8, a.total8_scale, a, row, g, lane, v);
    }
  }
}

// total of the gradient's rows, as stored or from its 8 bits
template <class ST>
__device__ __forceinline__ float grad_total(const RmsGradArgs& a, int64_t row, int64_t c) {
  if (a.total != nullptr) return load1<ST>(a.total, row * a.total_stride + c, extent(a.N, a.D, a.total_stride));
  const int64_t groups = groups_of(a.D), g = row * groups + c / kGroup;
  if (!in_range(row * a.D + c, a.N * a.D) || !in_range(g, a.N * groups)) return 0.f;
  return from_e4m3x2(a.total8[row * a.D + c]).x * a.total8_scale[g];
}

template <class ST>
__global__ void __launch_bounds__(kLongThreads) rms_grad_long_kernel(RmsGradArgs a) {
  pdl_trigger();
  pdl_wait();
  __shared__ float scratch[32];
  const int64_t dy_size = extent(a.N, a.D, a.dy_stride);
  for (int64_t row = blockIdx.x; row < a.N; row += gridDim.x) {
    const float rstd = a.rstd[row];
    float along = 0.f;
    for (int64_t c = threadIdx.x; c < a.D; c += kLongThreads) {
      const float g = load1<ST>(a.dy, row * a.dy_stride + c, dy_size) * load1<ST>(a.weight, c, a.D);
      along = fmaf(g, grad_total<ST>(a, row, c) * rstd, along);
    }
    along = cta_sum(along, scratch) / (float)a.D;
    for (int64_t c = threadIdx.x; c < a.D; c += kLongThreads) {
      const float g = load1<ST>(a.dy, row * a.dy_stride + c, dy_size) * load1<ST>(a.weight, c, a.D);
      float d = rstd * (g - grad_total<ST>(a, row, c) * rstd * along);
      if (a.d_total != nullptr) d += load1<ST>(a.d_total, row * a.d_total_stride + c, extent(a.N, a.D, a.d_total_stride));
      store1<ST>(a.dx, row * a.D + c, a.N * a.D, d);
    }
  }
}

// ... and the sums of dw, a slice of rows a CTA
constexpr int kSliceThreads = 256;
template <class ST>
__global__ void __launch_bounds__(kSliceThreads) rms_grad_slices_kernel(RmsGradArgs a, int64_t col_blocks, int64_t slice_rows) {
  pdl_trigger();
  pdl_wait();
  const int64_t slice = blockIdx.x / col_blocks;
  const int64_t c = (blockIdx.x % col_blocks) * kSliceThreads + threadIdx.x;
  if (c >= a.D) return;
  const int64_t i1 = min(a.N, (slice + 1) * slice_rows), dy_size = extent(a.N, a.D, a.dy_stride);
  float dw = 0.f;
  for (int64_t i = slice * slice_rows; i < i1; ++i)
    dw = fmaf(load1<ST>(a.dy, i * a.dy_stride + c, dy_size), grad_total<ST>(a, i, c) * a.rstd[i], dw);
  if (in_range(slice * a.D + c, a.D * (gridDim.x / col_blocks))) a.ws[slice * a.D + c] = dw;
}

// The partial sums ws[parts][D] of 32 columns a CTA: warp k adds the partials
// k, k + 32, ..., then the warps' sums are added in order.
__global__ void __launch_bounds__(1024) rms_grad_join_kernel(const float* ws, int64_t parts, int64_t D, float* dweight,
                                                             bool bf16_io) {
  pdl_trigger();
  pdl_wait();
  __shared__ float acc[32][33];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t c = (int64_t)blockIdx.x * 32 + lane;
  float s = 0.f;
  if (c < D) {
    constexpr int B = 8;  // loads in flight
    for (int64_t k0 = warp; k0 < parts; k0 += 32 * B) {
      float v[B];
#pragma unroll
      for (int u = 0; u < B; ++u) v[u] = k0 + 32 * u < parts ? load1<float>(ws, (k0 + 32 * u) * D + c, parts * D) : 0.f;
#pragma unroll
      for (int u = 0; u < B; ++u) s += v[u];
    }
  }
  acc[warp][lane] = s;
  __syncthreads();
  if (warp != 0 || c >= D) return;
  s = 0.f;
#pragma unroll
  for (int k = 0; k < 32; ++k) s += acc[k][lane];
  if (bf16_io) store1<bf16>(dweight, c, D, s);
  else store1<float>(dweight, c, D, s);
}

cudaError_t join(const RmsGradArgs& a, int64_t parts, cudaStream_t s) {
  if (a.dweight == nullptr) return cudaSuccess;
  return launch_pdl(rms_grad_join_kernel, div_up(a.D, 32), 1024, 0, s, (const float*)a.ws, parts, a.D, a.dweight, a.bf16_io);
}

// rows of a slice of the long rows' sum: enough slices to fill the SMs
int64_t slice_rows(int64_t N, int64_t D, int sm) {
  const int64_t want = std::max<int64_t>(1, 8 * (int64_t)sm / div_up(D, kSliceThreads));
  return std::max<int64_t>(1, div_up(N, want));
}

template <class ST>
cudaError_t grad_typed(const RmsGradArgs& a, int sm, cudaStream_t s) {
  if (a.N == 0) return join(a, 0, s);
  if (a.dx != nullptr) {
    const cudaError_t e = launch_pdl(rms_grad_long_kernel<ST>, std::min<int64_t>(a.N, 4 * (int64_t)sm), kLongThreads, 0, s, a);
    if (e != cudaSuccess) return e;
  }
  if (a.dweight == nullptr) return cudaSuccess;
  const int64_t col_blocks = div_up(a.D, kSliceThreads), rows = slice_rows(a.N, a.D, sm), slices = div_up(a.N, rows);
  const cudaError_t e =
      launch_pdl(rms_grad_slices_kernel<ST>, slices * col_blocks, kSliceThreads, 0, s, a, col_blocks, rows);
  return e == cudaSuccess ? join(a, slices, s) : e;
}

template <class ST>
cudaError_t norm_typed(const RmsArgs& a, int sm, cudaStream_t s) {
  return launch_pdl(rms_long_kernel<ST>, std::min<int64_t>(a.N, 4 * (int64_t)sm), kLongThreads, 0, s, a);
}

}  // namespace

cudaError_t run_rms_norm(const RmsArgs& a, int sm, cudaStream_t s) {
  return a.bf16_io ? norm_typed<bf16>(a, sm, s) : norm_typed<float>(a, sm, s);
}

size_t rms_norm_backward_workspace(int64_t N, int64_t D, int sm) {
  return (size_t)div_up(N, slice_rows(N, D, sm)) * (size_t)D * sizeof(float);
}

cudaError_t run_rms_norm_backward(const RmsGradArgs& a, int sm, cudaStream_t s) {
  return a.bf16_io ? grad_typed<bf16>(a, sm, s) : grad_typed<float>(a, sm, s);
}

cudaError_t status_rms(unsigned int* word, bool clear) { return unit_status(word, clear); }

}  // namespace rlca
