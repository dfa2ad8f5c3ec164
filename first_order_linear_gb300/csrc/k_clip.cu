// Global gradient norm over many tensors, and the tensors scaled by it.
#include <algorithm>

#include "policy.h"
#include "reduce.cuh"
#include "rlca.h"

namespace rlca {

namespace {

constexpr int kClipThreads = 256;
// elements of one tensor that one CTA takes at a time
constexpr int64_t kClipChunk = 32768;
// tensors of one launch: their table travels as a kernel parameter (of at
// most 32,764 bytes), so a call writes no device memory for it
constexpr int kClipTensors = 1000;

struct ClipTable {
  const void* grad[kClipTensors];
  void* out[kClipTensors];
  int64_t size[kClipTensors];  // elements; negative: bfloat16
  // first chunk of each tensor (chunks of all tensors are numbered in a row)
  uint32_t first[kClipTensors + 1];
  int count;
};
static_assert(sizeof(ClipTable) <= 32764 - 64, "kernel parameters");

struct ClipItem {
  const void* grad;
  void* out;
  int64_t at, n;  // first element and number of elements
  bool bf16_io;
};

// the piece of a tensor that chunk `chunk` of the launch is
__device__ __forceinline__ ClipItem clip_item(const ClipTable& t, uint32_t chunk) {
  int lo = 0, hi = t.count;  // first[lo] <= chunk < first[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (t.first[mid] <= chunk) lo = mid;
    else hi = mid;
  }
  const int64_t size = t.size[lo] < 0 ? -t.size[lo] : t.size[lo];
  ClipItem it;
  it.grad = t.grad[lo];
  it.out = t.out[lo];
  it.at = (int64_t)(chunk - t.first[lo]) * kClipChunk;
  it.n = min(kClipChunk, size - it.at);
  it.bf16_io = t.size[lo] < 0;
  return it;
}

__device__ __forceinline__ float load_any(const void* p, int64_t i, bool bf) {
  return bf ? Stor<bf16>::ld(static_cast<const float*>(p), i) : static_cast<const float*>(p)[i];
}

// partials[CTA] = sum of squares over the CTA's chunks
__global__ void __launch_bounds__(kClipThreads) clip_squares_kernel(const __grid_constant__ ClipTable t, double* partials) {
  pdl_trigger();
  pdl_wait();
  __shared__ double scratch[32];
  double total = 0.0;
  for (uint32_t chunk = blockIdx.x; chunk < t.first[t.count]; chunk += gridDim.x) {
    const ClipItem it = clip_item(t, chunk);
    float s = 0.f;
    for (int64_t k = threadIdx.x; k < it.n; k += kClipThreads) {
      const float g = load_any(it.grad, it.at + k, it.bf16_io);
      s += g * g;
    }
    total += (double)s;
  }
  total = cta_sum(total, scratch);
  if (threadIdx.x == 0) partials[blockIdx.x] = total;
}

__global__ void __launch_bounds__(kClipThreads) clip_norm_kernel(const double* partials, int64_t n, float* norm) {
  pdl_trigger();
  pdl_wait();
  __shared__ double scratch[32];
  double total = 0.0;
  for (int64_t k = threadIdx.x; k < n; k += kClipThreads) total += partials[k];
  total = cta_sum(total, scratch);
  if (threadIdx.x == 0) *norm = (float)sqrt(total);
}

__global__ void __launch_bounds__(kClipThreads)
    clip_scale_kernel(const __grid_constant__ ClipTable t, const float* norm, float max_norm, float eps) {
  pdl_trigger();
  pdl_wait();
  const float n = *norm;
  const float scale = isfinite(n) ? fminf(1.f, max_norm / (n + eps)) : 1.f;
  for (uint32_t chunk = blockIdx.x; chunk < t.first[t.count]; chunk += gridDim.x) {
    const ClipItem it = clip_item(t, chunk);
    if (scale == 1.f && it.out == it.grad) continue;
    for (int64_t k = threadIdx.x; k < it.n; k += kClipThreads) {
      const float g = load_any(it.grad, it.at + k, it.bf16_io) * scale;
      if (it.bf16_io) Stor<bf16>::st(static_cast<float*>(it.out), it.at + k, g);
      else static_cast<float*>(it.out)[it.at + k] = g;
    }
  }
}

int clip_grid(int sm_count) { return 8 * sm_count; }

}  // namespace

size_t clip_workspace(int64_t count, int sm_count) {
  return (size_t)std::max<int64_t>(1, div_up(count, kClipTensors)) * (size_t)clip_grid(sm_count) * sizeof(double);
}

cudaError_t run_clip_grads(const ClipArgs& a, int sm_count, cudaStream_t s) {
  const int grid = clip_grid(sm_count);
  // the next table of up to kClipTensors tensors (empty ones left out); a
  // device's memory holds far fewer than 2^32 chunks
  const auto fill = [&](int64_t k, ClipTable& t) {
    t.count = 0;
    int64_t chunks = 0;
    for (; k < a.count && t.count < kClipTensors; ++k) {
      if (a.sizes[k] == 0) continue;
      t.grad[t.count] = a.grads[k];
      t.out[t.count] = a.outs ? a.outs[k] : nullptr;
      t.size[t.count] = (a.dtypes[k] & RLCA_BF16) ? -a.sizes[k] : a.sizes[k];
      t.first[t.count++] = (uint32_t)chunks;
      chunks += div_up(a.sizes[k], kClipChunk);
    }
    t.first[t.count] = (uint32_t)chunks;
    return k;
  };
  ClipTable t;
  int64_t partials = 0;
  for (int64_t k = 0; k < a.count;) {
    k = fill(k, t);
    if (t.count == 0) continue;
    const int64_t g = std::min<int64_t>(grid, t.first[t.count]);
    const cudaError_t e = launch_pdl(clip_squares_kernel, g, kClipThreads, 0, s, t, a.ws + partials);
    if (e != cudaSuccess) return e;
    partials += g;
  }
  cudaError_t e = launch_pdl(clip_norm_kernel, 1, kClipThreads, 0, s, (const double*)a.ws, partials, a.norm);
  if (e != cudaSuccess || a.outs == nullptr) return e;
  for (int64_t k = 0; k < a.count;) {
    k = fill(k, t);
    if (t.count == 0) continue;
    const int64_t g = std::min<int64_t>(grid, t.first[t.count]);
    e = launch_pdl(clip_scale_kernel, g, kClipThreads, 0, s, t, (const float*)a.norm, a.max_norm, a.eps);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t status_clip(unsigned int* word, bool clear) { return unit_status(word, clear); }

}  // namespace rlca
