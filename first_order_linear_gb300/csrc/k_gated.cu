// Gated linear recurrence and its gradient.
//
//   a_t = sigma(gate_t),  h_t = k_t a_t h_{t-1} + (1 - a_t) x_t
//   G_t = dh_t + k_{t+1} a_{t+1} G_{t+1},  dx = (1 - a) G,  dgate = a (1 - a) G (k h_{t-1} - x)
//
// with k_t = 0 where step t-1 is flagged.  The state and all arithmetic are
// float32.
#include <algorithm>

#include "policy.h"
#include "reduce.cuh"
#include "trunk.h"

namespace rlca {

namespace {

// sigma(g) and 1 - sigma(g), each to a few units of its own last place: the
// smaller one from the exponential of -|g|, the larger as its difference to 1,
// rounded once.  (As the reciprocal of 1 + e it is biased by a fraction of a
// unit, which the products over thousands of steps next to 1 add up: states of
// 6000 steps came out 2e-5 off.)
struct Gate {
  float a, na;
};
__device__ __forceinline__ Gate gate_of(float g) {
  const float e = expf(-fabsf(g)), less = e * __fdividef(1.f, 1.f + e), more = 1.f - less;
  return g >= 0.f ? Gate{more, less} : Gate{less, more};
}

template <class ST>
__device__ __forceinline__ float load1(const float* p, int64_t i, int64_t n) {
  return in_range(i, n) ? Stor<ST>::ld(p, i) : 0.f;
}
template <class ST>
__device__ __forceinline__ void store1(float* p, int64_t i, int64_t n, float v) {
  if (in_range(i, n)) Stor<ST>::st(p, i, v);
}

__device__ __forceinline__ int row_length(const GatedArgs& a, int64_t e) {
  return a.lengths == nullptr ? (int)a.T : min(max(a.lengths[e], 0), (int)a.T);
}
__device__ __forceinline__ bool flagged(const GatedArgs& a, int64_t row) {
  return (a.terminated != nullptr && a.terminated[row] != 0) || (a.truncated != nullptr && a.truncated[row] != 0);
}

// ---------------------------------------------------------------------------
// a thread a channel, one step after the other
// ---------------------------------------------------------------------------
constexpr int kSerialThreads = 128;

template <class ST>
__global__ void __launch_bounds__(kSerialThreads) gated_serial_kernel(GatedArgs a) {
  pdl_trigger();
  pdl_wait();
  const int64_t n = a.E * a.T, total = a.E * a.D;
  for (int64_t i = (int64_t)blockIdx.x * kSerialThreads + threadIdx.x; i < total; i += (int64_t)gridDim.x * kSerialThreads) {
    const int64_t e = i / a.D, c = i % a.D;
    const int len = row_length(a, e);
    float h = a.state != nullptr ? a.state[i] : 0.f;
    for (int t = 0; t < len; ++t) {
      const int64_t row = e * a.step_e + t * a.step_t;
      const Gate g = gate_of(load1<ST>(a.gate, row * a.gate_stride + c, n * a.gate_stride));
      const float b = g.na * load1<ST>(a.x, row * a.x_stride + c, n * a.x_stride);
      h = t > 0 && flagged(a, row - a.step_t) ? b : fmaf(g.a, h, b);
      store1<ST>(a.h, row * a.D + c, n * a.D, h);
    }
    for (int64_t t = len; t < a.T; ++t) store1<ST>(a.h, (e * a.step_e + t * a.step_t) * a.D + c, n * a.D, 0.f);
    if (len > 0 && flagged(a, e * a.step_e + (len - 1) * a.step_t)) h = 0.f;
    if (a.last != nullptr) a.last[i] = h;
  }
}

template <class ST>
__global__ void __launch_bounds__(kSerialThreads) gated_grad_serial_kernel(GatedArgs a) {
  pdl_trigger();
  pdl_wait();
  const int64_t n = a.E * a.T, total = a.E * a.D;
  for (int64_t i = (int64_t)blockIdx.x * kSerialThreads + threadIdx.x; i < total; i += (int64_t)gridDim.x * kSerialThreads) {
    const int64_t e = i / a.D, c = i % a.D;
    const int len = row_length(a, e);
    for (int64_t t = len; t < a.T; ++t) {
      const int64_t row = e * a.step_e + t * a.step_t;
      store1<ST>(a.dx, row * a.dx_stride + c, n * a.dx_stride, 0.f);
      store1<ST>(a.dgate, row * a.dgate_stride + c, n * a.dgate_stride, 0.f);
    }
    float u = a.d_last != nullptr ? a.d_last[i] : 0.f;
    if (len > 0 && flagged(a, e * a.step_e + (len - 1) * a.step_t)) u = 0.f;
    for (int t = len - 1; t >= 0; --t) {
      const int64_t row = e * a.step_e + t * a.step_t;
      const Gate g = gate_of(load1<ST>(a.gate, row * a.gate_stride + c, n * a.gate_stride));
      const float x = load1<ST>(a.x, row * a.x_stride + c, n * a.x_stride);
      const float G = load1<ST>(a.dh, row * a.dh_stride + c, n * a.dh_stride) + u;
      const bool cut = t > 0 && flagged(a, row - a.step_t);
      float before = 0.f;
      if (!cut)
        before = t > 0 ? load1<ST>(a.in_h, (row - a.step_t) * a.h_stride + c, n * a.h_stride)
                       : (a.state != nullptr ? a.state[i] : 0.f);
      const float d = g.na * G;
      store1<ST>(a.dx, row * a.dx_stride + c, n * a.dx_stride, d);
      store1<ST>(a.dgate, row * a.dgate_stride + c, n * a.dgate_stride, g.a * d * (before - x));
      u = cut ? 0.f : g.a * G;
    }
    if (a.d_state != nullptr) a.d_state[i] = u;
  }
}

template <class K>
cudaError_t launch_serial(K kernel, const GatedArgs& a, int sm, cudaStream_t s) {
  const int64_t grid = std::min<int64_t>(div_up(a.E * a.D, kSerialThreads), (int64_t)sm * 16);
  return launch_pdl(kernel, grid, kSerialThreads, 0, s, a);
}

}  // namespace

cudaError_t run_gated_scan(const GatedArgs& a, int sm, cudaStream_t s) {
  return launch_serial(a.bf16_io ? gated_serial_kernel<bf16> : gated_serial_kernel<float>, a, sm, s);
}

cudaError_t run_gated_scan_backward(const GatedArgs& a, int sm, cudaStream_t s) {
  return launch_serial(a.bf16_io ? gated_grad_serial_kernel<bf16> : gated_grad_serial_kernel<float>, a, sm, s);
}

cudaError_t status_gated(unsigned int* word, bool clear) { return unit_status(word, clear); }

}  // namespace rlca
