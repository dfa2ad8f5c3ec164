// Gated linear recurrence and its gradient.
//
//   a_t = sigma(gate_t),  h_t = k_t a_t h_{t-1} + (1 - a_t) x_t
//   G_t = dh_t + k_{t+1} a_{t+1} G_{t+1},  dx = (1 - a) G,  dgate = a (1 - a) G (k h_{t-1} - x)
//
// with k_t = 0 where step t-1 is flagged.  The state and all arithmetic are
// float32.  A step reads two elements a channel and writes one, its gradient
// reads four and writes two: both are bound by HBM where the rows are many or
// long and aligned -- bfloat16, 256 x 512 x 1024: 125 us, 0.95 of the measured
// copy rate; 16 x 4096 x 2048 131 us, 0.90; one row of 65536 x 4096 in clusters
// 299 us, 0.79; the gradient, 32 x 4096 x 2048: 528 us, 6.1 TB/s, 0.90; float32
// 16 x 1024 x 2048 0.88 and 0.94.
#include <algorithm>
#include <initializer_list>
#include <type_traits>

#include "policy.h"
#include "reduce.cuh"
#include "tma.cuh"
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
template <class ST>
struct Sigma {
  __device__ __forceinline__ static Gate of(float g) {
    const float e = expf(-fabsf(g)), less = e * __fdividef(1.f, 1.f + e), more = 1.f - less;
    return g >= 0.f ? Gate{more, less} : Gate{less, more};
  }
};
// bfloat16 gates: 1 - sigma from one exponential and one reciprocal at either
// sign; sigma is that reciprocal itself below 0, where it keeps its digits
// however small it is (the gradient of a shut gate is proportional to it), and
// the difference to 1 above, unbiased.  The difference alone would leave of a
// gate of -10 three digits, of -17 none; the selection costs 1 to 3% (8 of 299 us
// on one row of 65536 x 4096; one Newton step of the reciprocal instead 14 us).
// The short exponential's error, (2 + 1.2 |g|) 2^-23 of the value, is far below
// the gate's own rounding.  (The exponent is bounded so that the product stays a
// number: a gate below -86 counts as one of -86, which lets 2^-125 through.)
template <>
struct Sigma<bf16> {
  __device__ __forceinline__ static Gate of(float g) {
    float t = g * -1.44269504f, r;
    asm("min.NaN.f32 %0, %0, %1;" : "+f"(t) : "f"(125.f));
    asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(t));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + t));
    const float na = t * r;
    return {g < 0.f ? r : 1.f - na, na};
  }
};

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
      const Gate g = Sigma<ST>::of(load1<ST>(a.gate, row * a.gate_stride + c, n * a.gate_stride));
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
      const Gate g = Sigma<ST>::of(load1<ST>(a.gate, row * a.gate_stride + c, n * a.gate_stride));
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

// The same for a few steps of rows on 16-byte boundaries, a thread a vector of
// channels: one step of acting, or a few tokens at once.
constexpr int kStepThreads = 128;

// 16 bytes of elements
__device__ __forceinline__ void widen(const uint4& r, float (&v)[4]) {
  v[0] = __uint_as_float(r.x), v[1] = __uint_as_float(r.y), v[2] = __uint_as_float(r.z), v[3] = __uint_as_float(r.w);
}
__device__ __forceinline__ void widen(const uint4& r, float (&v)[8]) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) v[2 * k] = __uint_as_float(w[k] << 16), v[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
}

template <class ST>
__global__ void __launch_bounds__(kStepThreads) gated_step_kernel(GatedArgs a, int64_t blocks) {
  constexpr int VE = 16 / Stor<ST>::kBytes;
  pdl_trigger();
  pdl_wait();
  const int64_t e = blockIdx.x / blocks, c = ((blockIdx.x % blocks) * kStepThreads + threadIdx.x) * VE;
  if (c >= a.D) return;
  const int64_t n = a.E * a.T, i = e * a.D + c;
  const int len = row_length(a, e);
  float h[VE];
#pragma unroll
  for (int k = 0; k < VE; k += 4) {
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (a.state != nullptr && span_in_range(i + k, 4, a.E * a.D)) s = *reinterpret_cast<const float4*>(a.state + i + k);
    h[k] = s.x, h[k + 1] = s.y, h[k + 2] = s.z, h[k + 3] = s.w;
  }
  bool cut = false;
  constexpr int kAhead = 4;  // steps whose loads are on their way together
  for (int t0 = 0; t0 < a.T; t0 += kAhead) {
    uint4 xs[kAhead], gs[kAhead];
    bool ends[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int64_t row = e * a.step_e + (t0 + u) * a.step_t;
      xs[u] = gs[u] = make_uint4(0u, 0u, 0u, 0u);
      ends[u] = false;
      if (t0 + u >= len) continue;
      const auto at = [&](const float* p, int64_t stride) {
        return reinterpret_cast<const uint4*>(reinterpret_cast<const unsigned char*>(p) + (row * stride + c) * Stor<ST>::kBytes);
      };
      if (span_in_range(row * a.x_stride + c, VE, n * a.x_stride)) xs[u] = __ldg(at(a.x, a.x_stride));
      if (span_in_range(row * a.gate_stride + c, VE, n * a.gate_stride)) gs[u] = __ldg(at(a.gate, a.gate_stride));
      ends[u] = flagged(a, row);
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int t = t0 + u;
      if (t >= a.T) break;
      const int64_t row = e * a.step_e + t * a.step_t;
      float v[VE], g[VE];
      widen(xs[u], v);
      widen(gs[u], g);
      if (t < len) {
#pragma unroll
        for (int k = 0; k < VE; ++k) {
          const Gate s = Sigma<ST>::of(g[k]);
          h[k] = v[k] = cut ? s.na * v[k] : fmaf(s.a, h[k], s.na * v[k]);
        }
        cut = ends[u];
      } else {
#pragma unroll
        for (int k = 0; k < VE; ++k) v[k] = 0.f;
      }
      if (span_in_range(row * a.D + c, VE, n * a.D)) {
        if constexpr (VE == 8) Stor<ST>::st8(a.h, row * a.D + c, v);
        else Stor<ST>::st4(a.h, row * a.D + c, v);
      }
    }
  }
  if (a.last == nullptr) return;
#pragma unroll
  for (int k = 0; k < VE; k += 4)
    if (span_in_range(i + k, 4, a.E * a.D))
      *reinterpret_cast<float4*>(a.last + i + k) = cut ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(h[k], h[k + 1], h[k + 2], h[k + 3]);
}

template <class ST>
__global__ void __launch_bounds__(kStepThreads) gated_grad_step_kernel(GatedArgs a, int64_t blocks) {
  constexpr int VE = 16 / Stor<ST>::kBytes;
  pdl_trigger();
  pdl_wait();
  const int64_t e = blockIdx.x / blocks, c = ((blockIdx.x % blocks) * kStepThreads + threadIdx.x) * VE;
  if (c >= a.D) return;
  const int64_t n = a.E * a.T, i = e * a.D + c;
  const int len = row_length(a, e);
  const auto load = [&](const float* p, int64_t row, int64_t stride) {
    if (!span_in_range(row * stride + c, VE, n * stride)) return make_uint4(0u, 0u, 0u, 0u);
    return __ldg(reinterpret_cast<const uint4*>(reinterpret_cast<const unsigned char*>(p) + (row * stride + c) * Stor<ST>::kBytes));
  };
  const auto store = [&](float* p, int64_t row, int64_t stride, const float* v) {
    if (!span_in_range(row * stride + c, VE, n * stride)) return;
    if constexpr (VE == 8) Stor<ST>::st8(p, row * stride + c, v);
    else Stor<ST>::st4(p, row * stride + c, v);
  };
  const auto states = [&](const float* p, float* v) {
#pragma unroll
    for (int k = 0; k < VE; k += 4) {
      float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
      if (p != nullptr && span_in_range(i + k, 4, a.E * a.D)) s = *reinterpret_cast<const float4*>(p + i + k);
      v[k] = s.x, v[k + 1] = s.y, v[k + 2] = s.z, v[k + 3] = s.w;
    }
  };
  float zero[VE], u[VE];
#pragma unroll
  for (int k = 0; k < VE; ++k) zero[k] = 0.f;
  for (int64_t t = len; t < a.T; ++t) {
    store(a.dx, e * a.step_e + t * a.step_t, a.dx_stride, zero);
    store(a.dgate, e * a.step_e + t * a.step_t, a.dgate_stride, zero);
  }
  states(a.d_last, u);
  if (len > 0 && flagged(a, e * a.step_e + (int64_t)(len - 1) * a.step_t)) {
#pragma unroll
    for (int k = 0; k < VE; ++k) u[k] = 0.f;
  }
  constexpr int kAhead = 2;  // steps whose loads are on their way together
  for (int t1 = len - 1; t1 >= 0; t1 -= kAhead) {
    uint4 xs[kAhead], gs[kAhead], ds[kAhead], hs[kAhead];
    bool cut[kAhead];
#pragma unroll
    for (int q = 0; q < kAhead; ++q) {
      const int t = t1 - q;
      const int64_t row = e * a.step_e + t * a.step_t;
      xs[q] = gs[q] = ds[q] = hs[q] = make_uint4(0u, 0u, 0u, 0u);
      cut[q] = false;
      if (t < 0) continue;
      xs[q] = load(a.x, row, a.x_stride);
      gs[q] = load(a.gate, row, a.gate_stride);
      ds[q] = load(a.dh, row, a.dh_stride);
      if (t > 0) {
        hs[q] = load(a.in_h, row - a.step_t, a.h_stride);
        cut[q] = flagged(a, row - a.step_t);
      }
    }
#pragma unroll
    for (int q = 0; q < kAhead; ++q) {
      const int t = t1 - q;
      if (t < 0) break;
      float x[VE], g[VE], d[VE], before[VE];
      widen(xs[q], x);
      widen(gs[q], g);
      widen(ds[q], d);
      widen(hs[q], before);
      if (t == 0) states(a.state, before);
#pragma unroll
      for (int k = 0; k < VE; ++k) {
        const Gate s = Sigma<ST>::of(g[k]);
        const float G = d[k] + u[k], dx = s.na * G;
        g[k] = s.a * dx * ((cut[q] ? 0.f : before[k]) - x[k]);
        x[k] = dx;
        u[k] = cut[q] ? 0.f : s.a * G;
      }
      store(a.dx, e * a.step_e + t * a.step_t, a.dx_stride, x);
      store(a.dgate, e * a.step_e + t * a.step_t, a.dgate_stride, g);
    }
  }
  if (a.d_state == nullptr) return;
#pragma unroll
  for (int k = 0; k < VE; k += 4)
    if (span_in_range(i + k, 4, a.E * a.D)) *reinterpret_cast<float4*>(a.d_state + i + k) = make_float4(u[k], u[k + 1], u[k + 2], u[k + 3]);
}

// ---------------------------------------------------------------------------
// Tiles: a CTA walks the steps of 64 channels of a row in tiles of a few steps
// a warp, a lane two channels, whose arithmetic is paired.  A thread scans its
// steps from 0 and keeps, for each, the value and the product of gates that
// the state before them still meets; the warps' maps (product, value) meet in
// shared memory, and one multiply-add a step brings the state in.  That is 19
// instructions an element forward and 28 backward; where HBM does not bound it,
// a tile's chain of waits does (50% of the issue slots, 4 CTAs an SM: copies in
// flight, the barrier, the fold).  Behind a flagged step nothing of the state before it arrives, whatever it holds: flags
// are the same for all channels, so that is a matter of branches and not of
// products with 0.
//
// Where the rows alone leave SMs idle, a cluster of CTAs shares a row: its
// CTAs take the tiles of a round side by side and send each other their maps,
// which are waited for by their bytes.
// ---------------------------------------------------------------------------
constexpr int kCols = 64, kMaxShare = 8;

// two channels' values
using V2 = uint64_t;
__device__ __forceinline__ V2 v2(float lo, float hi) {
  V2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 apart(V2 v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ V2 fma2(V2 a, V2 b, V2 c) {
  V2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ V2 mul2(V2 a, V2 b) {
  V2 d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ V2 add2(V2 a, V2 b) {
  V2 d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// two channels' elements as they lie in memory
template <class ST>
struct Two;
template <>
struct Two<float> {
  V2 raw;
  __device__ __forceinline__ static Two pair(const unsigned char* at) { return {*reinterpret_cast<const V2*>(at)}; }
  __device__ __forceinline__ static Two split(const unsigned char* at) {  // 32 channels apart
    return {v2(*reinterpret_cast<const float*>(at), *reinterpret_cast<const float*>(at + 128))};
  }
  __device__ __forceinline__ V2 wide() const { return raw; }
  __device__ __forceinline__ void sigma(V2* a, V2* na) const {
    const float2 g = apart(raw);
    const Gate s = Sigma<float>::of(g.x), t = Sigma<float>::of(g.y);
    *a = v2(s.a, t.a), *na = v2(s.na, t.na);
  }
};
template <>
struct Two<bf16> {
  uint32_t raw;
  __device__ __forceinline__ static Two pair(const unsigned char* at) { return {*reinterpret_cast<const uint32_t*>(at)}; }
  __device__ __forceinline__ static Two split(const unsigned char* at) {
    return {*reinterpret_cast<const uint16_t*>(at) | (uint32_t)*reinterpret_cast<const uint16_t*>(at + 64) << 16};
  }
  __device__ __forceinline__ V2 wide() const { return v2(__uint_as_float(raw << 16), __uint_as_float(raw & 0xffff0000u)); }
  // as Sigma<bf16>, the bound put on both gates at once
  __device__ __forceinline__ void sigma(V2* a, V2* na) const {
    uint32_t g;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(g) : "r"(raw), "r"(0xc2adc2adu));  // -86.5
    const float2 u = apart(mul2(Two{g}.wide(), v2(-1.44269504f, -1.44269504f)));
    float2 t, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(t.x) : "f"(u.x));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(t.y) : "f"(u.y));
    const V2 tt = v2(t.x, t.y), one = v2(1.f, 1.f);
    const float2 d = apart(add2(tt, one));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(d.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(d.y));
    *na = mul2(tt, v2(r.x, r.y));
    const float2 open = apart(fma2(*na, v2(-1.f, -1.f), one));
    *a = v2(u.x > 0.f ? r.x : open.x, u.y > 0.f ? r.y : open.y);
  }
};

// two channels' maps of a run of steps: h -> q + p h.  A severed one, of a run
// with a flagged step, is marked by a NaN in both p that no arithmetic gives (its
// results are 0x7fffffff).
struct Map2 {
  V2 p, q;
};
constexpr V2 kSevered = ~V2(0);
__device__ __forceinline__ Map2 identity() { return {v2(1.f, 1.f), 0}; }
__device__ __forceinline__ bool severed(const Map2& m) { return (uint32_t)m.p == (uint32_t)kSevered; }
__device__ __forceinline__ V2 pass(const Map2& m, V2 h) { return severed(m) ? m.q : fma2(m.p, h, m.q); }
// `then` behind `first`
__device__ __forceinline__ Map2 chain(const Map2& then, const Map2& first) {
  if (severed(then)) return then;
  return {severed(first) ? first.p : mul2(then.p, first.p), fma2(then.p, first.q, then.q)};
}
// one step, of gates s and input b, behind `first`
__device__ __forceinline__ Map2 step(V2 s, V2 b, const Map2& first) {
  return {severed(first) ? first.p : mul2(s, first.p), fma2(s, first.q, b)};
}

// Products of gates are above 0 however far below float32's least they lie, and
// an infinity stays one through any of them; the rounded product, 0, would make
// it NaN.  So the maps that threads hand each other keep products of 2^-126 at
// least (which moves no finite value by more than that of it), and a thread's own
// products are left out (`meeting`) where the value in front is not finite.  (One
// row of 65536 x 4096 5 us of 299; passing every map with regard to it 45 us.)
__device__ __forceinline__ Map2 lasting(const Map2& m) {
  const float2 p = apart(m.p);
  constexpr float kLeast = 1.17549435e-38f;
  return {severed(m) ? m.p : v2(fmaxf(p.x, kLeast), fmaxf(p.y, kLeast)), m.q};
}
constexpr float kLargest = 3.402823466e38f;
__device__ __forceinline__ bool finite(V2 v) {
  const float2 f = apart(v);
  return fabsf(f.x) <= kLargest && fabsf(f.y) <= kLargest;
}
__device__ __forceinline__ V2 meeting(V2 p, V2 h) {
  if ((uint32_t)p == (uint32_t)kSevered) return p;
  const float2 f = apart(h), r = apart(p);
  return v2(fabsf(f.x) <= kLargest ? r.x : 1.f, fabsf(f.y) <= kLargest ? r.y : 1.f);
}

// carry through the maps of W warps, in order of the steps or against it; at:
// what it is in front of this warp's
template <int W, bool kForward>
__device__ __forceinline__ void fold(const Map2 (*maps)[32], int lane, int warp, bool any_cut, V2* carry, V2* at) {
#pragma unroll
  for (int k = 0; k < W; ++k) {
    const int w = kForward ? k : W - 1 - k;
    if (w == warp) *at = *carry;
    const Map2 m = maps[w][lane];
    *carry = any_cut ? pass(m, *carry) : fma2(m.p, *carry, m.q);
  }
}

// a map into a peer's shared memory, its 16 bytes counted on the peer's barrier
__device__ __forceinline__ void send(Map2* mine, uint64_t* bar, int rank, const Map2& m) {
  uint32_t at, on;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(mine)), "r"(rank));
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(on) : "r"(smem_u32(bar)), "r"(rank));
  asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v2.b64 [%0], {%1, %2}, [%3];" ::"r"(at), "l"(m.p),
               "l"(m.q), "r"(on)
               : "memory");
}
__device__ __forceinline__ void cluster_meet() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// The tensor maps [D, T, E] of the arrays that tiles are copied from
struct GatedMaps {
  CUtensorMap in[4];
};
__device__ __forceinline__ void tile_load(void* to, const CUtensorMap* map, int c, int t, int e, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          smem_u32(to)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c), "r"(t), "r"(e), "r"(smem_u32(bar))
      : "memory");
}

// Where the rows of every array start on 16-byte boundaries (kBulk), a tile of
// an array is one tensor copy, and a lane's channels are next to each other.
// Other rows are copied in 16-byte vectors, from the boundary in front of them
// on -- 16 bytes that hold any byte of the row are readable as a whole.  (A bulk
// copy a row has to be issued thread by thread, some 12 instructions each.)
// Their pitch in shared memory is the matrix's modulo 16 bytes, so that a row's
// first column stays as far behind a boundary as it is in memory and a column
// lies at one pitch in all of them.  A lane's channels are 32 apart there.
template <class ST, bool kBulk, int L>
struct TileRows {
  static constexpr int kBytes = Stor<ST>::kBytes, kRow = kCols * kBytes;
  // (a row and what lies in front of and behind it in its boundaries)
  static constexpr int kLeast = kRow + 2 * (16 - kBytes), kMost = kLeast + 16 - kBytes;
  static constexpr int kTile = kBulk ? L * kRow : L * kMost + 16;
  // bytes from step to step of an array whose steps lie `step` bytes apart
  __device__ static uint32_t pitch(int64_t step) { return kBulk ? kRow : kLeast + (((uint32_t)step - kLeast) & 15); }
};

// Copies the tiles of one array by vectors: a thread one vector of some rows,
// each at the same place behind its boundary in every tile.
template <class ST, int L, int THREADS>
struct RowCopy {
  using R = TileRows<ST, false, L>;
  static constexpr int V = R::kRow / 16 + 1;                    // vectors that a row can touch
  static constexpr int kRows = THREADS / V, kTurns = (L + kRows - 1) / kRows;  // rows at a time
  uintptr_t at = 0;  // this thread's first vector in the next tile, shift included
  int64_t bytes = 0;
  uint32_t to = 0, pitch = 0;
  int row = L, past = 0;  // its first row; what the shift has to exceed for the vector to hold a column
  uintptr_t lo = 0, hi = 0;
  // array k; `first`: the first tile's first step
  __device__ void start(const GatedArgs& a, int k, const float* p, int64_t stride, int64_t e, int64_t c0, int first) {
    const int v = threadIdx.x % V;
    row = threadIdx.x / V < kRows ? threadIdx.x / V : L;
    bytes = a.step_t * stride * R::kBytes;
    pitch = R::pitch(bytes);
    at = (uintptr_t)p + ((e * a.step_e + first * a.step_t) * stride + c0) * R::kBytes;
    to = k * R::kTile + (uint32_t)(at & 15) + row * pitch + 16 * v;
    at += row * bytes + 16 * v;
    past = 16 * v - (int)min((int64_t)kCols, a.D - c0) * R::kBytes;
    if constexpr (kIndexCheck) lo = (uintptr_t)p, hi = lo + (uintptr_t)(a.E * a.T * stride) * R::kBytes;
  }
  // the tile of steps t .. t + L - 1, of which those in [0, len) are there; `move`: steps to the next one copied
  __device__ __forceinline__ void next(uint32_t stage, int t, int len, int move) {
    uintptr_t from = at;
    uint32_t dst = stage + to;
#pragma unroll
    for (int q = 0; q < kTurns; ++q) {
      const int r = row + q * kRows;
      if (r < L && t + r >= 0 && t + r < len && (int)(from & 15) > past) {
        const uintptr_t vec = from & ~(uintptr_t)15;
        if (!kIndexCheck || in_range((int64_t)(max(vec, lo) - lo), (int64_t)(hi - lo)))
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst & ~15u), "l"(vec) : "memory");
      }
      from += kRows * bytes;
      dst += kRows * pitch;
    }
    at += move * bytes;
  }
};
// an arrival on `bar` when this thread's copies so far have landed
__device__ __forceinline__ void copies_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// A lane's two channels of the warp's steps of a tile.  Tiles are whole multiples of 16 bytes in steps of any matrix, so a
// step lies at the same place in all of them.
template <class ST, bool kBulk, int L>
struct Reader {
  using R = TileRows<ST, kBulk, L>;
  static_assert(L * R::kBytes % 16 == 0, "a step's place in its 16 bytes does not change from tile to tile");
  uint32_t at, pitch;
  // array k from step r of a tile on; `row` of the matrix is the first step of one
  __device__ Reader(const GatedArgs& a, int k, int r, int lane, const float* p, int64_t row, int64_t stride, int64_t c0)
      : pitch(R::pitch(a.step_t * stride * R::kBytes)) {
    at = k * R::kTile + r * pitch + lane * (kBulk ? 2 : 1) * R::kBytes;
    if constexpr (!kBulk) at += ((uint32_t)(uintptr_t)p + (uint32_t)(row * stride + c0) * R::kBytes) & 15;
  }
  __device__ __forceinline__ Two<ST> get(const unsigned char* stage, int i) const {
    if constexpr (kBulk) return Two<ST>::pair(stage + at + i * R::kRow);
    else return Two<ST>::split(stage + at + i * pitch);
  }
};

// What a CTA works on, and where a lane's channels lie.
template <class ST, bool kPairs>
struct Cols {
  int64_t c0;
  int lane;
  int64_t D;
  __device__ int64_t ch(int k) const { return kPairs ? c0 + 2 * lane + k : c0 + lane + 32 * k; }
  __device__ bool on(int k) const { return ch(k) < D; }
  // v, without what channels that are none hold (their columns of a tile are not copied, or 0 by tensor copies)
  __device__ V2 there(V2 v) const {
    if constexpr (kPairs) return v;
    const float2 f = apart(v);
    return v2(on(0) ? f.x : 0.f, on(1) ? f.y : 0.f);
  }
  // the two channels' states in float32 [E, D]
  __device__ V2 state(const float* p, int64_t e, int64_t E) const {
    float v[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int64_t i = e * D + ch(k);
      v[k] = p != nullptr && on(k) && in_range(i, E * D) ? p[i] : 0.f;
    }
    return v2(v[0], v[1]);
  }
  __device__ void store_state(float* p, int64_t e, int64_t E, V2 v) const {
    const float2 f = apart(v);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int64_t i = e * D + ch(k);
      if (p != nullptr && on(k) && in_range(i, E * D)) p[i] = k == 0 ? f.x : f.y;
    }
  }
};

// Writes the warp's steps of a matrix: from `base` on, which moves from round to round.
template <class ST, bool kPairs>
struct Writer {
  unsigned char *base, *at;
  int64_t step, first, last;  // bytes a step; the matrix, for the index check
  bool on[2];
  __device__ Writer(const Cols<ST, kPairs>& cols, const GatedArgs& a, float* p, int64_t stride, int64_t row) {
    base = reinterpret_cast<unsigned char*>(p) + (row * stride + cols.ch(0)) * Stor<ST>::kBytes;
    step = a.step_t * stride * Stor<ST>::kBytes;
    first = (int64_t)p, last = (int64_t)p + a.E * a.T * stride * Stor<ST>::kBytes;
    on[0] = cols.on(0), on[1] = cols.on(1);
  }
  __device__ __forceinline__ void start() { at = base; }
  __device__ __forceinline__ void move(int steps) { base += steps * step; }
  __device__ __forceinline__ void put(V2 v) {
    const float2 f = apart(v);
    if constexpr (kPairs) {
      if (on[0] && span_in_range((int64_t)at - first, 2 * Stor<ST>::kBytes, last - first)) {
        if constexpr (Stor<ST>::kBytes == 4) *reinterpret_cast<V2*>(at) = v;
        else *reinterpret_cast<uint32_t*>(at) = Stor<bf16>::pack2(f.x, f.y);
      }
    } else {
      constexpr int kApart = 32 * Stor<ST>::kBytes;
      if (on[0] && in_range((int64_t)at - first, last - first)) Stor<ST>::st(reinterpret_cast<float*>(at), 0, f.x);
      if (on[1] && in_range((int64_t)at + kApart - first, last - first)) Stor<ST>::st(reinterpret_cast<float*>(at + kApart), 0, f.y);
    }
    at += step;
  }
};

// whether the state before step t counts as 0 (steps in front of `len` only)
__device__ __forceinline__ bool cut_before(const GatedArgs& a, int64_t e, int t, int len) {
  return t > 0 && t < len && flagged(a, e * a.step_e + (t - 1) * a.step_t);
}

// the value in front of a row's steps (behind them, backward)
template <bool kBack, class C>
__device__ __forceinline__ V2 outer_value(const C& cols, const GatedArgs& a, int64_t e, int len) {
  if constexpr (!kBack) return cols.state(a.state, e, a.E);
  if (len > 0 && flagged(a, e * a.step_e + (int64_t)(len - 1) * a.step_t)) return 0;
  return cols.state(a.d_last, e, a.E);
}

// What the CTAs of a row have in shared memory beside the ring, and how their
// maps meet.
template <int W, int STAGES, bool kShared>
struct GatedShared {
  Map2 warp_map[2][W][32];
  Map2 cta_map[2][kShared ? kMaxShare : 1][32];
  uint64_t full[STAGES], maps[2];
};

// The carry in front of this warp's steps (returned) and behind the round's
// (*carry).  Buffers alternate: a peer sends its map of round k + 2 only when it
// has this CTA's of round k + 1, which leaves behind the reads of round k.
template <int W, int STAGES, bool kShared, bool kForward>
__device__ __forceinline__ V2 meet(GatedShared<W, STAGES, kShared>& sh, int round, int rank, int share, bool any_cut, bool* ok, V2* carry) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, buf = round & 1;
  V2 at = *carry;
  if constexpr (!kShared) {
    fold<W, kForward>(sh.warp_map[buf], lane, warp, any_cut, carry, &at);
    return at;
  }
  if (warp == 0) {
    if (lane == 0) mbar_arrive_expect_tx(&sh.maps[buf], (uint32_t)share * 32 * sizeof(Map2));
    Map2 all = sh.warp_map[buf][kForward ? 0 : W - 1][lane];
#pragma unroll
    for (int k = 1; k < W; ++k) all = chain(sh.warp_map[buf][kForward ? k : W - 1 - k][lane], all);
    all = lasting(all);
    for (int r = 0; r < share; ++r) send(&sh.cta_map[buf][rank][lane], &sh.maps[buf], r, all);
  }
  if (*ok) *ok = mbar_wait_bounded<true>(&sh.maps[buf], (round >> 1) & 1);
  for (int k = 0; k < share; ++k) {
    const int r = kForward ? k : share - 1 - k;
    if (r == rank) at = *carry;
    *carry = pass(sh.cta_map[buf][r][lane], *carry);
  }
  for (int k = 0; k < W; ++k) {
    const int w = kForward ? k : W - 1 - k;
    if (w == warp) break;
    at = pass(sh.warp_map[buf][w][lane], at);
  }
  return at;
}

// Rows too few even for clusters are cut into segments: a first launch leaves
// every segment's map, and a segment's CTA starts from the value that the maps in
// front of its steps (behind them, backward) give.  The value in front of all
// segments comes through the workspace too: its buffer may be the one that the
// last segment writes.
__host__ __device__ constexpr int64_t segment_slots(int nseg) { return nseg + 1; }
__device__ __forceinline__ int64_t segment_at(const GatedArgs& a, int64_t unit, int segment) {
  return (unit * segment_slots(a.nseg) + segment) * 32 + (threadIdx.x & 31);
}
__device__ __forceinline__ int64_t segment_maps(const GatedArgs& a) {
  return a.E * ((a.D + kCols - 1) / kCols) * segment_slots(a.nseg) * 32;
}
__device__ __forceinline__ void leave_map(const GatedArgs& a, int64_t unit, int segment, const Map2& m) {
  const int64_t i = segment_at(a, unit, segment);
  if (in_range(i, segment_maps(a))) static_cast<Map2*>(a.ws)[i] = m;
}
__device__ __forceinline__ Map2 segment_map(const GatedArgs& a, int64_t unit, int segment) {
  const int64_t i = segment_at(a, unit, segment);
  return in_range(i, segment_maps(a)) ? static_cast<const Map2*>(a.ws)[i] : identity();
}

// ... through `count` maps from `first` on, one after or in front of the other (eight loads in flight)
template <bool kForward>
__device__ __forceinline__ V2 through_segments(const GatedArgs& a, int64_t unit, int first, int count, V2 carry) {
  constexpr int B = 8;
  for (int q = 0; q < count; q += B) {
    Map2 m[B];
#pragma unroll
    for (int u = 0; u < B; ++u) m[u] = q + u < count ? segment_map(a, unit, kForward ? first + q + u : first - q - u) : identity();
#pragma unroll
    for (int u = 0; u < B; ++u) carry = pass(m[u], carry);
  }
  return carry;
}

template <class ST, int C, int W, int STAGES, bool kBulk, bool kBack, int kResident>
__global__ void __launch_bounds__(32 * W, kResident) gated_map_kernel(GatedArgs a, const __grid_constant__ GatedMaps maps, int) {
  using R = TileRows<ST, kBulk, C * W>;
  constexpr int L = C * W, kArrays = 2;
  extern __shared__ __align__(128) unsigned char ring_tiles[];  // [STAGES][x (dh), gate]
  __shared__ __align__(16) GatedShared<W, STAGES, false> sh;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t blocks = (a.D + kCols - 1) / kCols, unit = blockIdx.x / a.nseg, e = unit / blocks;
  const int part = blockIdx.x % a.nseg;
  const Cols<ST, kBulk> cols{(unit % blocks) * kCols, lane, a.D};
  pdl_trigger();
  if (threadIdx.x == 0) {
    for (int i = 0; i < STAGES; ++i) mbar_init(&sh.full[i], kBulk ? 1 : 32 * W);
    mbar_fence_init();
  }
  __syncthreads();
  pdl_wait();
  const int begin = part * a.seg_len, len = row_length(a, e), lim = (int)min((int64_t)len, (int64_t)begin + a.seg_len);
  const int ntiles = (max(lim - begin, 0) + L - 1) / L;
  const float* const p = kBack ? a.dh : a.x;
  const int64_t stride = kBack ? a.dh_stride : a.x_stride;
  // in the order of the steps, or the last tile first
  const int first = kBack ? begin + (ntiles - 1) * L : begin, turn = kBack ? -L : L;
  RowCopy<ST, L, 32 * W> copy[kArrays];
  if constexpr (!kBulk) {
    copy[0].start(a, 0, p, stride, e, cols.c0, first);
    copy[1].start(a, 1, a.gate, a.gate_stride, e, cols.c0, first);
  }
  const auto fill = [&](int stage, int j) {
    if (!in_range(stage, STAGES)) return;
    unsigned char* to = ring_tiles + (size_t)stage * kArrays * R::kTile;
    if constexpr (kBulk) {
      if (threadIdx.x != 0) return;
      mbar_arrive_expect_tx(&sh.full[stage], kArrays * R::kTile);
      tile_load(to, &maps.in[kBack ? 2 : 0], (int)cols.c0, first + j * turn, (int)e, &sh.full[stage]);
      tile_load(to + R::kTile, &maps.in[1], (int)cols.c0, first + j * turn, (int)e, &sh.full[stage]);
    } else {
#pragma unroll
      for (int i = 0; i < kArrays; ++i) copy[i].next(smem_u32(to), first + j * turn, len, turn);
      copies_arrive(&sh.full[stage]);
    }
  };
  for (int j = 0; j < STAGES - 1 && j < ntiles; ++j) fill(j, j);
  FillRing<STAGES> ring;
  const int64_t tile0 = e * a.step_e + (int64_t)begin * a.step_t;
  const Reader<ST, kBulk, L> xs(a, 0, warp * C, lane, p, tile0, stride, cols.c0);
  const Reader<ST, kBulk, L> gs(a, 1, warp * C, lane, a.gate, tile0, a.gate_stride, cols.c0);
  const bool flags = a.terminated != nullptr || a.truncated != nullptr;
  int t0 = first + warp * C;
  bool cut_next = flags && lane < C && cut_before(a, e, t0 + lane, len);
  Map2 all = identity();
  for (int j = 0; j < ntiles; ++j, t0 += turn) {
    const int real = min(max(lim - t0, 0), C);
    uint32_t cut = 0;
    if (flags) {
      cut = __ballot_sync(kFullMask, cut_next);
      if (lane < C) cut_next = cut_before(a, e, t0 + turn + lane, len);
    }
    if (ring.ok && j + STAGES - 1 < ntiles) fill(ring.fill_stage(), j + STAGES - 1);
    if (ring.ok) ring.ok = mbar_wait_bounded(&sh.full[ring.stage], ring.phase);
    const unsigned char* tile = ring_tiles + (size_t)ring.stage * kArrays * R::kTile;
    ring.next();
    Map2 m = identity();
#pragma unroll
    for (int q = 0; q < C; ++q) {
      const int i = kBack ? C - 1 - q : q;
      if (i >= real) continue;
      V2 s, ns;
      gs.get(tile, i).sigma(&s, &ns);
      const V2 v = xs.get(tile, i).wide();
      const bool here = (cut >> i) & 1;
      if constexpr (kBack) {
        if (here) m = {kSevered, 0};
        else m = {severed(m) ? m.p : mul2(m.p, s), mul2(s, add2(v, m.q))};
      } else {
        if (here) m = {kSevered, mul2(ns, v)};
        else m = step(s, mul2(ns, v), m);
      }
    }
    sh.warp_map[j & 1][warp][lane] = lasting(m);
    __syncthreads();
    if (warp == 0) {
#pragma unroll
      for (int k = 0; k < W; ++k) all = chain(sh.warp_map[j & 1][kBack ? W - 1 - k : k][lane], all);
    }
  }
  if (warp == 0) {
    leave_map(a, unit, part, lasting(all));
    if (part == 0) leave_map(a, unit, a.nseg, {kSevered, outer_value<kBack>(cols, a, e, len)});
  }
  // (copies still on their way after a wait gave up land before the CTA ends)
  if (kBulk && !ring.ok && threadIdx.x == 0)
    for (int i = 0; i < STAGES; ++i) mbar_wait_bounded(&sh.full[i], ring.last_fill(i));
  if constexpr (!kBulk) asm volatile("cp.async.wait_all;" ::: "memory");
}

template <class ST, int C, int W, int STAGES, bool kBulk, bool kShared, int kResident>
__global__ void __launch_bounds__(32 * W, kResident) gated_tile_kernel(GatedArgs a, const __grid_constant__ GatedMaps maps, int share) {
  using R = TileRows<ST, kBulk, C * W>;
  constexpr int L = C * W, kArrays = 2;
  extern __shared__ __align__(128) unsigned char ring_tiles[];  // [STAGES][x, gate]
  __shared__ __align__(16) GatedShared<W, STAGES, kShared> sh;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int parts = kShared ? share : a.nseg, part = blockIdx.x % parts, rank = kShared ? part : 0;
  const int64_t blocks = (a.D + kCols - 1) / kCols, unit = blockIdx.x / parts, e = unit / blocks;
  // a row's steps, or a segment's
  const int begin = kShared ? 0 : part * a.seg_len, stop = kShared ? (int)a.T : (int)min(a.T, (int64_t)begin + a.seg_len);
  const Cols<ST, kBulk> cols{(unit % blocks) * kCols, lane, a.D};
  pdl_trigger();
  if (threadIdx.x == 0) {
    for (int i = 0; i < STAGES; ++i) mbar_init(&sh.full[i], kBulk ? 1 : 32 * W);
    mbar_init(&sh.maps[0], 1);
    mbar_init(&sh.maps[1], 1);
    mbar_fence_init();
  }
  if constexpr (kShared) cluster_meet();  // (a peer's memory is written only once it runs)
  else __syncthreads();
  pdl_wait();

  const int len = row_length(a, e), lim = min(len, stop);
  const int ntiles = (max(lim - begin, 0) + L - 1) / L, rounds = (ntiles + share - 1) / share;
  const int mine = ntiles > rank ? (ntiles - rank + share - 1) / share : 0;
  RowCopy<ST, L, 32 * W> copy[kArrays];
  if constexpr (!kBulk) {
    copy[0].start(a, 0, a.x, a.x_stride, e, cols.c0, begin + rank * L);
    copy[1].start(a, 1, a.gate, a.gate_stride, e, cols.c0, begin + rank * L);
  }
  const auto fill = [&](int stage, int j) {
    if (!in_range(stage, STAGES)) return;
    unsigned char* to = ring_tiles + (size_t)stage * kArrays * R::kTile;
    if constexpr (kBulk) {
      if (threadIdx.x != 0) return;
      const int t = begin + (rank + j * share) * L;
      mbar_arrive_expect_tx(&sh.full[stage], kArrays * R::kTile);
      tile_load(to, &maps.in[0], (int)cols.c0, t, (int)e, &sh.full[stage]);
      tile_load(to + R::kTile, &maps.in[1], (int)cols.c0, t, (int)e, &sh.full[stage]);
    } else {
      const int t = begin + (rank + j * share) * L;
#pragma unroll
      for (int i = 0; i < kArrays; ++i) copy[i].next(smem_u32(to), t, len, share * L);
      copies_arrive(&sh.full[stage]);
    }
  };
  for (int j = 0; j < STAGES - 1 && j < mine; ++j) fill(j, j);

  V2 carry = parts > 1 && !kShared ? segment_map(a, unit, parts).q : outer_value<false>(cols, a, e, len);
  if constexpr (!kShared) carry = through_segments<true>(a, unit, 0, part, carry);
  FillRing<STAGES> ring;
  bool met = true;
  int t0 = begin + rank * L + warp * C;  // the warp's first step of the round
  const int64_t row0 = e * a.step_e + t0 * a.step_t, tile0 = e * a.step_e + (int64_t)(begin + rank * L) * a.step_t;
  const Reader<ST, kBulk, L> xs(a, 0, warp * C, lane, a.x, tile0, a.x_stride, cols.c0);
  const Reader<ST, kBulk, L> gs(a, 1, warp * C, lane, a.gate, tile0, a.gate_stride, cols.c0);
  Writer<ST, kBulk> out(cols, a, a.h, a.D, row0);
  const bool flags = a.terminated != nullptr || a.truncated != nullptr;
  bool cut_next = flags && lane < C && cut_before(a, e, t0 + lane, len);
  for (int k = 0; k < rounds; ++k, t0 += share * L) {
    const int real = min(max(lim - t0, 0), C);
    uint32_t cut = 0;
    if (flags) {
      cut = __ballot_sync(kFullMask, cut_next);
      if (lane < C) cut_next = cut_before(a, e, t0 + share * L + lane, len);
    }
    V2 p[C], q[C];
    Map2 m = identity();
    if (k < mine) {
      if (ring.ok && k + STAGES - 1 < mine) fill(ring.fill_stage(), k + STAGES - 1);
      if (ring.ok) ring.ok = mbar_wait_bounded(&sh.full[ring.stage], ring.phase);
      const unsigned char* tile = ring_tiles + (size_t)ring.stage * kArrays * R::kTile;
      ring.next();
      if (cut == 0 && real == C) {
#pragma unroll
        for (int i = 0; i < C; ++i) {
          V2 s, ns;
          gs.get(tile, i).sigma(&s, &ns);
          m.q = q[i] = fma2(s, m.q, mul2(ns, xs.get(tile, i).wide()));
          m.p = p[i] = mul2(m.p, s);
        }
      } else {
#pragma unroll
        for (int i = 0; i < C; ++i) {
          if (i < real) {
            V2 s, ns;
            gs.get(tile, i).sigma(&s, &ns);
            const V2 b = mul2(ns, xs.get(tile, i).wide());
            if ((cut >> i) & 1) m = {kSevered, b};
            else m = step(s, b, m);
          }
          q[i] = m.q;
          p[i] = m.p;
        }
      }
    }
    sh.warp_map[k & 1][warp][lane] = lasting(m);
    const bool any_cut = __syncthreads_or(cut != 0);
    const V2 h = cols.there(meet<W, STAGES, kShared, true>(sh, k, rank, share, any_cut, &met, &carry));
    out.start();
    if (k < mine && real == C && cut == 0 && finite(h)) {
#pragma unroll
      for (int i = 0; i < C; ++i) out.put(fma2(p[i], h, q[i]));
    } else {
      if (!finite(h)) {
#pragma unroll
        for (int i = 0; i < C; ++i) p[i] = meeting(p[i], h);
      }
#pragma unroll
      for (int i = 0; i < C; ++i)
        if (t0 + i < stop) out.put(k < mine && i < real ? pass({p[i], q[i]}, h) : 0);
    }
    out.move(share * L);
  }
  // behind the row's last tile
  for (; t0 < stop; t0 += share * L) {
    out.start();
    for (int i = 0; i < C && t0 + i < stop; ++i) out.put(0);
    out.move(share * L);
  }
  if (warp == 0 && a.last != nullptr && part == (kShared ? 0 : parts - 1)) {
    if (len > 0 && flagged(a, e * a.step_e + (int64_t)(len - 1) * a.step_t)) carry = 0;
    cols.store_state(a.last, e, a.E, carry);
  }
  // (copies still on their way after a wait gave up land before the CTA ends)
  if (kBulk && !ring.ok && threadIdx.x == 0)
    for (int i = 0; i < STAGES; ++i) mbar_wait_bounded(&sh.full[i], ring.last_fill(i));
  if constexpr (!kBulk) asm volatile("cp.async.wait_all;" ::: "memory");
  if constexpr (kShared) cluster_meet();  // no CTA ends while a peer may still write to it
}

template <class ST, int C, int W, int STAGES, bool kBulk, bool kShared, int kResident>
__global__ void __launch_bounds__(32 * W, kResident) gated_grad_tile_kernel(GatedArgs a, const __grid_constant__ GatedMaps maps, int share) {
  using R = TileRows<ST, kBulk, C * W>;
  constexpr int L = C * W, kArrays = 4;
  extern __shared__ __align__(128) unsigned char ring_tiles[];  // [STAGES][x, gate, dh, h one step earlier]
  __shared__ __align__(16) GatedShared<W, STAGES, kShared> sh;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int parts = kShared ? share : a.nseg, part = blockIdx.x % parts, rank = kShared ? part : 0;
  const int64_t blocks = (a.D + kCols - 1) / kCols, unit = blockIdx.x / parts, e = unit / blocks;
  // a row's steps, or a segment's
  const int begin = kShared ? 0 : part * a.seg_len, stop = kShared ? (int)a.T : (int)min(a.T, (int64_t)begin + a.seg_len);
  const Cols<ST, kBulk> cols{(unit % blocks) * kCols, lane, a.D};
  pdl_trigger();
  if (threadIdx.x == 0) {
    for (int i = 0; i < STAGES; ++i) mbar_init(&sh.full[i], kBulk ? 1 : 32 * W);
    mbar_init(&sh.maps[0], 1);
    mbar_init(&sh.maps[1], 1);
    mbar_fence_init();
  }
  if constexpr (kShared) cluster_meet();
  else __syncthreads();
  pdl_wait();

  const int len = row_length(a, e), lim = min(len, stop);
  const int ntiles = (max(lim - begin, 0) + L - 1) / L, rounds = (ntiles + share - 1) / share;
  const int mine = ntiles > rank ? (ntiles - rank + share - 1) / share : 0;
  // the row's last tile first
  const int last_tile = begin + (rank + (mine - 1) * share) * L;
  RowCopy<ST, L, 32 * W> copy[kArrays];
  if constexpr (!kBulk) {
    copy[0].start(a, 0, a.x, a.x_stride, e, cols.c0, last_tile);
    copy[1].start(a, 1, a.gate, a.gate_stride, e, cols.c0, last_tile);
    copy[2].start(a, 2, a.dh, a.dh_stride, e, cols.c0, last_tile);
    copy[3].start(a, 3, a.in_h, a.h_stride, e, cols.c0, last_tile - 1);
  }
  const auto fill = [&](int stage, int j) {
    if (!in_range(stage, STAGES)) return;
    unsigned char* to = ring_tiles + (size_t)stage * kArrays * R::kTile;
    if constexpr (kBulk) {
      if (threadIdx.x != 0) return;
      const int t = last_tile - j * share * L;
      mbar_arrive_expect_tx(&sh.full[stage], kArrays * R::kTile);
#pragma unroll
      for (int i = 0; i < kArrays; ++i)
        tile_load(to + i * R::kTile, &maps.in[i], (int)cols.c0, i == 3 ? t - 1 : t, (int)e, &sh.full[stage]);
    } else {
      const int t = last_tile - j * share * L;
#pragma unroll
      for (int i = 0; i < kArrays; ++i) copy[i].next(smem_u32(to), i == 3 ? t - 1 : t, len, -share * L);
      copies_arrive(&sh.full[stage]);
    }
  };
  for (int j = 0; j < STAGES - 1 && j < mine; ++j) fill(j, j);

  V2 carry = parts > 1 && !kShared ? segment_map(a, unit, parts).q : outer_value<true>(cols, a, e, len);
  if constexpr (!kShared) carry = through_segments<false>(a, unit, parts - 1, parts - 1 - part, carry);
  FillRing<STAGES> ring;
  bool met = true;
  int j = 0;
  int t0 = begin + (rank + (rounds - 1) * share) * L + warp * C;
  const int64_t row0 = e * a.step_e + t0 * a.step_t;
  const auto reader = [&](int i, const float* p, int64_t row, int64_t stride) {
    return Reader<ST, kBulk, L>(a, i, warp * C, lane, p, row, stride, cols.c0);
  };
  const int64_t tile0 = e * a.step_e + (int64_t)(begin + rank * L) * a.step_t;
  const auto xs = reader(0, a.x, tile0, a.x_stride), gs = reader(1, a.gate, tile0, a.gate_stride),
             ds = reader(2, a.dh, tile0, a.dh_stride), hs = reader(3, a.in_h, tile0 - a.step_t, a.h_stride);
  Writer<ST, kBulk> to_x(cols, a, a.dx, a.dx_stride, row0), to_gate(cols, a, a.dgate, a.dgate_stride, row0);
  // behind the row's last tile
  for (int t = t0 + share * L; t < stop; t += share * L) {
    Writer<ST, kBulk> x = to_x, g = to_gate;
    x.move(t - t0), g.move(t - t0);
    x.start(), g.start();
    for (int i = 0; i < C && t + i < stop; ++i) x.put(0), g.put(0);
  }
  const bool flags = a.terminated != nullptr || a.truncated != nullptr;
  bool cut_next = flags && lane < C && cut_before(a, e, t0 + lane, len);
  for (int k = rounds - 1; k >= 0; --k, t0 -= share * L) {
    const int real = min(max(lim - t0, 0), C);
    uint32_t cut = 0;
    if (flags) {
      cut = __ballot_sync(kFullMask, cut_next);
      if (lane < C) cut_next = cut_before(a, e, t0 - share * L + lane, len);
    }
    // a step's G is g + p u, u from behind the chunk; dx = na G, dgate = w G
    V2 p[C], g[C], na[C], w[C];
    Map2 m = identity();
    const V2 minus = v2(-1.f, -1.f);
    if (k < mine) {
      if (ring.ok && j + STAGES - 1 < mine) fill(ring.fill_stage(), j + STAGES - 1);
      if (ring.ok) ring.ok = mbar_wait_bounded(&sh.full[ring.stage], ring.phase);
      const unsigned char* tile = ring_tiles + (size_t)ring.stage * kArrays * R::kTile;
      ring.next();
      ++j;
      if (cut == 0 && real == C && t0 > 0) {
#pragma unroll
        for (int i = C - 1; i >= 0; --i) {
          V2 s;
          gs.get(tile, i).sigma(&s, &na[i]);
          p[i] = m.p;
          g[i] = add2(ds.get(tile, i).wide(), m.q);
          w[i] = mul2(mul2(s, na[i]), fma2(xs.get(tile, i).wide(), minus, hs.get(tile, i).wide()));
          m.q = mul2(s, g[i]);
          m.p = mul2(m.p, s);
        }
      } else {
        const V2 first = t0 == 0 ? cols.state(a.state, e, a.E) : 0;
#pragma unroll
        for (int i = C - 1; i >= 0; --i) {
          p[i] = m.p;
          g[i] = m.q;
          na[i] = w[i] = 0;
          if (i < real) {
            V2 s;
            gs.get(tile, i).sigma(&s, &na[i]);
            const bool here = (cut >> i) & 1;
            const V2 before = here ? 0 : t0 + i == 0 ? first : hs.get(tile, i).wide();
            g[i] = add2(ds.get(tile, i).wide(), m.q);
            w[i] = mul2(mul2(s, na[i]), fma2(xs.get(tile, i).wide(), minus, before));
            if (here) m = {kSevered, 0};
            else m = {severed(m) ? m.p : mul2(m.p, s), mul2(s, g[i])};
          }
        }
      }
    }
    sh.warp_map[(rounds - 1 - k) & 1][warp][lane] = lasting(m);
    const bool any_cut = __syncthreads_or(cut != 0);
    const V2 u = cols.there(meet<W, STAGES, kShared, false>(sh, rounds - 1 - k, rank, share, any_cut, &met, &carry));
    to_x.start(), to_gate.start();
    if (k < mine && real == C && cut == 0 && finite(u)) {
#pragma unroll
      for (int i = 0; i < C; ++i) {
        const V2 G = fma2(p[i], u, g[i]);
        to_x.put(mul2(na[i], G));
        to_gate.put(mul2(w[i], G));
      }
    } else {
      if (!finite(u)) {
#pragma unroll
        for (int i = 0; i < C; ++i) p[i] = meeting(p[i], u);
      }
#pragma unroll
      for (int i = 0; i < C; ++i) {
        if (t0 + i >= stop) continue;
        const bool on = k < mine && i < real;
        const V2 G = on ? pass({p[i], g[i]}, u) : 0;
        to_x.put(on ? mul2(na[i], G) : 0);
        to_gate.put(on ? mul2(w[i], G) : 0);
      }
    }
    to_x.move(-share * L), to_gate.move(-share * L);
  }
  if (warp == 0 && part == 0 && a.d_state != nullptr) cols.store_state(a.d_state, e, a.E, carry);
  if (kBulk && !ring.ok && threadIdx.x == 0)
    for (int i = 0; i < STAGES; ++i) mbar_wait_bounded(&sh.full[i], ring.last_fill(i));
  if constexpr (!kBulk) asm volatile("cp.async.wait_all;" ::: "memory");
  if constexpr (kShared) cluster_meet();
}

template <class K>
cudaError_t launch_serial(K kernel, const GatedArgs& a, int sm, cudaStream_t s) {
  const int64_t grid = std::min<int64_t>(div_up(a.E * a.D, kSerialThreads), (int64_t)sm * 16);
  return launch_pdl(kernel, grid, kSerialThreads, 0, s, a);
}

// a tile kernel's launch: clusters of `share` CTAs
cudaError_t launch_tiles(void (*kernel)(GatedArgs, GatedMaps, int), int64_t grid, int threads, size_t smem, int share,
                         cudaStream_t s, const GatedArgs& a, const GatedMaps& maps) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)share;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = share > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, a, maps, share);
}

// The shape of a tile kernel: C steps a thread, W warps, STAGES tiles in the
// ring, RES CTAs an SM.  More CTAs cover a tile's chain of waits better than
// deeper rings: forward bfloat16 (256 x 512 x 1024 time-major) {16, 4, 2, 4} 141
// us, {16, 4, 3, 3} 155, {16, 8, 3, 2} 155, {8, 8, 3, 3} 164; the gradient, whose
// 16 steps keep 128 values a thread, {16, 4, 3, 2} (one row of 65536 x 2048) 268 us,
// {8, 8, 3, 2} 308, {8, 4, 2, 4} 485.  Unaligned rows have room for fewer tiles: the
// gradient, float32, {4, 8, 2, 2} / {8, 4, 2, 2}: 37 x 515 x 1001 time-major with
// lengths 73 / 76 us, without 80 / 81, 256 x 512 x 201 156 / 159, 64 x 256 x 333
// 41.7 / 42.3, 8 x 4000 x 2049 282 / 281; a few rows in clusters rather the other
// way, 1 x 20000 x 1001 144 / 139, 3 x 900 x 501 14.2 / 13.4.
template <int kChunk, int kWarps, int kStages, int kRes>
struct Shape {
  static constexpr int C = kChunk, W = kWarps, STAGES = kStages, RES = kRes;
};
template <class ST, bool kBack, bool kBulk>
struct TileShape;
template <bool kBulk>
struct TileShape<bf16, false, kBulk> : Shape<16, 4, 2, 4> {};
template <bool kBulk>
struct TileShape<float, false, kBulk> : Shape<8, 4, 2, 4> {};
template <>
struct TileShape<bf16, true, true> : Shape<16, 4, 3, 2> {};
template <>
struct TileShape<bf16, true, false> : Shape<8, 4, 2, 4> {};
template <>
struct TileShape<float, true, true> : Shape<8, 4, 3, 2> {};
template <>
struct TileShape<float, true, false> : Shape<4, 8, 2, 2> {};

// CTAs of a row: as many as fit the SMs beside each other in clusters of up to
// 8; where those would leave two thirds of them idle, segments of at least two
// tiles, which read the inputs twice.  The gradient, whose first launch needs two
// of its four inputs, is cut where half would idle if its rows are long, and
// then finely enough that its first launch fills the SMs too.  (bfloat16, one
// row of 65536 steps, us clusters / segments: 256 channels 182 / 41, 1024 246 /
// 125, 1536 234 / 191, 2048 277 / 251 -- on the wrong side of the rule --, 4096
// 299 / 527; the gradient of 64 205 / 37, of 256 206 / 69, of 1024 261 / 201.
// 4096 steps of 1024 channels 19.9 / 14.9, the gradient 20.4 / 24.9; 2048 steps of
// 256 channels 7.2 / 10.5.)  A segment's CTA walks the maps in front of it, eight
// loads in flight, all its warps the same ones: with hundreds of segments that
// takes longer than the rest (64 channels, 512 segments: 24 of 38 us; 256: 7 of
// 41; 1024: 1 of 125; the gradient of 256, 16 of 69).
//
// The CTAs an SM are those of the aligned shape for every alignment: the size of
// the workspace follows from this, and is asked for before there are addresses.
// (Two shapes of unaligned rows hold another number: the bfloat16 gradient's
// twice as many, the float32 one's as many of twice the warps.)
constexpr int kSegStep = 64;  // whole tiles of every shape
struct Split {
  int share = 1, nseg = 1, seg_len = 0;
};
Split split_rows(int64_t E, int64_t T, int64_t D, int64_t slots, bool back) {
  const int64_t units = E * div_up(D, kCols), tiles = div_up(T, kSegStep), most = units * kMaxShare;
  Split r;
  r.seg_len = (int)T;
  if ((3 * most <= slots && tiles > 4 * kMaxShare) || (back && 2 * most <= slots && tiles >= 16 * kMaxShare)) {
    int64_t segs = slots / units;
    if (back && tiles >= 8 * segs) segs *= 2;
    segs = std::min(segs, tiles / 2);
    r.seg_len = (int)(div_up(tiles, segs) * kSegStep);
    r.nseg = (int)div_up(T, r.seg_len);
    return r;
  }
  while (r.share < kMaxShare && 2 * r.share * units <= slots && 2 * r.share <= tiles) r.share *= 2;
  return r;
}
template <class ST, bool kBack>
Split split_rows(int64_t E, int64_t T, int64_t D, int sm) {
  return split_rows(E, T, D, (int64_t)TileShape<ST, kBack, true>::RES * sm, kBack);
}

template <class ST, bool kBack, bool kBulk, bool kShared, bool kMaps>
cudaError_t launch_shape(const GatedArgs& a, const GatedMaps& maps, int share, cudaStream_t s) {
  using H = TileShape<ST, kBack && !kMaps, kBulk>;
  static_assert(kSegStep % (H::C * H::W) == 0, "segments of whole tiles");
  constexpr int L = H::C * H::W;
  constexpr size_t smem = (size_t)H::STAGES * (kBack && !kMaps ? 4 : 2) * TileRows<ST, kBulk, L>::kTile;
  static_assert(H::RES * (smem + sizeof(GatedShared<H::W, H::STAGES, kShared>) + 1024) <= 228 * 1024, "RES CTAs fit an SM");
  void (*kernel)(GatedArgs, GatedMaps, int);
  if constexpr (kMaps) kernel = gated_map_kernel<ST, H::C, H::W, H::STAGES, kBulk, kBack, H::RES>;
  else if constexpr (kBack) kernel = gated_grad_tile_kernel<ST, H::C, H::W, H::STAGES, kBulk, kShared, H::RES>;
  else kernel = gated_tile_kernel<ST, H::C, H::W, H::STAGES, kBulk, kShared, H::RES>;
  static std::atomic<uint64_t> allowed;
  const cudaError_t e = allow_smem(kernel, smem, allowed);
  if (e != cudaSuccess) return e;
  return launch_tiles(kernel, a.E * div_up(a.D, kCols) * share * a.nseg, 32 * H::W, smem, share, s, a, maps);
}

template <class ST, bool kBack, bool kBulk>
cudaError_t run_tiles(GatedArgs a, const GatedMaps& maps, int sm, cudaStream_t s) {
  const Split r = split_rows<ST, kBack>(a.E, a.T, a.D, sm);
  a.nseg = r.nseg, a.seg_len = r.seg_len;
  if (r.share > 1) return launch_shape<ST, kBack, kBulk, true, false>(a, maps, r.share, s);
  if (r.nseg > 1) {
    const cudaError_t e = launch_shape<ST, kBack, kBulk, false, true>(a, maps, 1, s);
    if (e != cudaSuccess) return e;
  }
  return launch_shape<ST, kBack, kBulk, false, false>(a, maps, 1, s);
}

// Whether rows of T steps are walked by threads of their own, step by step,
// instead of by tiles: up to 8 steps, and up to 64 where the rows are many
// times what fits the SMs as tile CTAs, each of which takes some 3 us to begin.
// (us, steps / tiles, 2048 channels bfloat16: forward 16 rows of 8 steps 3.0 /
// 3.8, of 16 4.7 / 3.1; 256 rows of 16 15 / 40, of 64 53 / 43.  Gradient: 64
// rows of 16 19 / 31, of 32 36 / 33; 256 rows of 64 80 / 114.)
bool by_steps(int64_t E, int64_t T, int64_t D, int64_t slots) {
  const int64_t units = E * div_up(D, kCols);
  return T <= 8 || (T <= 64 && T * slots <= 4 * units) || units > INT32_MAX / kMaxShare;
}
template <class ST, bool kBack>
bool by_steps(int64_t E, int64_t T, int64_t D, int sm) {
  return by_steps(E, T, D, (int64_t)TileShape<ST, kBack, true>::RES * sm);
}
template <class ST, bool kBack>
size_t workspace_of(int64_t E, int64_t T, int64_t D, int sm) {
  if (by_steps<ST, kBack>(E, T, D, sm)) return 0;
  const Split r = split_rows<ST, kBack>(E, T, D, sm);
  return r.nseg > 1 ? (size_t)(E * div_up(D, kCols)) * segment_slots(r.nseg) * 32 * sizeof(Map2) : 0;
}

// In vectors where every row starts on a 16-byte boundary (`even`)
cudaError_t launch_steps(void (*vectors)(GatedArgs, int64_t), void (*single)(GatedArgs), bool even, int es, const GatedArgs& a,
                         int sm, cudaStream_t s) {
  const int64_t blocks = div_up(a.D, kStepThreads * 16 / es);
  if (even && a.E * blocks <= INT32_MAX) return launch_pdl(vectors, a.E * blocks, kStepThreads, 0, s, a, blocks);
  return launch_serial(single, a, sm, s);
}

template <class ST>
cudaError_t scan_typed(const GatedArgs& a, int sm, cudaStream_t s) {
  constexpr int es = Stor<ST>::kBytes, L = TileShape<ST, false, true>::C * TileShape<ST, false, true>::W;
  if (by_steps<ST, false>(a.E, a.T, a.D, sm))
    return launch_steps(gated_step_kernel<ST>, gated_serial_kernel<ST>,
                        rows_aligned({a.x, a.gate, a.h}, {a.D, a.x_stride, a.gate_stride}, es, 16) &&
                            rows_aligned({a.state, a.last}, {}, 4, 16),
                        es, a, sm, s);
  GatedMaps maps = {};
  const float* in[2] = {a.x, a.gate};
  const int64_t stride[2] = {a.x_stride, a.gate_stride};
  bool bulk = rows_aligned({a.x, a.gate}, {a.x_stride, a.gate_stride}, es, 16) && rows_aligned({a.h}, {a.D}, es, 2 * es);
  for (int i = 0; bulk && i < 2; ++i)
    bulk = encode_steps_map(&maps.in[i], in[i], es, a.D, a.T, a.E, stride[i] * a.step_t, stride[i] * a.step_e, kCols, L);
  return bulk ? run_tiles<ST, false, true>(a, maps, sm, s) : run_tiles<ST, false, false>(a, maps, sm, s);
}

template <class ST>
cudaError_t grad_typed(const GatedArgs& a, int sm, cudaStream_t s) {
  using H = TileShape<ST, true, true>;
  constexpr int es = Stor<ST>::kBytes, L = H::C * H::W;
  static_assert(L == TileShape<ST, false, true>::C * TileShape<ST, false, true>::W, "one box of steps for both launches");
  if (by_steps<ST, true>(a.E, a.T, a.D, sm))
    return launch_steps(gated_grad_step_kernel<ST>, gated_grad_serial_kernel<ST>,
                        rows_aligned({a.x, a.gate, a.dh, a.in_h, a.dx, a.dgate},
                                     {a.D, a.x_stride, a.gate_stride, a.dh_stride, a.h_stride, a.dx_stride, a.dgate_stride}, es, 16) &&
                            rows_aligned({a.state, a.d_last, a.d_state}, {}, 4, 16),
                        es, a, sm, s);
  GatedMaps maps = {};
  const float* in[4] = {a.x, a.gate, a.dh, a.in_h};
  const int64_t stride[4] = {a.x_stride, a.gate_stride, a.dh_stride, a.h_stride};
  bool bulk = rows_aligned({a.x, a.gate, a.dh, a.in_h}, {a.x_stride, a.gate_stride, a.dh_stride, a.h_stride}, es, 16) &&
              rows_aligned({a.dx, a.dgate}, {a.D, a.dx_stride, a.dgate_stride}, es, 2 * es);
  for (int i = 0; bulk && i < 4; ++i)
    bulk = encode_steps_map(&maps.in[i], in[i], es, a.D, a.T, a.E, stride[i] * a.step_t, stride[i] * a.step_e, kCols, L);
  return bulk ? run_tiles<ST, true, true>(a, maps, sm, s) : run_tiles<ST, true, false>(a, maps, sm, s);
}

}  // namespace

cudaError_t run_gated_scan(const GatedArgs& a, int sm, cudaStream_t s) {
  return a.bf16_io ? scan_typed<bf16>(a, sm, s) : scan_typed<float>(a, sm, s);
}

cudaError_t run_gated_scan_backward(const GatedArgs& a, int sm, cudaStream_t s) {
  return a.bf16_io ? grad_typed<bf16>(a, sm, s) : grad_typed<float>(a, sm, s);
}

size_t gated_scan_workspace(int64_t E, int64_t T, int64_t D, bool bf16_io, bool backward, int sm) {
  if (E == 0 || T == 0 || D == 0) return 0;
  if (backward) return bf16_io ? workspace_of<bf16, true>(E, T, D, sm) : workspace_of<float, true>(E, T, D, sm);
  return bf16_io ? workspace_of<bf16, false>(E, T, D, sm) : workspace_of<float, false>(E, T, D, sm);
}

cudaError_t status_gated(unsigned int* word, bool clear) { return unit_status(word, clear); }

}  // namespace rlca
