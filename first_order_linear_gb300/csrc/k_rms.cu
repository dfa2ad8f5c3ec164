// Root-mean-square norm with the residual's addition, its result and its
// input in 8 bits, and its gradient.
//
//   total = x + residual,  y = total rstd w,  rstd = 1 / sqrt(mean(total^2) + eps)
//   dx = d_total + rstd (g - s mean(g s)),  g = dy w,  s = total rstd
//   dw = sum over rows of dy s
//
// Both directions are bound by HBM: every input is read once and every output
// written once.  65536 x 4096 bfloat16 with a residual, y and total in 8 bits:
// 320 us, 6.7 TB/s, as fast as the measured copy; without total's 8 bits 0.99,
// without either 0.96 of it.  The gradient from total in 8 bits, 32768 x 4096
// bfloat16: 148 us, 6.3 TB/s, 0.94, of which joining dw takes about 5 us.
// total is rounded before it is normalised: the gradient reads what was stored.
// y's 8 bits come from its float32 values, one rounding.
#include <algorithm>
#include <atomic>
#include <initializer_list>
#include <type_traits>

#include "eight.cuh"
#include "policy.h"
#include "reduce.cuh"
#include "tma.cuh"
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
// Rows in registers.  A thread holds VPT parts of a row, VE elements of one
// group of columns each:
//   aligned rows    part j is the 16-byte vector lane + j TPR; the 16 (float32:
//                   32) lanes of a group are next to each other
//   other rows      a warp takes a group, a lane four of its elements, 32 apart
// so a group's maximum is a reduction over lanes of one warp in both.  CTAs
// are persistent: a thread keeps its columns' weight over all its rows and
// loads the next row before it works on the current one.
//
// Aligned rows are bound by HBM.  Other rows are bound by their instructions:
// single elements (20000 x 2001 bfloat16 with both 8-bit outputs: 93 us, 0.51 of
// the copy rate, 71% of the issue slots; 5001 x 1001 float32 12.3 us, 1.0).
// ---------------------------------------------------------------------------
template <class ST, bool kAligned>
struct Part {
  static constexpr int VE = kAligned ? 16 / Stor<ST>::kBytes : 4;
  static constexpr int kLanes = kGroup / VE;  // of a group
  using E = std::conditional_t<Stor<ST>::kBytes == 4, float, uint16_t>;
  // as they lie in memory, taken apart when used: at the load that would wait for it
  struct Apart {
    E e[VE];
  };
  struct Apart8 {
    uint8_t e[VE];
  };
  using Raw = std::conditional_t<kAligned, uint4, Apart>;
  using Raw8 = std::conditional_t<kAligned, std::conditional_t<VE == 8, uint2, uint32_t>, Apart8>;
  int lane;  // of the row
  int D;     // (rows that fit registers)

  // column of element k of part j, of a row shared by TPR threads
  template <int TPR>
  __device__ int col(int j, int k) const {
    if constexpr (kAligned) return lane * VE + j * TPR * VE + k;
    return (lane >> 5) * kGroup + (lane & 31) + j * (TPR / 32) * kGroup + 32 * k;
  }
  template <int TPR>
  __device__ bool on(int j, int k) const {
    return col<TPR>(j, kAligned ? 0 : k) < D;
  }
  template <int TPR>
  __device__ Raw load(const float* p, int64_t row, int64_t n, int j) const {
    Raw r;
    const E* base = reinterpret_cast<const E*>(p) + row;
    if constexpr (kAligned) {
      r = make_uint4(0u, 0u, 0u, 0u);
      if (on<TPR>(j, 0) && span_in_range(row + col<TPR>(j, 0), VE, n)) r = *reinterpret_cast<const uint4*>(base + col<TPR>(j, 0));
    } else {
#pragma unroll
      for (int k = 0; k < VE; ++k) r.e[k] = on<TPR>(j, k) && in_range(row + col<TPR>(j, k), n) ? base[col<TPR>(j, k)] : E(0);
    }
    return r;
  }
  __device__ static void open(const Raw& r, float* v) {
    if constexpr (kAligned) {
      const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if constexpr (VE == 4) v[k] = __uint_as_float(w[k]);
        else v[2 * k] = __uint_as_float(w[k] << 16), v[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
      }
    } else {
#pragma unroll
      for (int k = 0; k < VE; ++k) {
        if constexpr (Stor<ST>::kBytes == 4) v[k] = r.e[k];
        else v[k] = Stor<ST>::from_bits(r.e[k]);
      }
    }
  }
  template <int TPR>
  __device__ void store(float* p, int64_t row, int64_t n, int j, const float* v) const {
    if constexpr (kAligned) {
      if (!on<TPR>(j, 0) || !span_in_range(row + col<TPR>(j, 0), VE, n)) return;
      if constexpr (VE == 8) Stor<ST>::st8(p, row + col<TPR>(j, 0), v);
      else Stor<ST>::st4(p, row + col<TPR>(j, 0), v);
    } else {
#pragma unroll
      for (int k = 0; k < VE; ++k)
        if (on<TPR>(j, k)) store1<ST>(p, row + col<TPR>(j, k), n, v[k]);
    }
  }

  // ---- in 8 bits
  template <int TPR>
  __device__ Raw8 load8(const uint8_t* q, int64_t row, int64_t N, int j) const {
    Raw8 r{};
    if constexpr (kAligned) {
      const int64_t i = row * D + col<TPR>(j, 0);
      if (on<TPR>(j, 0) && span_in_range(i, VE, N * D)) r = *reinterpret_cast<const Raw8*>(q + i);
    } else {
#pragma unroll
      for (int k = 0; k < VE; ++k) {
        const int64_t i = row * D + col<TPR>(j, k);
        r.e[k] = on<TPR>(j, k) && in_range(i, N * D) ? q[i] : (uint8_t)0;
      }
    }
    return r;
  }
  // the scale of part j's group
  template <int TPR>
  __device__ float scale8(const float* scale, int64_t row, int64_t N, int j) const {
    const int c = col<TPR>(j, 0);
    const int64_t i = row * groups_of(D) + c / kGroup;
    return c / kGroup * kGroup < D && in_range(i, N * groups_of(D)) ? scale[i] : 0.f;
  }
  __device__ static void open8(const Raw8& r, float scale, float* v) {
#pragma unroll
    for (int k = 0; k < VE; k += 2) {
      uint32_t two;
      if constexpr (!kAligned) two = (uint32_t)r.e[k] | (uint32_t)r.e[k + 1] << 8;
      else if constexpr (VE == 8) two = (k < 4 ? r.x : r.y) >> 8 * (k % 4);
      else two = r >> 8 * k;
      const float2 f = from_e4m3x2(two);
      v[k] = f.x * scale, v[k + 1] = f.y * scale;
    }
  }
  // part j of the row in 8 bits, and its group's scale
  template <int TPR>
  __device__ void store8(uint8_t* q, float* scale, int64_t row, int64_t N, int j, const float* v) const {
    float m = 0.f;
#pragma unroll
    for (int k = 0; k < VE; ++k) m = fmaxf(m, fabsf(v[k]));
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFullMask, m, o));
    const float sc = group_scale(m), inv = __frcp_rn(sc);
    const int c = col<TPR>(j, 0);
    const int64_t groups = groups_of(D), n = N * D;
    if (c % kGroup == 0 && c < D && in_range(row * groups + c / kGroup, N * groups)) scale[row * groups + c / kGroup] = sc;
    uint32_t w[VE / 2];
#pragma unroll
    for (int k = 0; k < VE / 2; ++k) w[k] = to_e4m3x2(v[2 * k] * inv, v[2 * k + 1] * inv);
    if constexpr (kAligned) {
      if (!on<TPR>(j, 0) || !span_in_range(row * D + c, VE, n)) return;
      if constexpr (VE == 8) *reinterpret_cast<uint2*>(q + row * D + c) = make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
      else *reinterpret_cast<uint32_t*>(q + row * D + c) = w[0] | w[1] << 16;
    } else {
#pragma unroll
      for (int k = 0; k < VE; ++k)
        if (on<TPR>(j, k) && in_range(row * D + col<TPR>(j, k), n)) q[row * D + col<TPR>(j, k)] = (uint8_t)(w[k / 2] >> 8 * (k % 2));
    }
  }
};

// Threads of a CTA: whole warps of rows, or one row over the CTA.
__host__ __device__ constexpr int cta_threads(int tpr) { return tpr < 128 ? 128 : tpr; }
// CTAs of `threads` threads an SM is to hold, by the values a thread has in
// registers (32768 x 4096 bfloat16, 16 values: 768 threads 162 us, 512 179 us)
__host__ __device__ constexpr int rms_resident(int threads, int values) {
    const int n = (values >= 32 ? 512 : values >= 16 ? 768 : 1024) / threads;
  return n > 0 ? n : 1;
}

// Sum of a row's values over its TPR threads; `slot` as in a ring of two: one
// is written again only after a barrier that follows its last read.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float (*scratch)[32], int slot) {
  v = warp_sum(v);
  if constexpr (TPR > 32) {
    constexpr int W = TPR / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) scratch[slot][warp] = v;
    __syncthreads();
    v = warp_sum(lane < W ? scratch[slot][warp / W * W + lane] : 0.f);
  }
  return v;
}

template <class ST, bool kAligned, int VPT, int TPR>
__global__ void __launch_bounds__(cta_threads(TPR), rms_resident(cta_threads(TPR), VPT * Part<ST, kAligned>::VE))
    rms_kernel(RmsArgs a) {
  using P = Part<ST, kAligned>;
  constexpr int ROWS = cta_threads(TPR) / TPR, VE = P::VE;
  __shared__ float scratch[2][32];
  const P part{(int)(threadIdx.x % TPR), (int)a.D};
  const float inv_d = 1.f / (float)a.D;
  const int64_t step = (int64_t)gridDim.x * ROWS, nd = a.N * a.D;
  const int64_t x_size = extent(a.N, a.D, a.x_stride), r_size = extent(a.N, a.D, a.residual_stride);
  int64_t row = (int64_t)blockIdx.x * ROWS + threadIdx.x / TPR;
  pdl_trigger();
  pdl_wait();
  typename P::Raw w[VPT], x[VPT], r[VPT];
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    w[j] = part.template load<TPR>(a.weight, 0, a.D, j);
    if (row < a.N) {
      x[j] = part.template load<TPR>(a.x, row * a.x_stride, x_size, j);
      if (a.residual != nullptr) r[j] = part.template load<TPR>(a.residual, row * a.residual_stride, r_size, j);
    }
  }
  int slot = 0;
  // (the rows of a warp, and of a CTA where a row takes all of it, end together)
  for (int64_t first = row - threadIdx.x / TPR; first < a.N; first += step, row += step) {
    const bool here = row < a.N;
    float v[VPT][VE];
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      P::open(x[j], v[j]);
      if (a.residual != nullptr) {
        float f[VE];
        P::open(r[j], f);
#pragma unroll
        for (int k = 0; k < VE; ++k) v[j][k] = stored<ST>(v[j][k] + f[k]);
        if (here) part.template store<TPR>(a.total, row * a.D, nd, j, v[j]);
      }
#pragma unroll
      for (int k = 0; k < VE; ++k) ss = fmaf(v[j][k], v[j][k], ss);
    }
    const int64_t next = row + step;
    if (next < a.N) {
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        x[j] = part.template load<TPR>(a.x, next * a.x_stride, x_size, j);
        if (a.residual != nullptr) r[j] = part.template load<TPR>(a.residual, next * a.residual_stride, r_size, j);
      }
    }
    const float rstd = rsqrtf(row_sum<TPR>(ss, scratch, slot) * inv_d + a.eps);
    slot ^= 1;
    if (!here) continue;
    if (a.rstd != nullptr && part.lane == 0 && in_range(row, a.N)) a.rstd[row] = rstd;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      if (a.total8 != nullptr) part.template store8<TPR>(a.total8, a.total8_scale, row, a.N, j, v[j]);
      float f[VE];
      P::open(w[j], f);
#pragma unroll
      for (int k = 0; k < VE; ++k) f[k] = v[j][k] * rstd * f[k];
      if (a.y != nullptr) part.template store<TPR>(a.y, row * a.D, nd, j, f);
      if (a.y8 != nullptr) part.template store8<TPR>(a.y8, a.y8_scale, row, a.N, j, f);
    }
  }
}

// ---------------------------------------------------------------------------
// A CTA a row, two passes over it: a warp takes a group of columns at a time,
// a lane four of them, 32 apart.  Rows wider than registers hold, bound by their
// single elements: 5000 x 12288 float32 with a residual 262 us, 0.55 of the copy
// rate; 10000 x 20000 bfloat16 836 us, 0.28.  The gradients further down, three passes with
// dw's: 10000 x 12288 bfloat16 463 us, 0.31; 5000 x 20000 from 8 bits 467 us, 0.22.
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

// ---------------------------------------------------------------------------
// Gradient: rows in registers as above, the next one loaded ahead; each CTA
// leaves the sums of dw over its rows in ws[CTA][D], which a second kernel
// joins in order.  (131072 x 512 bfloat16: 87 us, 0.91 of the copy rate;
// unaligned rows, 20000 x 2001 bfloat16: 73 us, 0.57, bound by instructions; rows
// of 4097 to 8192 unaligned columns, whose 16 values, their products and sums a
// thread do not fit 128 registers (56 to 84 bytes spilled), 10000 x 7001 bfloat16
// 202 us, 0.36, 5000 x 7001 float32 95 us, 0.71.)
// ---------------------------------------------------------------------------
// CTAs an SM is to hold: 512 threads with up to 16 values (5001 x 1001 float32: 768
// threads 22.3 us, 512 15.9 us)
__host__ __device__ constexpr int rms_grad_resident(int threads) { return threads < 512 ? 512 / threads : 1; }
// (rows of a CTA beside each other leave one set of sums: 5001 x 1001 float32
// with 128 threads 19.4 us, 256 15.9 us, 512 15.1 us, but 20000 x 2001 bfloat16
// 73, 73 and 78 us)
__host__ __device__ constexpr int grad_threads(int tpr) { return tpr < 256 ? 256 : tpr; }

template <class ST, bool kAligned, bool k8, int VPT, int TPR>
__global__ void __launch_bounds__(grad_threads(TPR), rms_grad_resident(grad_threads(TPR)))
    rms_grad_kernel(RmsGradArgs a) {
  using P = Part<ST, kAligned>;
  constexpr int T = grad_threads(TPR), ROWS = T / TPR, VE = P::VE;
  __shared__ float scratch[2][32];
  const P part{(int)(threadIdx.x % TPR), (int)a.D};
  const float inv_d = 1.f / (float)a.D;
  const int64_t step = (int64_t)gridDim.x * ROWS, nd = a.N * a.D;
  const int64_t dy_size = extent(a.N, a.D, a.dy_stride), dt_size = extent(a.N, a.D, a.d_total_stride),
                t_size = extent(a.N, a.D, a.total_stride);
  int64_t row = (int64_t)blockIdx.x * ROWS + threadIdx.x / TPR;
  pdl_trigger();
  pdl_wait();
  typename P::Raw w[VPT], dy[VPT], dt[VPT], t[k8 ? 1 : VPT];
  typename P::Raw8 t8[k8 ? VPT : 1];
  float scale[k8 ? VPT : 1], dw[VPT][VE];
  float rstd = 0.f;
  const auto load = [&](int64_t at) {
    rstd = a.rstd[at];
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      dy[j] = part.template load<TPR>(a.dy, at * a.dy_stride, dy_size, j);
      if (a.d_total != nullptr && a.dx != nullptr) dt[j] = part.template load<TPR>(a.d_total, at * a.d_total_stride, dt_size, j);
      if constexpr (k8) {
        t8[j] = part.template load8<TPR>(a.total8, at, a.N, j);
        scale[j] = part.template scale8<TPR>(a.total8_scale, at, a.N, j);
      } else {
        t[j] = part.template load<TPR>(a.total, at * a.total_stride, t_size, j);
      }
    }
  };
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    w[j] = part.template load<TPR>(a.weight, 0, a.D, j);
#pragma unroll
    for (int k = 0; k < VE; ++k) dw[j][k] = 0.f;
  }
  if (row < a.N) load(row);
  int slot = 0;
  for (int64_t first = row - threadIdx.x / TPR; first < a.N; first += step, row += step) {
    const bool here = row < a.N;
    float g[VPT][VE], s[VPT][VE], d[VPT][VE];
    float along = 0.f;
    const float r = rstd;
    if (here) {
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        float fw[VE];
        P::open(dy[j], g[j]);
        P::open(w[j], fw);
        if constexpr (k8) P::open8(t8[j], scale[j] * r, s[j]);
        else P::open(t[j], s[j]);
        if (a.d_total != nullptr) P::open(dt[j], d[j]);
#pragma unroll
        for (int k = 0; k < VE; ++k) {
          if constexpr (!k8) s[j][k] *= r;
          dw[j][k] = fmaf(g[j][k], s[j][k], dw[j][k]);
          g[j][k] *= fw[k];
          along = fmaf(g[j][k], s[j][k], along);
        }
      }
    }
    const int64_t next = row + step;
    if (next < a.N) load(next);
    if (a.dx == nullptr) continue;
    along = row_sum<TPR>(along, scratch, slot) * inv_d;
    slot ^= 1;
    if (!here) continue;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
#pragma unroll
      for (int k = 0; k < VE; ++k) {
        g[j][k] = r * fmaf(-s[j][k], along, g[j][k]);
        if (a.d_total != nullptr) g[j][k] += d[j][k];
      }
      part.template store<TPR>(a.dx, row * a.D, nd, j, g[j]);
    }
  }
  if (a.dweight == nullptr) return;
  const int64_t at = (int64_t)blockIdx.x * a.D, ws_size = a.D * (int64_t)gridDim.x;
  if constexpr (ROWS == 1) {
#pragma unroll
    for (int j = 0; j < VPT; ++j)
#pragma unroll
      for (int k = 0; k < VE; ++k)
        if (part.template on<TPR>(j, k)) store1<float>(a.ws, at + part.template col<TPR>(j, k), ws_size, dw[j][k]);
  } else {
    // the CTA's rows side by side, added in order
    __shared__ float acc[VPT * TPR * VE];
    for (int q = 0; q < ROWS; ++q) {
      if (threadIdx.x / TPR == q) {
#pragma unroll
        for (int j = 0; j < VPT; ++j)
#pragma unroll
          for (int k = 0; k < VE; ++k) {
            const int c = part.template col<TPR>(j, k);
            if (in_range(c, VPT * TPR * VE)) acc[c] = dw[j][k] + (q > 0 ? acc[c] : 0.f);
          }
      }
      __syncthreads();
    }
    for (int c = threadIdx.x; c < a.D; c += T) store1<float>(a.ws, at + c, ws_size, acc[c]);
  }
}

// The same for aligned rows of a CTA of their own (32768 x 4096 bfloat16 from 8
// bits: 148 us), fed by bulk copies: thread 0 keeps kRows - 1 rows of dy, d_total and total on their way into shared
// memory, so what is in flight does not depend on the registers that the
// columns' sums leave.  A stage is filled again after the barrier that follows
// its reads (the one the row's sum needs anyway).  A wait that gives up is
// recorded in the status word; the rows are then walked without further
// copies or waits.
template <class ST, bool k8, int VPT, int TPR, int kRows>
__global__ void __launch_bounds__(TPR, rms_grad_resident(TPR)) rms_grad_ring_kernel(RmsGradArgs a) {
  using P = Part<ST, true>;
  constexpr int VE = P::VE;
  extern __shared__ __align__(128) unsigned char ring_rows[];  // [kRows][dy, total, d_total]
  __shared__ __align__(8) uint64_t full[kRows];
  __shared__ float scratch[2][32];
  const P part{(int)threadIdx.x, (int)a.D};
  const uint32_t row_bytes = (uint32_t)(a.D * Stor<ST>::kBytes), t_bytes = k8 ? (uint32_t)a.D : row_bytes;
  const bool has_dt = a.d_total != nullptr && a.dx != nullptr;
  const uint32_t stage_bytes = row_bytes + t_bytes + (has_dt ? row_bytes : 0);
  const float inv_d = 1.f / (float)a.D;
  const int64_t step = gridDim.x, nd = a.N * a.D;
  pdl_trigger();
  if (threadIdx.x == 0) {
    for (int i = 0; i < kRows; ++i) mbar_init(&full[i], 1);
    mbar_fence_init();
  }
  __syncthreads();
  pdl_wait();
  const auto fill = [&](int stage, int64_t row) {
    if (!in_range(stage, kRows) || !in_range(row, a.N)) return;
    unsigned char* to = ring_rows + (size_t)stage * stage_bytes;
    const auto at = [&](const float* p, int64_t stride) {
      return reinterpret_cast<const unsigned char*>(p) + row * stride * Stor<ST>::kBytes;
    };
    mbar_arrive_expect_tx(&full[stage], stage_bytes);
    bulk_load(to, at(a.dy, a.dy_stride), row_bytes, &full[stage]);
    bulk_load(to + row_bytes, k8 ? a.total8 + row * a.D : at(a.total, a.total_stride), t_bytes, &full[stage]);
    if (has_dt) bulk_load(to + row_bytes + t_bytes, at(a.d_total, a.d_total_stride), row_bytes, &full[stage]);
  };
  int64_t row = blockIdx.x;
  if (threadIdx.x == 0)
    for (int i = 0; i < kRows - 1; ++i)
      if (row + i * step < a.N) fill(i, row + i * step);
  typename P::Raw w[VPT];
  float dw[VPT][VE], scale[k8 ? VPT : 1];
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    w[j] = part.template load<TPR>(a.weight, 0, a.D, j);
#pragma unroll
    for (int k = 0; k < VE; ++k) dw[j][k] = 0.f;
  }
  float rstd = 0.f;
  const auto load = [&](int64_t at) {
    rstd = a.rstd[at];
    if constexpr (k8) {
#pragma unroll
      for (int j = 0; j < VPT; ++j) scale[j] = part.template scale8<TPR>(a.total8_scale, at, a.N, j);
    }
  };
  if (row < a.N) load(row);
  int slot = 0;
  FillRing<kRows> ring;
  for (; row < a.N; row += step) {
    // the stage before this one was read in the last round
    if (threadIdx.x == 0 && ring.ok && row + (kRows - 1) * step < a.N) fill(ring.fill_stage(), row + (kRows - 1) * step);
    if (ring.ok) ring.ok = mbar_wait_bounded(&full[ring.stage], ring.phase);
    const unsigned char* at = ring_rows + (size_t)ring.stage * stage_bytes;
    float g[VPT][VE], s[VPT][VE];
    typename P::Raw dt[VPT];
    float along = 0.f;
    const float r = rstd;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int v = threadIdx.x + j * TPR;
      uint4 raw = make_uint4(0u, 0u, 0u, 0u), traw = raw;
      typename P::Raw8 q{};
      dt[j] = raw;
      if (part.template on<TPR>(j, 0) &&
          span_in_range((int64_t)ring.stage * stage_bytes + v * 16, (int64_t)stage_bytes - row_bytes + 16, (int64_t)kRows * stage_bytes)) {
        raw = *reinterpret_cast<const uint4*>(at + v * 16);
        if constexpr (k8) q = *reinterpret_cast<const typename P::Raw8*>(at + row_bytes + v * VE);
        else traw = *reinterpret_cast<const uint4*>(at + row_bytes + v * 16);
        if (has_dt) dt[j] = *reinterpret_cast<const uint4*>(at + row_bytes + t_bytes + v * 16);
      }
      float fw[VE];
      P::open(raw, g[j]);
      P::open(w[j], fw);
      if constexpr (k8) P::open8(q, scale[j] * r, s[j]);
      else P::open(traw, s[j]);
#pragma unroll
      for (int k = 0; k < VE; ++k) {
        if constexpr (!k8) s[j][k] *= r;
        dw[j][k] = fmaf(g[j][k], s[j][k], dw[j][k]);
        g[j][k] *= fw[k];
        along = fmaf(g[j][k], s[j][k], along);
      }
    }
    if (row + step < a.N) load(row + step);
    along = row_sum<TPR>(along, scratch, slot) * inv_d;
    slot ^= 1;
    ring.next();
    if (a.dx == nullptr) continue;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      float d[VE];
      P::open(dt[j], d);  // (zeros without d_total)
#pragma unroll
      for (int k = 0; k < VE; ++k) g[j][k] = fmaf(r, fmaf(-s[j][k], along, g[j][k]), d[k]);
      part.template store<TPR>(a.dx, row * a.D, nd, j, g[j]);
    }
  }
  // (copies still on their way after a wait gave up land before the CTA ends)
  if (!ring.ok && threadIdx.x == 0)
    for (int i = 0; i < kRows; ++i) mbar_wait_bounded(&full[i], ring.last_fill(i));
  if (a.dweight == nullptr) return;
  const int64_t to = (int64_t)blockIdx.x * a.D, ws_size = a.D * (int64_t)gridDim.x;
#pragma unroll
  for (int j = 0; j < VPT; ++j)
#pragma unroll
    for (int k = 0; k < VE; ++k)
      if (part.template on<TPR>(j, 0)) store1<float>(a.ws, to + part.template col<TPR>(j, k), ws_size, dw[j][k]);
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

bool aligned_to(const void* p, int to) { return ((uintptr_t)p % to) == 0; }

template <class ST, bool kAligned, int VPT, int TPR>
cudaError_t launch_rms(const RmsArgs& a, int sm, cudaStream_t s) {
  constexpr int T = cta_threads(TPR), R = rms_resident(T, VPT * Part<ST, kAligned>::VE);
  return launch_pdl(rms_kernel<ST, kAligned, VPT, TPR>, std::min<int64_t>(div_up(a.N, T / TPR), (int64_t)R * sm), T, 0, s, a);
}

// Threads a row, and parts of one a thread (bfloat16 with both 8-bit outputs:
// 32768 x 4096 with 256 threads x 2 parts 162 us, 128 x 4 175 us, 512 x 1 174 us;
// 60000 x 1000 with 128 x 1 79 us, 32 x 4 89 us; 131072 x 512 with 64 x 1 84 us,
// 32 x 2 89 us; unaligned 300000 x 201 with 64 x 1 171 us, 32 x 2 164 us);
// `parts`: of a row
template <class ST, bool kAligned>
cudaError_t rms_width(const RmsArgs& a, int64_t parts, int sm, cudaStream_t s) {
  if (parts <= 32) return launch_rms<ST, kAligned, 1, 32>(a, sm, s);
  if (parts <= 64) {
    if constexpr (kAligned) return launch_rms<ST, kAligned, 1, 64>(a, sm, s);
    else return launch_rms<ST, kAligned, 2, 32>(a, sm, s);
  }
  if (parts <= 128) return launch_rms<ST, kAligned, 1, 128>(a, sm, s);
  if (parts <= 256) return launch_rms<ST, kAligned, 2, 128>(a, sm, s);
  if (parts <= 512) return launch_rms<ST, kAligned, 2, 256>(a, sm, s);
  if (parts <= 1024) return launch_rms<ST, kAligned, 2, 512>(a, sm, s);
  return launch_rms<ST, kAligned, 4, 512>(a, sm, s);
}

template <class ST>
cudaError_t norm_typed(const RmsArgs& a, int sm, cudaStream_t s) {
  constexpr int es = Stor<ST>::kBytes, VE = 16 / es;
  const bool even = rows_aligned({a.x, a.residual, a.weight, a.total, a.y}, {a.D, a.x_stride, a.residual_stride}, es) &&
                    aligned_to(a.y8, VE) && aligned_to(a.total8, VE);
  const int64_t parts = even ? a.D / VE : groups_of(a.D) * 32;
  if (parts <= 2048) return even ? rms_width<ST, true>(a, parts, sm, s) : rms_width<ST, false>(a, parts, sm, s);
  return launch_pdl(rms_long_kernel<ST>, std::min<int64_t>(a.N, 4 * (int64_t)sm), kLongThreads, 0, s, a);
}

// CTAs of a backward launch of T threads, R rows at a time: those that fit
// the SMs, but four rounds of rows each where that still gives every SM one
// (each CTA leaves D partial sums to be joined)
int64_t grad_grid(int64_t N, int T, int R, int sm) {
  const int64_t rounds = div_up(N, R);
  return std::min({rounds, (int64_t)rms_grad_resident(T) * sm, std::max<int64_t>(sm, div_up(rounds, 4))});
}

template <class ST, bool kAligned, bool k8, int VPT, int TPR>
cudaError_t launch_grad(const RmsGradArgs& a, int sm, cudaStream_t s) {
  constexpr int T = grad_threads(TPR);
  const int64_t grid = grad_grid(a.N, T, T / TPR, sm);
  const cudaError_t e = launch_pdl(rms_grad_kernel<ST, kAligned, k8, VPT, TPR>, grid, T, 0, s, a);
  return e == cudaSuccess ? join(a, grid, s) : e;
}

template <class ST, bool k8, int VPT, int TPR, int kRows>
cudaError_t launch_grad_ring(const RmsGradArgs& a, int sm, cudaStream_t s) {
  const auto kernel = rms_grad_ring_kernel<ST, k8, VPT, TPR, kRows>;
  constexpr int es = Stor<ST>::kBytes;
  static std::atomic<uint64_t> allowed;
  cudaError_t e = allow_smem(kernel, (size_t)kRows * TPR * VPT * (32 + (k8 ? 16 / es : 16)), allowed);
  if (e != cudaSuccess) return e;
  const size_t row = (size_t)a.D * es;
  const size_t smem = kRows * (row + (k8 ? (size_t)a.D : row) + (a.d_total != nullptr && a.dx != nullptr ? row : 0));
  const int64_t grid = grad_grid(a.N, TPR, 1, sm);
  e = launch_pdl(kernel, grid, TPR, smem, s, a);
  return e == cudaSuccess ? join(a, grid, s) : e;
}

// Rows that start on 16-byte boundaries (`parts` vectors each) or not (32
// parts a group); from 65 vectors on the former take the ring, if rows in 8 bits
// are whole multiples of 16 bytes too (20000 x 4088 bfloat16 without: 104 us; as
// unaligned rows 150 us).
template <class ST, bool k8>
cudaError_t grad_width(const RmsGradArgs& a, bool even, bool ring, int64_t parts, int sm, cudaStream_t s, bool* taken) {
  *taken = true;
  if (even) {
    if (parts <= 32) return launch_grad<ST, true, k8, 1, 32>(a, sm, s);
    if (parts <= 64) return launch_grad<ST, true, k8, 2, 32>(a, sm, s);
    if (ring && parts <= 128) return launch_grad_ring<ST, k8, 1, 128, 4>(a, sm, s);
    if (ring && parts <= 256) return launch_grad_ring<ST, k8, 2, 128, 4>(a, sm, s);
    if (ring && parts <= 512) return launch_grad_ring<ST, k8, 2, 256, 4>(a, sm, s);
    if (ring && parts <= 1024) return launch_grad_ring<ST, k8, 2, 512, 4>(a, sm, s);
    if constexpr (k8) {  // (without rows in 8 bits every aligned row takes the ring)
      if (!ring && parts <= 128) return launch_grad<ST, true, k8, 1, 128>(a, sm, s);
      if (!ring && parts <= 256) return launch_grad<ST, true, k8, 2, 128>(a, sm, s);
      if (!ring && parts <= 512) return launch_grad<ST, true, k8, 2, 256>(a, sm, s);
      if (!ring && parts <= 1024) return launch_grad<ST, true, k8, 2, 512>(a, sm, s);
    }
    if constexpr (Stor<ST>::kBytes == 4)
      if (ring && parts <= 2048) return launch_grad_ring<ST, k8, 4, 512, 2>(a, sm, s);
  }
  parts = groups_of(a.D) * 32;
  if (parts <= 32) return launch_grad<ST, false, k8, 1, 32>(a, sm, s);
  if (parts <= 64) return launch_grad<ST, false, k8, 2, 32>(a, sm, s);
  if (parts <= 128) return launch_grad<ST, false, k8, 1, 128>(a, sm, s);
  if (parts <= 256) return launch_grad<ST, false, k8, 2, 128>(a, sm, s);
  if (parts <= 512) return launch_grad<ST, false, k8, 2, 256>(a, sm, s);
  if (parts <= 1024) return launch_grad<ST, false, k8, 2, 512>(a, sm, s);
  if (parts <= 2048) return launch_grad<ST, false, k8, 4, 512>(a, sm, s);
  *taken = false;
  return cudaSuccess;
}

template <class ST>
cudaError_t grad_typed(const RmsGradArgs& a, int sm, cudaStream_t s) {
  if (a.N == 0) return join(a, 0, s);
  constexpr int es = Stor<ST>::kBytes, VE = 16 / es;
  const bool k8 = a.total == nullptr;
  const bool even = rows_aligned({a.dy, a.d_total, a.total, a.weight, a.dx},
                                 {a.D, a.dy_stride, a.d_total_stride, a.total_stride}, es) &&
                    aligned_to(a.total8, VE);
  const bool ring = !k8 || (a.D % 16 == 0 && aligned_to(a.total8, 16));  // (bulk copies of rows in 8 bits)
  bool taken = false;
  const cudaError_t done = k8 ? grad_width<ST, true>(a, even, ring, a.D / VE, sm, s, &taken)
                              : grad_width<ST, false>(a, even, ring, a.D / VE, sm, s, &taken);
  if (taken) return done;
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

}  // namespace

cudaError_t run_rms_norm(const RmsArgs& a, int sm, cudaStream_t s) {
  return a.bf16_io ? norm_typed<bf16>(a, sm, s) : norm_typed<float>(a, sm, s);
}

// the most partial sums any variant leaves: CTAs of 128 threads, or slices
size_t rms_norm_backward_workspace(int64_t N, int64_t D, int sm) {
  const int64_t parts = std::max(grad_grid(N, 128, 1, sm), div_up(N, slice_rows(N, D, sm)));
  return (size_t)parts * (size_t)D * sizeof(float);
}

cudaError_t run_rms_norm_backward(const RmsGradArgs& a, int sm, cudaStream_t s) {
  return a.bf16_io ? grad_typed<bf16>(a, sm, s) : grad_typed<float>(a, sm, s);
}

cudaError_t status_rms(unsigned int* word, bool clear) { return unit_status(word, clear); }

}  // namespace rlca
