// Layer norm and its gradient.
//
//   y = (x - mean) rstd w + b
//   dx = rstd (g - mean(g) - xh mean(g xh)),  g = dy w,  xh = (x - mean) rstd
//   dw = sum over rows of dy xh,  db = sum over rows of dy
//
// Both directions are bound by HBM: the forward pass reads and writes a row
// once, the backward pass reads two rows and writes one.  A row is held in
// registers (VPT vectors of 16 bytes a thread, TPR threads a row), so the
// variance is the mean square of the centred row at no second read --
// sum(x^2) - mean^2 would cancel for rows whose mean is large against their
// spread.  CTAs are persistent: a thread keeps its columns' weight and bias
// (and, backward, its columns' sums of dw and db) in registers over all its
// rows, and loads the next row before it works on the current one.
#include <algorithm>

#include "policy.h"
#include "reduce.cuh"
#include "tma.cuh"

namespace rlca {

namespace {

// VE consecutive elements of type ST as they lie in memory, from element i of
// the n that there are (in the index-check build a miss reads zero, and is not
// written)
template <class ST, int VE>
struct Pack;
template <>
struct Pack<float, 4> {
  using Raw = float4;
  __device__ static Raw load(const float* p, int64_t i, int64_t n) {
    return span_in_range(i, 4, n) ? __ldg(reinterpret_cast<const float4*>(p + i)) : zero();
  }
  __device__ static Raw zero() { return make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ static void open(const Raw& r, float* v) { v[0] = r.x, v[1] = r.y, v[2] = r.z, v[3] = r.w; }
  __device__ static void store(float* p, int64_t i, int64_t n, const float* v) {
    if (span_in_range(i, 4, n)) Stor<float>::st4(p, i, v);
  }
};
template <>
struct Pack<bf16, 8> {
  using Raw = uint4;
  __device__ static Raw load(const float* p, int64_t i, int64_t n) {
    return span_in_range(i, 8, n) ? __ldg(reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(p) + i)) : zero();
  }
  __device__ static Raw zero() { return make_uint4(0u, 0u, 0u, 0u); }
  __device__ static void open(const Raw& r, float* v) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) v[2 * k] = __uint_as_float(w[k] << 16), v[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
  }
  __device__ static void store(float* p, int64_t i, int64_t n, const float* v) {
    if (span_in_range(i, 8, n)) Stor<bf16>::st8(p, i, v);
  }
};
template <>
struct Pack<float, 1> {
  using Raw = float;
  __device__ static Raw load(const float* p, int64_t i, int64_t n) { return in_range(i, n) ? __ldg(p + i) : zero(); }
  __device__ static Raw zero() { return 0.f; }
  __device__ static void open(const Raw& r, float* v) { v[0] = r; }
  __device__ static void store(float* p, int64_t i, int64_t n, const float* v) {
    if (in_range(i, n)) p[i] = v[0];
  }
};
template <>
struct Pack<bf16, 1> {
  using Raw = uint16_t;  // widened when used: a conversion at the load would wait for it
  __device__ static Raw load(const float* p, int64_t i, int64_t n) {
    return in_range(i, n) ? __ldg(reinterpret_cast<const uint16_t*>(p) + i) : zero();
  }
  __device__ static Raw zero() { return 0; }
  __device__ static void open(const Raw& r, float* v) { v[0] = Stor<bf16>::from_bits(r); }
  __device__ static void store(float* p, int64_t i, int64_t n, const float* v) {
    if (in_range(i, n)) Stor<bf16>::st(p, i, v[0]);
  }
};

// ... single elements, and the elements from the first to the last of a
// matrix's rows
template <class ST>
__device__ __forceinline__ float load1(const float* p, int64_t i, int64_t n) {
  return in_range(i, n) ? Stor<ST>::ld(p, i) : 0.f;
}
template <class ST>
__device__ __forceinline__ void store1(float* p, int64_t i, int64_t n, float v) {
  if (in_range(i, n)) Stor<ST>::st(p, i, v);
}
// a column's partial sums of dw and db, `apart` elements apart
__device__ __forceinline__ void store2(float* ws, int64_t i, int64_t apart, int64_t n, float dw, float db) {
  if (in_range(i, n) && in_range(i + apart, n)) ws[i] = dw, ws[i + apart] = db;
}
__device__ __forceinline__ int64_t extent(int64_t rows, int64_t width, int64_t stride) { return (rows - 1) * stride + width; }

// Threads of a CTA: whole warps of rows, or one row over the CTA.
__host__ __device__ constexpr int cta_threads(int tpr) { return tpr < 128 ? 128 : tpr; }

// CTAs of `threads` threads an SM is to hold in the forward pass, by the
// values a thread has in registers.  (bfloat16 32768 x 4096, 32 values: 512
// threads 90 us, 768 121 us -- they spill --, 256 115 us; 131072 x 512, 16 values:
// 768 threads 49 us, 1024 59 us, 512 55 us.)
__host__ __device__ constexpr int norm_resident(int threads, int values) {
  const int n = (values >= 32 ? 512 : values >= 16 ? 768 : 1024) / threads;
  return n > 0 ? n : 1;
}

// Sum of a row's values over its TPR threads.  `slot` selects one of two
// scratch rows: a slot is written again only after a barrier that follows
// its last read, so one barrier a sum is enough.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float (*scratch)[32], int slot) {
  v = warp_sum(v);
  if constexpr (TPR > 32) {
    constexpr int W = TPR / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) scratch[slot][warp] = v;
    __syncthreads();
    v = lane < W ? scratch[slot][lane] : 0.f;
    v = warp_sum(v);
  }
  return v;
}

// ---------------------------------------------------------------------------
// Forward: bound by HBM.  65536 x 4096 bfloat16: 166 us, 6.46 TB/s, 0.97 of
// the measured copy rate; 32768 x 4096: 128 threads x 4 vectors a row 91 us,
// 256 x 2 97 us, 512 x 1 138 us (more threads wait for the same two sums).
// Single elements (8000 x 7001 bfloat16): 3.2 TB/s, bound by the loads' issue.
// (The row loop's trip count is the same for all threads of a CTA
// where a row takes the whole CTA, so the barriers match.)
// ---------------------------------------------------------------------------
template <class ST, int VE, int VPT, int TPR>
__global__ void __launch_bounds__(cta_threads(TPR), norm_resident(cta_threads(TPR), VPT * VE))
    norm_kernel(NormArgs a) {
  using P = Pack<ST, VE>;
  constexpr int ROWS = cta_threads(TPR) / TPR;  // rows of a CTA at a time
  __shared__ float scratch[2][32];
  const int lane = threadIdx.x % TPR;
  const int nv = (int)(a.D / VE);
  const float inv_d = 1.f / (float)a.D;
  const int64_t step = (int64_t)gridDim.x * ROWS, x_size = extent(a.N, a.D, a.x_stride);
  int64_t row = (int64_t)blockIdx.x * ROWS + threadIdx.x / TPR;
  pdl_trigger();
  pdl_wait();

  typename P::Raw w[VPT], b[VPT], x[VPT];
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int v = lane + j * TPR;
    const bool on = v < nv;
    w[j] = on ? P::load(a.weight, (int64_t)v * VE, a.D) : P::zero();
    b[j] = on && a.bias ? P::load(a.bias, (int64_t)v * VE, a.D) : P::zero();
    x[j] = on && row < a.N ? P::load(a.x, row * a.x_stride + (int64_t)v * VE, x_size) : P::zero();
  }
  for (; row < a.N; row += step) {
    float f[VPT][VE];
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      P::open(x[j], f[j]);
#pragma unroll
      for (int e = 0; e < VE; ++e) s += f[j][e];
    }
    const int64_t next = row + step;
    if (next < a.N) {
#pragma unroll
      for (int j = 0; j < VPT; ++j)
        if (lane + j * TPR < nv) x[j] = P::load(a.x, next * a.x_stride + (int64_t)(lane + j * TPR) * VE, x_size);
    }
    const float mean = row_sum<TPR>(s, scratch, 0) * inv_d;
    float q = 0.f;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const bool on = lane + j * TPR < nv;
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        f[j][e] = on ? f[j][e] - mean : 0.f;
        q = fmaf(f[j][e], f[j][e], q);
      }
    }
    const float rstd = rsqrtf(row_sum<TPR>(q, scratch, 1) * inv_d + a.eps);
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int v = lane + j * TPR;
      float fw[VE], fb[VE];
      P::open(w[j], fw);
      P::open(b[j], fb);
#pragma unroll
      for (int e = 0; e < VE; ++e) f[j][e] = fmaf(f[j][e] * rstd, fw[e], fb[e]);
      if (v < nv) P::store(a.y, row * a.D + (int64_t)v * VE, a.N * a.D, f[j]);
    }
    if (lane == 0 && in_range(row, a.N)) {
      if (a.mean) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = rstd;
    }
  }
}

// rows too long for registers: three passes over the row
constexpr int kLongThreads = 512;
template <class ST>
__global__ void __launch_bounds__(kLongThreads) norm_long_kernel(NormArgs a) {
  pdl_trigger();
  pdl_wait();
  __shared__ float scratch[32];
  const int64_t i = blockIdx.x, x_size = extent(a.N, a.D, a.x_stride);
  const float inv_d = 1.f / (float)a.D;
  const int64_t at = i * a.x_stride;
  float s = 0.f;
  for (int64_t c = threadIdx.x; c < a.D; c += kLongThreads) s += load1<ST>(a.x, at + c, x_size);
  const float mean = cta_sum(s, scratch) * inv_d;
  float q = 0.f;
  for (int64_t c = threadIdx.x; c < a.D; c += kLongThreads) {
    const float d = load1<ST>(a.x, at + c, x_size) - mean;
    q += d * d;
  }
  const float rstd = rsqrtf(cta_sum(q, scratch) * inv_d + a.eps);
  for (int64_t c = threadIdx.x; c < a.D; c += kLongThreads) {
    const float xh = (load1<ST>(a.x, at + c, x_size) - mean) * rstd;
    const float b = a.bias ? load1<ST>(a.bias, c, a.D) : 0.f;
    store1<ST>(a.y, i * a.D + c, a.N * a.D, xh * load1<ST>(a.weight, c, a.D) + b);
  }
  if (threadIdx.x == 0 && in_range(i, a.N)) {
    if (a.mean) a.mean[i] = mean;
    if (a.rstd) a.rstd[i] = rstd;
  }
}

// ---------------------------------------------------------------------------
// Backward: bound by HBM.  Rows next to each other in a warp or a CTA, the
// next one loaded into registers ahead: for rows up to 64 vectors and for rows
// of single elements.  (262144 x 256 bfloat16: 91 us, 4.4 TB/s: 94 registers allow
// 20 warps an SM, each with one row, 1 KB, on its way -- DRAM 59% busy, the issue
// slots 51%.)  Longer rows of vectors take the ring below: 131072 x 512, 64
// vectors a row, 82 us here and 99 us on the ring; 65536 x 1024, 95 and 96 us;
// 32768 x 4096, 156 and 144 us.  Each CTA leaves the sums of dw and db over its rows in
// ws[CTA][2][D]; a second kernel joins them in order.
// ---------------------------------------------------------------------------
// (threads an SM, by the values a thread has: 32768 x 4096 bfloat16, 16 values, 512
// threads 144 us, 384 191 us, 768 205 us; 262144 x 256, 8 values, 640 threads 91
// us, 512 102 us, 768 87 us, 1024 97 us, but 5001 x 1001 float32 21, 23, 23 and 27 us.)
__host__ __device__ constexpr int grad_resident(int threads, int values) {
  const int n = (values >= 32 ? 384 : values >= 16 ? 512 : 640) / threads;
  return n > 0 ? n : 1;
}

template <class ST, int VE, int VPT, int TPR>
__global__ void __launch_bounds__(cta_threads(TPR), grad_resident(cta_threads(TPR), VPT * VE)) norm_grad_kernel(NormGradArgs a) {
  using P = Pack<ST, VE>;
  constexpr int ROWS = cta_threads(TPR) / TPR;
  __shared__ float scratch[2][2][32];
  const int lane = threadIdx.x % TPR;
  const int nv = (int)(a.D / VE);
  const float inv_d = 1.f / (float)a.D;
  const int64_t step = (int64_t)gridDim.x * ROWS;
  int64_t row = (int64_t)blockIdx.x * ROWS + threadIdx.x / TPR;
  const int64_t x_size = extent(a.N, a.D, a.x_stride), dy_size = extent(a.N, a.D, a.dy_stride);
  const bool sums = a.dweight != nullptr || a.dbias != nullptr;
  pdl_trigger();
  pdl_wait();

  typename P::Raw w[VPT], x[VPT], dy[VPT];
  float dw[VPT][VE], db[VPT][VE];
  float mean = 0.f, rstd = 0.f;
  if (row < a.N) mean = a.mean[row], rstd = a.rstd[row];
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int v = lane + j * TPR;
    const bool on = v < nv;
    w[j] = on ? P::load(a.weight, (int64_t)v * VE, a.D) : P::zero();
    x[j] = on && row < a.N ? P::load(a.x, row * a.x_stride + (int64_t)v * VE, x_size) : P::zero();
    dy[j] = on && row < a.N ? P::load(a.dy, row * a.dy_stride + (int64_t)v * VE, dy_size) : P::zero();
#pragma unroll
    for (int e = 0; e < VE; ++e) dw[j][e] = db[j][e] = 0.f;
  }
  int slot = 0;
  for (; row < a.N; row += step) {
    float xh[VPT][VE], g[VPT][VE];
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      float fw[VE];
      P::open(x[j], xh[j]);
      P::open(dy[j], g[j]);
      P::open(w[j], fw);
      const bool on = lane + j * TPR < nv;
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        xh[j][e] = on ? (xh[j][e] - mean) * rstd : 0.f;
        dw[j][e] = fmaf(g[j][e], xh[j][e], dw[j][e]);
        db[j][e] += g[j][e];
        g[j][e] *= fw[e];
        s1 += g[j][e];
        s2 = fmaf(g[j][e], xh[j][e], s2);
      }
    }
    const float r = rstd;
    const int64_t next = row + step;
    if (next < a.N) {
      mean = a.mean[next], rstd = a.rstd[next];
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        const int v = lane + j * TPR;
        if (v < nv) {
          x[j] = P::load(a.x, next * a.x_stride + (int64_t)v * VE, x_size);
          dy[j] = P::load(a.dy, next * a.dy_stride + (int64_t)v * VE, dy_size);
        }
      }
    }
    if (a.dx == nullptr) continue;
    s1 = warp_sum(s1);
    s2 = warp_sum(s2);
    if constexpr (TPR > 32) {
      // both sums over one barrier; the slots alternate from row to row, so
      // one is written again only after the other row's barrier
      const int warp = threadIdx.x >> 5, l = threadIdx.x & 31;
      if (l == 0) scratch[slot][0][warp] = s1, scratch[slot][1][warp] = s2;
      __syncthreads();
      s1 = warp_sum(l < TPR / 32 ? scratch[slot][0][l] : 0.f);
      s2 = warp_sum(l < TPR / 32 ? scratch[slot][1][l] : 0.f);
      slot ^= 1;
    }
    s1 *= inv_d;
    s2 *= inv_d;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int v = lane + j * TPR;
#pragma unroll
      for (int e = 0; e < VE; ++e) g[j][e] = r * (g[j][e] - s1 - xh[j][e] * s2);
      if (v < nv) P::store(a.dx, row * a.D + (int64_t)v * VE, a.N * a.D, g[j]);
    }
  }
  if (!sums) return;
  const int64_t at = (int64_t)blockIdx.x * 2 * a.D, ws_size = 2 * a.D * (int64_t)gridDim.x;
  if constexpr (ROWS == 1) {
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int v = lane + j * TPR;
      if (v < nv) {
#pragma unroll
        for (int e = 0; e < VE; ++e) store2(a.ws, at + v * VE + e, a.D, ws_size, dw[j][e], db[j][e]);
      }
    }
  } else {
    // the CTA's rows side by side, added in order
    __shared__ float acc[2][VPT * TPR * VE];
    for (int k = 0; k < ROWS; ++k) {
      if (threadIdx.x / TPR == k) {
#pragma unroll
        for (int j = 0; j < VPT; ++j)
#pragma unroll
          for (int e = 0; e < VE; ++e) {
            const int c = (lane + j * TPR) * VE + e;
            if (!in_range(c, VPT * TPR * VE)) continue;
            acc[0][c] = dw[j][e] + (k > 0 ? acc[0][c] : 0.f);
            acc[1][c] = db[j][e] + (k > 0 ? acc[1][c] : 0.f);
          }
      }
      __syncthreads();
    }
    for (int c = threadIdx.x; c < a.D; c += cta_threads(TPR)) store2(a.ws, at + c, a.D, ws_size, acc[0][c], acc[1][c]);
  }
}

// The same for rows of a CTA of their own, fed by bulk copies (32768 x 4096
// bfloat16: 143 us with the join, 5.6 TB/s, against 156 us with the next row
// in registers; two such CTAs an SM are all that 120 registers allow): thread 0 keeps
// kRingRows - 1 rows of x and dy on their way into shared memory, so what is
// in flight does not depend on the registers that the columns' sums leave.  A
// stage is filled again after the barrier that follows its reads (the one the
// row's sums need anyway).  A wait that gives up is recorded in the status
// word; the rows are then walked without further copies or waits.
template <class ST, int VE, int VPT, int TPR, int kRingRows>
__global__ void __launch_bounds__(TPR, grad_resident(TPR, VPT * VE)) norm_grad_ring_kernel(NormGradArgs a) {
  using P = Pack<ST, VE>;
  extern __shared__ __align__(128) unsigned char ring_rows[];  // [kRingRows][x, dy][D]
  __shared__ __align__(8) uint64_t full[kRingRows];
  __shared__ float scratch[2][2][32];
  const int lane = threadIdx.x, warp = lane >> 5, l = lane & 31;
  const int nv = (int)(a.D / VE);
  const uint32_t row_bytes = (uint32_t)(a.D * Stor<ST>::kBytes);
  const float inv_d = 1.f / (float)a.D;
  const int64_t step = gridDim.x;
  pdl_trigger();
  if (lane == 0) {
    for (int i = 0; i < kRingRows; ++i) mbar_init(&full[i], 1);
    mbar_fence_init();
  }
  __syncthreads();
  pdl_wait();

  const auto fill = [&](int stage, int64_t row) {
    // (an index that is off is recorded, and the row is waited for in vain)
    if (!in_range(stage, kRingRows) || !in_range(row, a.N)) return;
    unsigned char* to = ring_rows + (size_t)stage * 2 * row_bytes;
    mbar_arrive_expect_tx(&full[stage], 2 * row_bytes);
    bulk_load(to, reinterpret_cast<const unsigned char*>(a.x) + row * a.x_stride * Stor<ST>::kBytes, row_bytes, &full[stage]);
    bulk_load(to + row_bytes, reinterpret_cast<const unsigned char*>(a.dy) + row * a.dy_stride * Stor<ST>::kBytes, row_bytes,
              &full[stage]);
  };
  int64_t row = blockIdx.x;
  if (lane == 0) {
    for (int i = 0; i < kRingRows - 1; ++i)
      if (row + i * step < a.N) fill(i, row + i * step);
  }
  typename P::Raw w[VPT];
  float dw[VPT][VE], db[VPT][VE];
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int v = lane + j * TPR;
    w[j] = v < nv ? P::load(a.weight, (int64_t)v * VE, a.D) : P::zero();
#pragma unroll
    for (int e = 0; e < VE; ++e) dw[j][e] = db[j][e] = 0.f;
  }
  float mean = 0.f, rstd = 0.f;
  if (row < a.N) mean = a.mean[row], rstd = a.rstd[row];
  int slot = 0;
  FillRing<kRingRows> ring;
  for (; row < a.N; row += step) {
    // the stage before this one was read in the last round
    if (lane == 0 && ring.ok && row + (kRingRows - 1) * step < a.N) fill(ring.fill_stage(), row + (kRingRows - 1) * step);
    if (ring.ok) ring.ok = mbar_wait_bounded(&full[ring.stage], ring.phase);
    const unsigned char* at = ring_rows + (size_t)ring.stage * 2 * row_bytes;
    float xh[VPT][VE], g[VPT][VE];
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int v = lane + j * TPR;
      const bool on = v < nv;
      typename P::Raw x = P::zero(), dy = P::zero();
      if (on && span_in_range((int64_t)ring.stage * 2 * row_bytes + v * 16, row_bytes + 16, (int64_t)kRingRows * 2 * row_bytes)) {
        x = *reinterpret_cast<const typename P::Raw*>(at + v * 16);
        dy = *reinterpret_cast<const typename P::Raw*>(at + row_bytes + v * 16);
      }
      float fw[VE];
      P::open(x, xh[j]);
      P::open(dy, g[j]);
      P::open(w[j], fw);
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        xh[j][e] = on ? (xh[j][e] - mean) * rstd : 0.f;
        dw[j][e] = fmaf(g[j][e], xh[j][e], dw[j][e]);
        db[j][e] += g[j][e];
        g[j][e] *= fw[e];
        s1 += g[j][e];
        s2 = fmaf(g[j][e], xh[j][e], s2);
      }
    }
    const float r = rstd;
    if (row + step < a.N) mean = a.mean[row + step], rstd = a.rstd[row + step];
    s1 = warp_sum(s1);
    s2 = warp_sum(s2);
    if (l == 0) scratch[slot][0][warp] = s1, scratch[slot][1][warp] = s2;
    __syncthreads();
    s1 = warp_sum(l < TPR / 32 ? scratch[slot][0][l] : 0.f) * inv_d;
    s2 = warp_sum(l < TPR / 32 ? scratch[slot][1][l] : 0.f) * inv_d;
    slot ^= 1;
    ring.next();
    if (a.dx == nullptr) continue;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int v = lane + j * TPR;
#pragma unroll
      for (int e = 0; e < VE; ++e) g[j][e] = r * (g[j][e] - s1 - xh[j][e] * s2);
      if (v < nv) P::store(a.dx, row * a.D + (int64_t)v * VE, a.N * a.D, g[j]);
    }
  }
  // (copies still on their way after a wait gave up land before the CTA ends)
  if (!ring.ok && lane == 0)
    for (int i = 0; i < kRingRows; ++i) mbar_wait_bounded(&full[i], ring.last_fill(i));
  if (a.dweight == nullptr && a.dbias == nullptr) return;
  const int64_t to = (int64_t)blockIdx.x * 2 * a.D, ws_size = 2 * a.D * (int64_t)gridDim.x;
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int v = lane + j * TPR;
    if (v < nv) {
#pragma unroll
      for (int e = 0; e < VE; ++e) store2(a.ws, to + v * VE + e, a.D, ws_size, dw[j][e], db[j][e]);
    }
  }
}

// rows too long for registers
template <class ST>
__global__ void __launch_bounds__(kLongThreads) norm_grad_long_kernel(NormGradArgs a) {
  pdl_trigger();
  pdl_wait();
  __shared__ float scratch[32];
  const int64_t i = blockIdx.x, x_size = extent(a.N, a.D, a.x_stride), dy_size = extent(a.N, a.D, a.dy_stride);
  const float inv_d = 1.f / (float)a.D;
  const float mean = a.mean[i], rstd = a.rstd[i];
  float s1 = 0.f, s2 = 0.f;
  for (int64_t c = threadIdx.x; c < a.D; c += kLongThreads) {
    const float g = load1<ST>(a.dy, i * a.dy_stride + c, dy_size) * load1<ST>(a.weight, c, a.D);
    const float xh = (load1<ST>(a.x, i * a.x_stride + c, x_size) - mean) * rstd;
    s1 += g;
    s2 += g * xh;
  }
  s1 = cta_sum(s1, scratch) * inv_d;
  s2 = cta_sum(s2, scratch) * inv_d;
  for (int64_t c = threadIdx.x; c < a.D; c += kLongThreads) {
    const float g = load1<ST>(a.dy, i * a.dy_stride + c, dy_size) * load1<ST>(a.weight, c, a.D);
    const float xh = (load1<ST>(a.x, i * a.x_stride + c, x_size) - mean) * rstd;
    store1<ST>(a.dx, i * a.D + c, a.N * a.D, rstd * (g - s1 - xh * s2));
  }
}

// ... and their sums of dw and db, a slice of rows a CTA
constexpr int kSliceThreads = 256;
template <class ST>
__global__ void __launch_bounds__(kSliceThreads)
    norm_grad_slices_kernel(NormGradArgs a, int64_t col_blocks, int64_t slice_rows) {
  pdl_trigger();
  pdl_wait();
  const int64_t slice = blockIdx.x / col_blocks;
  const int64_t c = (blockIdx.x % col_blocks) * kSliceThreads + threadIdx.x;
  if (c >= a.D) return;
  const int64_t i1 = min(a.N, (slice + 1) * slice_rows);
  const int64_t x_size = extent(a.N, a.D, a.x_stride), dy_size = extent(a.N, a.D, a.dy_stride);
  float dw = 0.f, db = 0.f;
  for (int64_t i = slice * slice_rows; i < i1; ++i) {
    const float dy = load1<ST>(a.dy, i * a.dy_stride + c, dy_size);
    dw += dy * ((load1<ST>(a.x, i * a.x_stride + c, x_size) - a.mean[i]) * a.rstd[i]);
    db += dy;
  }
  store2(a.ws, 2 * slice * a.D + c, a.D, 2 * a.D * (gridDim.x / col_blocks), dw, db);
}

// (10 MB of partial sums at 32768 x 4096, from L2: about 5 us.)
// The partial sums of 32 columns, joined by 32 x 32 threads: warp k adds the
// partials k, k + 32, ... of its columns, then the warps' sums are added in
// order.  blockIdx.x < col_blocks: dw, else db.
__global__ void __launch_bounds__(1024)
    norm_grad_join_kernel(const float* ws, int64_t parts, int64_t D, float* dweight, float* dbias, bool bf16_io) {
  pdl_trigger();
  pdl_wait();
  __shared__ float acc[32][33];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t col_blocks = (D + 31) / 32;
  const int which = blockIdx.x >= col_blocks;
  float* out = which ? dbias : dweight;
  if (out == nullptr) return;
  const int64_t c = (blockIdx.x - which * col_blocks) * 32 + lane;
  float s = 0.f;
  if (c < D) {
    constexpr int B = 8;  // loads in flight
    for (int64_t k0 = warp; k0 < parts; k0 += 32 * B) {
      float v[B];
#pragma unroll
      for (int u = 0; u < B; ++u) v[u] = k0 + 32 * u < parts ? load1<float>(ws, (2 * (k0 + 32 * u) + which) * D + c, 2 * parts * D) : 0.f;
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
  if (bf16_io) store1<bf16>(out, c, D, s);
  else store1<float>(out, c, D, s);
}

// ---------------------------------------------------------------------------
// Which variant: vectors of 16 bytes where every row of every array starts on
// such a boundary, else single elements; the fewest threads a row with up to
// 4 vectors (forward; 2 backward, whose sums take the registers) or 8 single
// elements a thread.
// ---------------------------------------------------------------------------
bool rows_aligned(std::initializer_list<const void*> bases, std::initializer_list<int64_t> strides, int es) {
  for (const void* p : bases)
    if (((uintptr_t)p & 15) != 0) return false;
  for (int64_t s : strides)
    if ((s * es) % 16 != 0) return false;
  return true;
}

template <class ST, int VE, int VPT, int TPR>
cudaError_t launch_norm(const NormArgs& a, int sm, cudaStream_t s) {
  constexpr int T = cta_threads(TPR), R = norm_resident(T, VPT * VE);
  const int64_t grid = std::min<int64_t>(div_up(a.N, T / TPR), (int64_t)R * sm);
  return launch_pdl(norm_kernel<ST, VE, VPT, TPR>, grid, T, 0, s, a);
}

template <class ST>
cudaError_t norm_typed(const NormArgs& a, int sm, cudaStream_t s) {
  constexpr int VE = 16 / Stor<ST>::kBytes;
  if (rows_aligned({a.x, a.y, a.weight, a.bias}, {a.D, a.x_stride}, Stor<ST>::kBytes)) {
    const int64_t nv = a.D / VE;
    if (nv <= 32) return launch_norm<ST, VE, 1, 32>(a, sm, s);
    if (nv <= 64) return launch_norm<ST, VE, 2, 32>(a, sm, s);
    if (nv <= 128) return launch_norm<ST, VE, 4, 32>(a, sm, s);
    if (nv <= 256) return launch_norm<ST, VE, 2, 128>(a, sm, s);
    if (nv <= 512) return launch_norm<ST, VE, 4, 128>(a, sm, s);
    if (nv <= 1024) return launch_norm<ST, VE, 4, 256>(a, sm, s);
    if (nv <= 2048) return launch_norm<ST, VE, 4, 512>(a, sm, s);
  } else {
    if (a.D <= 32) return launch_norm<ST, 1, 1, 32>(a, sm, s);
    if (a.D <= 256) return launch_norm<ST, 1, 8, 32>(a, sm, s);
    if (a.D <= 1024) return launch_norm<ST, 1, 8, 128>(a, sm, s);
    if (a.D <= 2048) return launch_norm<ST, 1, 8, 256>(a, sm, s);
    if (a.D <= 4096) return launch_norm<ST, 1, 8, 512>(a, sm, s);
    if (a.D <= 8192) return launch_norm<ST, 1, 16, 512>(a, sm, s);
  }
  return launch_pdl(norm_long_kernel<ST>, a.N, kLongThreads, 0, s, a);
}

// CTAs of a backward launch of T threads, R rows at a time: those that fit
// the SMs, but four rounds of rows each where that still gives every SM one
// (each CTA leaves 2 D partial sums to be joined)
int64_t grad_grid(int64_t N, int T, int R, int values, int sm) {
  const int64_t rounds = div_up(N, R);
  return std::min({rounds, (int64_t)grad_resident(T, values) * sm, std::max<int64_t>(sm, div_up(rounds, 4))});
}

cudaError_t join(const NormGradArgs& a, int64_t parts, cudaStream_t s) {
  if (a.dweight == nullptr && a.dbias == nullptr) return cudaSuccess;
  return launch_pdl(norm_grad_join_kernel, 2 * div_up(a.D, 32), 1024, 0, s, (const float*)a.ws, parts, a.D, a.dweight,
                    a.dbias, a.bf16_io);
}

template <class ST, int VE, int VPT, int TPR>
cudaError_t launch_grad(const NormGradArgs& a, int sm, cudaStream_t s) {
  constexpr int T = cta_threads(TPR);
  const int64_t grid = grad_grid(a.N, T, T / TPR, VPT * VE, sm);
  const cudaError_t e = launch_pdl(norm_grad_kernel<ST, VE, VPT, TPR>, grid, T, 0, s, a);
  return e == cudaSuccess ? join(a, grid, s) : e;
}

template <class ST, int VE, int VPT, int TPR, int kRingRows = 4>
cudaError_t launch_grad_ring(const NormGradArgs& a, int sm, cudaStream_t s) {
  const size_t smem = (size_t)kRingRows * 2 * a.D * Stor<ST>::kBytes;
  const auto kernel = norm_grad_ring_kernel<ST, VE, VPT, TPR, kRingRows>;
  static std::atomic<uint64_t> allowed;
  cudaError_t e = allow_smem(kernel, (size_t)kRingRows * 2 * TPR * VPT * 16, allowed);
  if (e != cudaSuccess) return e;
  const int64_t grid = grad_grid(a.N, TPR, 1, VPT * VE, sm);
  e = launch_pdl(kernel, grid, TPR, smem, s, a);
  return e == cudaSuccess ? join(a, grid, s) : e;
}

// rows of a slice of the long rows' first sum: enough slices to fill the SMs
int64_t slice_rows(int64_t N, int64_t D, int sm) {
  const int64_t want = std::max<int64_t>(1, 8 * (int64_t)sm / div_up(D, kSliceThreads));
  return std::max<int64_t>(1, div_up(N, want));
}

template <class ST>
cudaError_t grad_typed(const NormGradArgs& a, int sm, cudaStream_t s) {
  if (a.N == 0) return join(a, 0, s);
  constexpr int VE = 16 / Stor<ST>::kBytes;
  if (rows_aligned({a.x, a.dy, a.dx, a.weight}, {a.D, a.x_stride, a.dy_stride}, Stor<ST>::kBytes)) {
    const int64_t nv = a.D / VE;
    if (nv <= 32) return launch_grad<ST, VE, 1, 32>(a, sm, s);
    if (nv <= 64) return launch_grad<ST, VE, 2, 32>(a, sm, s);
    if (nv <= 128) return launch_grad_ring<ST, VE, 1, 128>(a, sm, s);
    if (nv <= 256) return launch_grad_ring<ST, VE, 2, 128>(a, sm, s);
    if (nv <= 512) return launch_grad_ring<ST, VE, 2, 256>(a, sm, s);
    if (nv <= 1024) return launch_grad_ring<ST, VE, 2, 512>(a, sm, s);
    if constexpr (VE == 4)  // (three rows of 32 KB, twice, fill the shared memory)
      if (nv <= 2048) return launch_grad_ring<ST, VE, 4, 512, 3>(a, sm, s);
  } else {
    if (a.D <= 32) return launch_grad<ST, 1, 1, 32>(a, sm, s);
    if (a.D <= 256) return launch_grad<ST, 1, 8, 32>(a, sm, s);
    if (a.D <= 1024) return launch_grad<ST, 1, 8, 128>(a, sm, s);
    if (a.D <= 2048) return launch_grad<ST, 1, 8, 256>(a, sm, s);
    if (a.D <= 4096) return launch_grad<ST, 1, 8, 512>(a, sm, s);
    if (a.D <= 8192) return launch_grad<ST, 1, 16, 512>(a, sm, s);
  }
  if (a.dx != nullptr) {
    const cudaError_t e = launch_pdl(norm_grad_long_kernel<ST>, a.N, kLongThreads, 0, s, a);
    if (e != cudaSuccess) return e;
  }
  if (a.dweight == nullptr && a.dbias == nullptr) return cudaSuccess;
  const int64_t col_blocks = div_up(a.D, kSliceThreads), rows = slice_rows(a.N, a.D, sm), slices = div_up(a.N, rows);
  const cudaError_t e =
      launch_pdl(norm_grad_slices_kernel<ST>, slices * col_blocks, kSliceThreads, 0, s, a, col_blocks, rows);
  return e == cudaSuccess ? join(a, slices, s) : e;
}

}  // namespace

cudaError_t run_layer_norm(const NormArgs& a, int sm, cudaStream_t s) {
  return a.bf16_io ? norm_typed<bf16>(a, sm, s) : norm_typed<float>(a, sm, s);
}

// the most partial sums any variant leaves: CTAs of 128 threads, or slices
size_t layer_norm_backward_workspace(int64_t N, int64_t D, int sm) {
  const int64_t parts = std::max(grad_grid(N, 128, 1, 1, sm), div_up(N, slice_rows(N, D, sm)));
  return (size_t)parts * 2 * (size_t)D * sizeof(float);
}

cudaError_t run_layer_norm_backward(const NormGradArgs& a, int sm, cudaStream_t s) {
  return a.bf16_io ? grad_typed<bf16>(a, sm, s) : grad_typed<float>(a, sm, s);
}

cudaError_t status_norm(unsigned int* word, bool clear) { return unit_status(word, clear); }

}  // namespace rlca
