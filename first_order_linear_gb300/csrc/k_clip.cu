// Global gradient norm over many tensors, and the tensors scaled by it.
//
// Bound by HBM: the norm reads everything before the first element can be
// scaled, so what does not fit in L2 is read twice and written once.  1.34 G
// elements (2.7 GB) in 50 tensors: 1200 us for 8.05 GB, 6.7 TB/s, the measured
// copy rate; one load a thread in flight took 2998 us.  Chunks of 32768
// elements of all tensors are dealt to 8 CTAs an SM, so neither one large
// tensor nor thousands of small ones leave SMs idle, and the whole list is two
// launches.  18 small tensors: 20 us on the device, launch latency.
#include <algorithm>

#include "policy.h"
#include "reduce.cuh"
#include "rlca.h"

namespace rlca {

namespace {

constexpr int kClipThreads = 256;
// elements of one tensor that one CTA takes at a time
constexpr int64_t kClipChunk = 32768;
// Tensors of one launch: their table travels as a kernel parameter (of at
// most 32,764 bytes), so a call writes no device memory for it.  Up to 64
// tensors take a small table: copying 28 KB of parameters twice costs the
// host 3 us.
constexpr int kClipTensors = 1000, kClipFewTensors = 64;

template <int CAP>
struct ClipTable {
  const void* grad[CAP];
  void* out[CAP];
  int64_t size[CAP];  // elements; negative: bfloat16
  // first chunk of each tensor (chunks of all tensors are numbered in a row)
  uint32_t first[CAP + 1];
  int count;
};
static_assert(sizeof(ClipTable<kClipTensors>) <= 32764 - 64, "kernel parameters");

struct ClipItem {
  const void* grad;
  void* out;
  int64_t at, n;  // first element and number of elements
  bool bf16_io;
};

// the piece of a tensor that chunk `chunk` of the launch is
template <int CAP>
__device__ __forceinline__ ClipItem clip_item(const ClipTable<CAP>& t, uint32_t chunk) {
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
  // (an empty chunk, so nothing is touched, where this one is not the tensor's)
  if (!in_range(lo, t.count) || !in_range(it.at, size) || !span_in_range(it.at, it.n, size)) it.at = it.n = 0;
  return it;
}

__device__ __forceinline__ float load_any(const void* p, int64_t i, bool bf) {
  // plain loads: in place, the kernel that reads also writes
  return bf ? Stor<bf16>::from_bits(static_cast<const uint16_t*>(p)[i]) : static_cast<const float*>(p)[i];
}
__device__ __forceinline__ void store_any(void* p, int64_t i, bool bf, float v) {
  if (bf) Stor<bf16>::st(static_cast<float*>(p), i, v);
  else static_cast<float*>(p)[i] = v;
}

// the four float32 or eight bfloat16 values of a 16-byte vector
template <bool BF>
__device__ __forceinline__ float vec_squares(const uint4& r) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
  float s = 0.f;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if constexpr (BF) {
      const float lo = __uint_as_float(w[k] << 16), hi = __uint_as_float(w[k] & 0xffff0000u);
      s = fmaf(lo, lo, s);
      s = fmaf(hi, hi, s);
    } else {
      const float v = __uint_as_float(w[k]);
      s = fmaf(v, v, s);
    }
  }
  return s;
}
template <bool BF>
__device__ __forceinline__ uint4 vec_scaled(const uint4& r, float f) {
  uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if constexpr (BF)
      w[k] = Stor<bf16>::pack2(__uint_as_float(w[k] << 16) * f, __uint_as_float(w[k] & 0xffff0000u) * f);
    else
      w[k] = __float_as_uint(__uint_as_float(w[k]) * f);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

constexpr int kClipUnroll = 8;  // 16-byte loads a thread has in flight

// sum of squares of n vectors, this thread's share
template <bool BF>
__device__ __forceinline__ float chunk_squares(const uint4* p, int n) {
  float s = 0.f;
  int k = threadIdx.x;
  for (; k + (kClipUnroll - 1) * kClipThreads < n; k += kClipUnroll * kClipThreads) {
    uint4 r[kClipUnroll];
#pragma unroll
    for (int u = 0; u < kClipUnroll; ++u) r[u] = __ldg(p + k + u * kClipThreads);
#pragma unroll
    for (int u = 0; u < kClipUnroll; ++u) s += vec_squares<BF>(r[u]);
  }
  for (; k < n; k += kClipThreads) s += vec_squares<BF>(__ldg(p + k));
  return s;
}

template <bool BF>
__device__ __forceinline__ void chunk_scale(const uint4* p, uint4* o, int n, float f) {
  int k = threadIdx.x;
  for (; k + (kClipUnroll - 1) * kClipThreads < n; k += kClipUnroll * kClipThreads) {
    uint4 r[kClipUnroll];
#pragma unroll
    for (int u = 0; u < kClipUnroll; ++u) r[u] = p[k + u * kClipThreads];
#pragma unroll
    for (int u = 0; u < kClipUnroll; ++u) o[k + u * kClipThreads] = vec_scaled<BF>(r[u], f);
  }
  for (; k < n; k += kClipThreads) o[k] = vec_scaled<BF>(p[k], f);
}

// A chunk as vectors with single elements around them: `lead` elements up to
// the first 16-byte boundary, `vecs` vectors, the rest.
struct ClipSpan {
  int64_t lead, vecs, tail;  // tail: first element after the vectors
};
__device__ __forceinline__ ClipSpan clip_span(const ClipItem& it) {
  const int es = it.bf16_io ? 2 : 4;
  const uintptr_t at = (uintptr_t)it.grad + (uintptr_t)it.at * es;
  ClipSpan s;
  s.lead = min((int64_t)(((16 - (at & 15)) & 15) / es), it.n);
  s.vecs = (it.n - s.lead) / (16 / es);
  s.tail = s.lead + s.vecs * (16 / es);
  // (only single elements, each checked, where the vectors are not the chunk's or not on their boundary)
  if (s.vecs > 0 && (!span_in_range(s.lead, s.vecs * (16 / es), it.n) || !in_range((int64_t)((at + s.lead * es) & 15), 1)))
    s.lead = s.vecs = s.tail = 0;
  return s;
}

// partials[CTA] = sum of squares over the CTA's chunks
template <int CAP>
__global__ void __launch_bounds__(kClipThreads)
    clip_squares_kernel(const __grid_constant__ ClipTable<CAP> t, double* partials) {
  pdl_trigger();
  pdl_wait();
  __shared__ double scratch[32];
  double total = 0.0;
  for (uint32_t chunk = blockIdx.x; chunk < t.first[t.count]; chunk += gridDim.x) {
    const ClipItem it = clip_item(t, chunk);
    const ClipSpan sp = clip_span(it);
    const int es = it.bf16_io ? 2 : 4;
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const unsigned char*>(it.grad) + (it.at + sp.lead) * es);
    // float32 over at most kClipChunk / kClipThreads squares, float64 beyond
    float s = it.bf16_io ? chunk_squares<true>(p, (int)sp.vecs) : chunk_squares<false>(p, (int)sp.vecs);
    if (threadIdx.x < sp.lead && in_range(threadIdx.x, it.n)) {
      const float g = load_any(it.grad, it.at + threadIdx.x, it.bf16_io);
      s = fmaf(g, g, s);
    }
    if (sp.tail + threadIdx.x < it.n) {
      const float g = load_any(it.grad, it.at + sp.tail + threadIdx.x, it.bf16_io);
      s = fmaf(g, g, s);
    }
    total += (double)s;
  }
  total = cta_sum(total, scratch);
  if (threadIdx.x == 0) partials[blockIdx.x] = total;
}

// The norm from all partial sums, in the same order by every CTA that asks.
__device__ __forceinline__ float norm_of(const double* partials, int64_t n) {
  __shared__ double scratch[32];
  double total = 0.0;
  for (int64_t k = threadIdx.x; k < n; k += kClipThreads) total += __ldg(partials + k);
  total = cta_sum(total, scratch);
  return (float)sqrt(total);
}

__global__ void __launch_bounds__(kClipThreads) clip_norm_kernel(const double* partials, int64_t n, float* norm) {
  pdl_trigger();
  pdl_wait();
  const float v = norm_of(partials, n);
  if (threadIdx.x == 0) *norm = v;
}

// Each CTA forms the norm by itself (at most 8 doubles an SM, from L2) rather
// than wait for a kernel that does; the first writes it.
template <int CAP>
__global__ void __launch_bounds__(kClipThreads, 5)
    clip_scale_kernel(const __grid_constant__ ClipTable<CAP> t, const double* partials, int64_t parts, float* norm,
                      float max_norm, float eps) {
  pdl_trigger();
  pdl_wait();
  const float n = norm_of(partials, parts);
  if (blockIdx.x == 0 && threadIdx.x == 0) *norm = n;
  const float scale = isfinite(n) ? fminf(1.f, max_norm / (n + eps)) : 1.f;
  // the squares walked the chunks upwards: downwards, the first ones here are
  // the last ones read there and still in L2
  const uint32_t chunks = t.first[t.count];
  for (uint32_t k = blockIdx.x; k < chunks; k += gridDim.x) {
    const ClipItem it = clip_item(t, chunks - 1 - k);
    if (scale == 1.f && it.out == it.grad) continue;
    const int es = it.bf16_io ? 2 : 4;
    ClipSpan sp = clip_span(it);
    // vectors need both sides on 16-byte boundaries at the same element
    if ((((uintptr_t)it.grad ^ (uintptr_t)it.out) & 15) != 0) sp.lead = sp.vecs = sp.tail = 0;
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const unsigned char*>(it.grad) + (it.at + sp.lead) * es);
    uint4* o = reinterpret_cast<uint4*>(static_cast<unsigned char*>(it.out) + (it.at + sp.lead) * es);
    if (it.bf16_io) chunk_scale<true>(p, o, (int)sp.vecs, scale);
    else chunk_scale<false>(p, o, (int)sp.vecs, scale);
    if (threadIdx.x < sp.lead && in_range(threadIdx.x, it.n))
      store_any(it.out, it.at + threadIdx.x, it.bf16_io, load_any(it.grad, it.at + threadIdx.x, it.bf16_io) * scale);
    for (int64_t e = sp.tail + threadIdx.x; e < it.n; e += kClipThreads)
      store_any(it.out, it.at + e, it.bf16_io, load_any(it.grad, it.at + e, it.bf16_io) * scale);
  }
}

int clip_grid(int sm_count) { return 8 * sm_count; }

}  // namespace

size_t clip_workspace(int64_t count, int sm_count) {
  return (size_t)std::max<int64_t>(1, div_up(count, kClipTensors)) * (size_t)clip_grid(sm_count) * sizeof(double);
}

namespace {

template <int CAP>
cudaError_t clip_with_tables(const ClipArgs& a, int sm_count, cudaStream_t s) {
  const int grid = clip_grid(sm_count);
  // the next table of up to CAP tensors (empty ones left out); a
  // device's memory holds far fewer than 2^32 chunks
  const auto fill = [&](int64_t k, ClipTable<CAP>& t) {
    t.count = 0;
    int64_t chunks = 0;
    for (; k < a.count && t.count < CAP; ++k) {
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
  ClipTable<CAP> t;
  int64_t partials = 0;
  for (int64_t k = 0; k < a.count;) {
    k = fill(k, t);
    if (t.count == 0) continue;
    const int64_t g = std::min<int64_t>(grid, t.first[t.count]);
    const cudaError_t e = launch_pdl(clip_squares_kernel<CAP>, g, kClipThreads, 0, s, t, a.ws + partials);
    if (e != cudaSuccess) return e;
    partials += g;
  }
  cudaError_t e = cudaSuccess;
  if (a.outs == nullptr || partials == 0)
    return launch_pdl(clip_norm_kernel, 1, kClipThreads, 0, s, (const double*)a.ws, partials, a.norm);
  for (int64_t k = 0; k < a.count;) {
    k = fill(k, t);
    if (t.count == 0) continue;
    const int64_t g = std::min<int64_t>(grid, t.first[t.count]);
    e = launch_pdl(clip_scale_kernel<CAP>, g, kClipThreads, 0, s, t, (const double*)a.ws, partials, a.norm, a.max_norm, a.eps);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace

cudaError_t run_clip_grads(const ClipArgs& a, int sm_count, cudaStream_t s) {
  return a.count <= kClipFewTensors ? clip_with_tables<kClipFewTensors>(a, sm_count, s)
                                    : clip_with_tables<kClipTensors>(a, sm_count, s);
}

cudaError_t status_clip(unsigned int* word, bool clear) { return unit_status(word, clear); }

}  // namespace rlca
