// host_checks.h -- argument checks and device queries shared by the C entry
// points.
#pragma once

#include <atomic>
#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>
#include <initializer_list>

namespace rlca {

inline std::atomic<int> g_sm_count[256];

inline cudaError_t sm_count_of_current_device(int* out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 0 && dev < 256) {
    int c = g_sm_count[dev].load(std::memory_order_relaxed);
    if (c > 0) {
      *out = c;
      return cudaSuccess;
    }
  }
  int c = 0;
  e = cudaDeviceGetAttribute(&c, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  if (dev >= 0 && dev < 256) g_sm_count[dev].store(c, std::memory_order_relaxed);
  *out = c;
  return cudaSuccess;
}

struct Span {
  const void* p;
  size_t bytes;
};

inline bool overlap(const Span& a, const Span& b) {
  if (a.p == nullptr || b.p == nullptr || a.bytes == 0 || b.bytes == 0) return false;
  const uintptr_t a0 = (uintptr_t)a.p, b0 = (uintptr_t)b.p;
  return a0 < b0 + b.bytes && b0 < a0 + a.bytes;
}

// every output against every input and every other output
inline bool any_overlap(std::initializer_list<Span> ins, std::initializer_list<Span> outs) {
  for (const Span& o : outs) {
    for (const Span& i : ins)
      if (overlap(o, i)) return true;
    for (const Span& o2 : outs)
      if (&o2 != &o && overlap(o, o2)) return true;
  }
  return false;
}

inline bool aligned(const void* p, uintptr_t a) { return p == nullptr || ((uintptr_t)p % a) == 0; }

inline bool flags_ok(uint32_t flags, uint32_t allowed) { return (flags & ~allowed) == 0u; }

// a workspace of `have` bytes where `need` are asked for
inline bool workspace_ok(const void* ws, size_t have, size_t need) {
  return need == 0 || (ws != nullptr && have >= need && aligned(ws, 16));
}

}  // namespace rlca
