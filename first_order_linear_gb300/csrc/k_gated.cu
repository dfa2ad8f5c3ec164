// Gated linear recurrence and its gradient.
//
//   a_t = sigma(gate_t),  h_t = k_t a_t h_{t-1} + (1 - a_t) x_t
//   G_t = dh_t + k_{t+1} a_{t+1} G_{t+1},  dx = (1 - a) G,  dgate = a (1 - a) G (k h_{t-1} - x)
//
// with k_t = 0 where step t-1 is flagged.  The state and all arithmetic are
// float32.
#include <algorithm>
#include <initializer_list>

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
// sign, sigma as its difference to 1, seven instructions.  What that leaves of a
// gate below 1e-4 is 6e-8 of the state it lets through, and the short
// exponential's error, 2^-22 of the value at |g| = 4, is far below the gate's own
// rounding.  (The exponent is bounded so that the product stays a number: a gate
// below -87 lets 2^-126 through.)
template <>
struct Sigma<bf16> {
  __device__ __forceinline__ static Gate of(float g) {
    float t = g * -1.44269504f, r;
    asm("min.NaN.f32 %0, %0, %1;" : "+f"(t) : "f"(126.f));
    asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(t));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + t));
    const float na = t * r;
    return {1.f - na, na};
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

// ---------------------------------------------------------------------------
// Tiles: a CTA walks the steps of 64 channels of a row in tiles of a few steps
// a warp, a lane two channels, whose arithmetic is paired.  A thread scans its
// steps from 0 and keeps, for each, the value and the product of gates that
// the state before them still meets; the warps' maps (product, value) meet in
// shared memory, and one multiply-add a step brings the state in.  Behind a
// flagged step nothing of the state before it arrives, whatever it holds: flags
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
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(g) : "r"(raw), "r"(0xc2aec2aeu));  // -87
    const float2 u = apart(mul2(Two{g}.wide(), v2(-1.44269504f, -1.44269504f)));
    float2 t, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(t.x) : "f"(u.x));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(t.y) : "f"(u.y));
    const V2 tt = v2(t.x, t.y), one = v2(1.f, 1.f);
    const float2 d = apart(add2(tt, one));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(d.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(d.y));
    *na = mul2(tt, v2(r.x, r.y));
    *a = fma2(*na, v2(-1.f, -1.f), one);
  }
};

// two channels' maps of a run of steps: h -> q + p h, a severed one marked by
// p = -0 in both (products of gates are not negative)
struct Map2 {
  V2 p, q;
};
__device__ __forceinline__ Map2 identity() { return {v2(1.f, 1.f), 0}; }
__device__ __forceinline__ bool severed(const Map2& m) { return (uint32_t)m.p == 0x80000000u; }
__device__ __forceinline__ V2 pass(const Map2& m, V2 h) { return severed(m) ? m.q : fma2(m.p, h, m.q); }
// `then` behind `first`
__device__ __forceinline__ Map2 chain(const Map2& then, const Map2& first) {
  if (severed(then)) return then;
  return {severed(first) ? first.p : mul2(then.p, first.p), fma2(then.p, first.q, then.q)};
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
// Other rows are copied in 16-byte vectors from the boundary in front of
// them -- a vector that holds any byte of the row is readable as a whole --, and
// a lane's channels are 32 apart.
template <class ST, bool kBulk, int L>
struct TileRows {
  static constexpr int kBytes = Stor<ST>::kBytes, kPitch = kCols * kBytes + (kBulk ? 0 : 16), kTile = L * kPitch;
  static constexpr int kVectors = kCols * kBytes / 16 + 1;
};

// this thread's vectors of the steps t0 .. t0 + L - 1 in front of `len` of one array
template <class ST, int L, int THREADS>
__device__ __forceinline__ void copy_rows(unsigned char* tile, const float* p, const GatedArgs& a, int64_t stride, int64_t e,
                                          int64_t t0, int64_t len, int64_t c0) {
  using R = TileRows<ST, false, L>;
  const uint32_t width = (uint32_t)min((int64_t)kCols, a.D - c0) * R::kBytes;
  for (int i = threadIdx.x; i < L * R::kVectors; i += THREADS) {
    const int r = i / R::kVectors, v = i % R::kVectors;
    if (t0 + r < 0 || t0 + r >= len) continue;
    const int64_t row = ((e * a.step_e + (t0 + r) * a.step_t) * stride + c0) * R::kBytes;
    const uintptr_t at = (uintptr_t)p + row;
    const uint32_t shift = at & 15;
    if (16 * (uint32_t)v >= shift + width) continue;
    if (!in_range((row + max(16 * v - (int)shift, 0)) / R::kBytes, a.E * a.T * stride) ||
        !span_in_range(r * R::kPitch + 16 * v, 16, R::kTile))
      continue;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(tile + r * R::kPitch + 16 * v)),
                 "l"(at - shift + 16 * v)
                 : "memory");
  }
}
// an arrival on `bar` when this thread's copies so far have landed
__device__ __forceinline__ void copies_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// A lane's two channels of consecutive steps of a tile.
template <class ST, bool kBulk, int L>
struct Reader {
  using R = TileRows<ST, kBulk, L>;
  const unsigned char* at;
  uint32_t shift = 0, move = 0;
  // from step r of the tile on; the array's address of that row's first column, and its bytes from step to step
  __device__ Reader(const unsigned char* tile, int r, int lane, uint32_t address, uint32_t step)
      : at(tile + r * R::kPitch + lane * (kBulk ? 2 : 1) * R::kBytes), shift(address & 15), move(step & 15) {}
  __device__ __forceinline__ Two<ST> get(int i) const {
    if constexpr (kBulk) return Two<ST>::pair(at + i * R::kPitch);
    else return Two<ST>::split(at + i * R::kPitch + ((shift + i * move) & 15));
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

// Writes consecutive steps of a matrix: the address moves by one row a step.
template <class ST, bool kPairs>
struct Writer {
  unsigned char* at;
  int64_t step, first, last;  // bytes a step; the matrix, for the index check
  bool on[2];
  __device__ Writer(const Cols<ST, kPairs>& cols, const GatedArgs& a, float* p, int64_t stride, int64_t row) {
    at = reinterpret_cast<unsigned char*>(p) + (row * stride + cols.ch(0)) * Stor<ST>::kBytes;
    step = a.step_t * stride * Stor<ST>::kBytes;
    first = (int64_t)p, last = (int64_t)p + a.E * a.T * stride * Stor<ST>::kBytes;
    on[0] = cols.on(0), on[1] = cols.on(1);
  }
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
__device__ __forceinline__ bool cut_before(const GatedArgs& a, int64_t e, int64_t t, int len) {
  return t > 0 && t < len && flagged(a, e * a.step_e + (t - 1) * a.step_t);
}

// What the CTAs of a row have in shared memory beside the ring, and how their
// maps meet.
template <int W, int STAGES>
struct GatedShared {
  Map2 warp_map[2][W][32];
  Map2 cta_map[2][kMaxShare][32];
  uint64_t full[STAGES], maps[2];
};

// The carry in front of this warp's steps (returned) and behind the round's
// (*carry).  Buffers alternate: a peer sends its map of round k + 2 only when it
// has this CTA's of round k + 1, which leaves behind the reads of round k.
template <int W, int STAGES, bool kForward>
__device__ __forceinline__ V2 meet(GatedShared<W, STAGES>& sh, int round, int rank, int share, bool any_cut, bool* ok, V2* carry) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, buf = round & 1;
  V2 at = *carry;
  if (share == 1) {
    fold<W, kForward>(sh.warp_map[buf], lane, warp, any_cut, carry, &at);
    return at;
  }
  if (warp == 0) {
    if (lane == 0) mbar_arrive_expect_tx(&sh.maps[buf], (uint32_t)share * 32 * sizeof(Map2));
    Map2 all = sh.warp_map[buf][kForward ? 0 : W - 1][lane];
#pragma unroll
    for (int k = 1; k < W; ++k) all = chain(sh.warp_map[buf][kForward ? k : W - 1 - k][lane], all);
    for (int r = 0; r < share; ++r) send(&sh.cta_map[buf][rank][lane], &sh.maps[buf], r, all);
  }
  if (*ok) *ok = mbar_wait_bounded(&sh.maps[buf], (round >> 1) & 1);
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

template <class ST, int C, int W, int STAGES, bool kBulk, int kResident>
__global__ void __launch_bounds__(32 * W, kResident) gated_tile_kernel(GatedArgs a, const __grid_constant__ GatedMaps maps, int share) {
  using R = TileRows<ST, kBulk, C * W>;
  constexpr int L = C * W, kArrays = 2;
  extern __shared__ __align__(128) unsigned char ring_tiles[];  // [STAGES][x, gate]
  __shared__ __align__(16) GatedShared<W, STAGES> sh;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rank = share > 1 ? blockIdx.x % share : 0;
  const int64_t blocks = (a.D + kCols - 1) / kCols, unit = blockIdx.x / share, e = unit / blocks;
  const Cols<ST, kBulk> cols{(unit % blocks) * kCols, lane, a.D};
  pdl_trigger();
  if (threadIdx.x == 0) {
    for (int i = 0; i < STAGES; ++i) mbar_init(&sh.full[i], kBulk ? 1 : 32 * W);
    mbar_init(&sh.maps[0], 1);
    mbar_init(&sh.maps[1], 1);
    mbar_fence_init();
  }
  if (share > 1) cluster_meet();  // (a peer's memory is written only once it runs)
  else __syncthreads();
  pdl_wait();

  const int len = row_length(a, e);
  const int ntiles = (len + L - 1) / L, rounds = (ntiles + share - 1) / share;
  const int mine = ntiles > rank ? (ntiles - rank + share - 1) / share : 0;
  const auto fill = [&](int stage, int j) {
    if (!in_range(stage, STAGES)) return;
    unsigned char* to = ring_tiles + (size_t)stage * kArrays * R::kTile;
    const int t = (rank + j * share) * L;
    if constexpr (kBulk) {
      if (threadIdx.x != 0) return;
      mbar_arrive_expect_tx(&sh.full[stage], kArrays * R::kTile);
      tile_load(to, &maps.in[0], (int)cols.c0, t, (int)e, &sh.full[stage]);
      tile_load(to + R::kTile, &maps.in[1], (int)cols.c0, t, (int)e, &sh.full[stage]);
    } else {
      copy_rows<ST, L, 32 * W>(to, a.x, a, a.x_stride, e, t, len, cols.c0);
      copy_rows<ST, L, 32 * W>(to + R::kTile, a.gate, a, a.gate_stride, e, t, len, cols.c0);
      copies_arrive(&sh.full[stage]);
    }
  };
  for (int j = 0; j < STAGES - 1 && j < mine; ++j) fill(j, j);

  V2 carry = cols.state(a.state, e, a.E);
  FillRing<STAGES> ring;
  bool met = true;
  const bool flags = a.terminated != nullptr || a.truncated != nullptr;
  bool cut_next = flags && lane < C && cut_before(a, e, (int64_t)rank * L + warp * C + lane, len);
  for (int k = 0; k < rounds; ++k) {
    const int64_t t0 = ((int64_t)rank + (int64_t)k * share) * L + warp * C;  // the warp's first step
    const int real = (int)min(max(len - t0, (int64_t)0), (int64_t)C);
    const int64_t row0 = e * a.step_e + t0 * a.step_t;
    const uint32_t cut = __ballot_sync(kFullMask, cut_next);
    if (flags && lane < C) cut_next = cut_before(a, e, t0 + (int64_t)share * L + lane, len);
    V2 p[C], q[C];
    Map2 m = identity();
    if (k < mine) {
      if (ring.ok && k + STAGES - 1 < mine) fill(ring.fill_stage(), k + STAGES - 1);
      if (ring.ok) ring.ok = mbar_wait_bounded(&sh.full[ring.stage], ring.phase);
      const unsigned char* tile = ring_tiles + (size_t)ring.stage * kArrays * R::kTile;
      ring.next();
      const Reader<ST, kBulk, L> xs(tile, warp * C, lane, (uint32_t)(uintptr_t)a.x + (uint32_t)(row0 * a.x_stride + cols.c0) * R::kBytes,
                                    (uint32_t)(a.step_t * a.x_stride) * R::kBytes);
      const Reader<ST, kBulk, L> gs(tile + R::kTile, warp * C, lane,
                                    (uint32_t)(uintptr_t)a.gate + (uint32_t)(row0 * a.gate_stride + cols.c0) * R::kBytes,
                                    (uint32_t)(a.step_t * a.gate_stride) * R::kBytes);
      if (cut == 0 && real == C) {
#pragma unroll
        for (int i = 0; i < C; ++i) {
          V2 s, ns;
          gs.get(i).sigma(&s, &ns);
          m.q = q[i] = fma2(s, m.q, mul2(ns, xs.get(i).wide()));
          m.p = p[i] = mul2(m.p, s);
        }
      } else {
#pragma unroll
        for (int i = 0; i < C; ++i) {
          if (i < real) {
            V2 s, ns;
            gs.get(i).sigma(&s, &ns);
            const V2 b = mul2(ns, xs.get(i).wide());
            if ((cut >> i) & 1) m = {0x8000000080000000ull, b};
            else m = chain({s, b}, m);
          }
          q[i] = m.q;
          p[i] = m.p;
        }
      }
    }
    sh.warp_map[k & 1][warp][lane] = m;
    const bool any_cut = __syncthreads_or(cut != 0);
    const V2 h = meet<W, STAGES, true>(sh, k, rank, share, any_cut, &met, &carry);
    Writer<ST, kBulk> out(cols, a, a.h, a.D, row0);
    if (k < mine && real == C && cut == 0) {
#pragma unroll
      for (int i = 0; i < C; ++i) out.put(fma2(p[i], h, q[i]));
    } else {
#pragma unroll
      for (int i = 0; i < C; ++i)
        if (t0 + i < a.T) out.put(k < mine && i < real ? pass({p[i], q[i]}, h) : 0);
    }
  }
  // behind the row's last tile
  for (int64_t t = ((int64_t)rounds * share + rank) * L + warp * C; t < a.T; t += (int64_t)share * L) {
    Writer<ST, kBulk> out(cols, a, a.h, a.D, e * a.step_e + t * a.step_t);
    for (int i = 0; i < C && t + i < a.T; ++i) out.put(0);
  }
  if (rank == 0 && warp == 0 && a.last != nullptr) {
    if (len > 0 && flagged(a, e * a.step_e + (int64_t)(len - 1) * a.step_t)) carry = 0;
    cols.store_state(a.last, e, a.E, carry);
  }
  // (copies still on their way after a wait gave up land before the CTA ends)
  if (kBulk && !ring.ok && threadIdx.x == 0)
    for (int i = 0; i < STAGES; ++i) mbar_wait_bounded(&sh.full[i], ring.last_fill(i));
  if (!kBulk) asm volatile("cp.async.wait_all;" ::: "memory");
  if (share > 1) cluster_meet();  // no CTA ends while a peer may still write to it
}

template <class ST, int C, int W, int STAGES, bool kBulk, int kResident>
__global__ void __launch_bounds__(32 * W, kResident) gated_grad_tile_kernel(GatedArgs a, const __grid_constant__ GatedMaps maps, int share) {
  using R = TileRows<ST, kBulk, C * W>;
  constexpr int L = C * W, kArrays = 4;
  extern __shared__ __align__(128) unsigned char ring_tiles[];  // [STAGES][x, gate, dh, h one step earlier]
  __shared__ __align__(16) GatedShared<W, STAGES> sh;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rank = share > 1 ? blockIdx.x % share : 0;
  const int64_t blocks = (a.D + kCols - 1) / kCols, unit = blockIdx.x / share, e = unit / blocks;
  const Cols<ST, kBulk> cols{(unit % blocks) * kCols, lane, a.D};
  pdl_trigger();
  if (threadIdx.x == 0) {
    for (int i = 0; i < STAGES; ++i) mbar_init(&sh.full[i], kBulk ? 1 : 32 * W);
    mbar_init(&sh.maps[0], 1);
    mbar_init(&sh.maps[1], 1);
    mbar_fence_init();
  }
  if (share > 1) cluster_meet();
  else __syncthreads();
  pdl_wait();

  const int len = row_length(a, e);
  const int ntiles = (len + L - 1) / L, rounds = (ntiles + share - 1) / share;
  const int mine = ntiles > rank ? (ntiles - rank + share - 1) / share : 0;
  // the row's last tile first
  const auto fill = [&](int stage, int j) {
    if (!in_range(stage, STAGES)) return;
    unsigned char* to = ring_tiles + (size_t)stage * kArrays * R::kTile;
    const int t = (rank + (mine - 1 - j) * share) * L;
    if constexpr (kBulk) {
      if (threadIdx.x != 0) return;
      mbar_arrive_expect_tx(&sh.full[stage], kArrays * R::kTile);
#pragma unroll
      for (int i = 0; i < kArrays; ++i)
        tile_load(to + i * R::kTile, &maps.in[i], (int)cols.c0, i == 3 ? t - 1 : t, (int)e, &sh.full[stage]);
    } else {
      copy_rows<ST, L, 32 * W>(to, a.x, a, a.x_stride, e, t, len, cols.c0);
      copy_rows<ST, L, 32 * W>(to + R::kTile, a.gate, a, a.gate_stride, e, t, len, cols.c0);
      copy_rows<ST, L, 32 * W>(to + 2 * R::kTile, a.dh, a, a.dh_stride, e, t, len, cols.c0);
      copy_rows<ST, L, 32 * W>(to + 3 * R::kTile, a.in_h, a, a.h_stride, e, t - 1, len, cols.c0);
      copies_arrive(&sh.full[stage]);
    }
  };
  for (int j = 0; j < STAGES - 1 && j < mine; ++j) fill(j, j);

  V2 carry = cols.state(a.d_last, e, a.E);
  if (len > 0 && flagged(a, e * a.step_e + (int64_t)(len - 1) * a.step_t)) carry = 0;
  FillRing<STAGES> ring;
  bool met = true;
  int j = 0;
  const bool flags = a.terminated != nullptr || a.truncated != nullptr;
  bool cut_next = flags && lane < C && cut_before(a, e, ((int64_t)rank + (int64_t)(rounds - 1) * share) * L + warp * C + lane, len);
  for (int k = rounds - 1; k >= 0; --k) {
    const int64_t t0 = ((int64_t)rank + (int64_t)k * share) * L + warp * C;
    const int real = (int)min(max(len - t0, (int64_t)0), (int64_t)C);
    const int64_t row0 = e * a.step_e + t0 * a.step_t;
    const uint32_t cut = __ballot_sync(kFullMask, cut_next);
    if (flags && lane < C) cut_next = cut_before(a, e, t0 - (int64_t)share * L + lane, len);
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
      const auto reader = [&](int i, const float* base, int64_t row, int64_t stride) {
        return Reader<ST, kBulk, L>(tile + i * R::kTile, warp * C, lane,
                                    (uint32_t)(uintptr_t)base + (uint32_t)(row * stride + cols.c0) * R::kBytes,
                                    (uint32_t)(a.step_t * stride) * R::kBytes);
      };
      const auto xs = reader(0, a.x, row0, a.x_stride), gs = reader(1, a.gate, row0, a.gate_stride),
                 ds = reader(2, a.dh, row0, a.dh_stride), hs = reader(3, a.in_h, row0 - a.step_t, a.h_stride);
      if (cut == 0 && real == C && t0 > 0) {
#pragma unroll
        for (int i = C - 1; i >= 0; --i) {
          V2 s;
          gs.get(i).sigma(&s, &na[i]);
          p[i] = m.p;
          g[i] = add2(ds.get(i).wide(), m.q);
          w[i] = mul2(mul2(s, na[i]), fma2(xs.get(i).wide(), minus, hs.get(i).wide()));
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
            gs.get(i).sigma(&s, &na[i]);
            const bool here = (cut >> i) & 1;
            const V2 before = here ? 0 : t0 + i == 0 ? first : hs.get(i).wide();
            g[i] = add2(ds.get(i).wide(), m.q);
            w[i] = mul2(mul2(s, na[i]), fma2(xs.get(i).wide(), minus, before));
            if (here) m = {0x8000000080000000ull, 0};
            else m = {severed(m) ? m.p : mul2(m.p, s), mul2(s, g[i])};
          }
        }
      }
    }
    sh.warp_map[(rounds - 1 - k) & 1][warp][lane] = m;
    const bool any_cut = __syncthreads_or(cut != 0);
    const V2 u = meet<W, STAGES, false>(sh, rounds - 1 - k, rank, share, any_cut, &met, &carry);
    Writer<ST, kBulk> to_x(cols, a, a.dx, a.dx_stride, row0), to_gate(cols, a, a.dgate, a.dgate_stride, row0);
    if (k < mine && real == C && cut == 0) {
#pragma unroll
      for (int i = 0; i < C; ++i) {
        const V2 G = fma2(p[i], u, g[i]);
        to_x.put(mul2(na[i], G));
        to_gate.put(mul2(w[i], G));
      }
    } else {
#pragma unroll
      for (int i = 0; i < C; ++i) {
        if (t0 + i >= a.T) continue;
        const bool on = k < mine && i < real;
        const V2 G = on ? pass({p[i], g[i]}, u) : 0;
        to_x.put(on ? mul2(na[i], G) : 0);
        to_gate.put(on ? mul2(w[i], G) : 0);
      }
    }
  }
  for (int64_t t = ((int64_t)rounds * share + rank) * L + warp * C; t < a.T; t += (int64_t)share * L) {
    const int64_t row = e * a.step_e + t * a.step_t;
    Writer<ST, kBulk> to_x(cols, a, a.dx, a.dx_stride, row), to_gate(cols, a, a.dgate, a.dgate_stride, row);
    for (int i = 0; i < C && t + i < a.T; ++i) to_x.put(0), to_gate.put(0);
  }
  if (rank == 0 && warp == 0 && a.d_state != nullptr) cols.store_state(a.d_state, e, a.E, carry);
  if (kBulk && !ring.ok && threadIdx.x == 0)
    for (int i = 0; i < STAGES; ++i) mbar_wait_bounded(&sh.full[i], ring.last_fill(i));
  if (!kBulk) asm volatile("cp.async.wait_all;" ::: "memory");
  if (share > 1) cluster_meet();
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

// rows of every matrix on 16-byte boundaries: tensor copies can take them
bool rows_aligned(std::initializer_list<const void*> bases, std::initializer_list<int64_t> strides, int es, int to) {
  for (const void* p : bases)
    if (((uintptr_t)p % to) != 0) return false;
  for (int64_t r : strides)
    if ((r * es) % to != 0) return false;
  return true;
}

// CTAs of a row: enough to give every SM two, as far as the row has tiles for them
int row_share(int64_t units, int64_t ntiles, int sm) {
  int share = 1;
  while (share < kMaxShare && units * share < 2 * (int64_t)sm && ntiles >= 2 * share) share *= 2;
  return share;
}

template <class ST>
cudaError_t scan_typed(const GatedArgs& a, int sm, cudaStream_t s) {
#ifndef FC
#define FC 16
#define FW 4
#define FR 4
#define FS 2
#endif
  constexpr int kChunk = Stor<ST>::kBytes == 2 ? FC : 8, W = Stor<ST>::kBytes == 2 ? FW : 4, L = kChunk * W, kStages = FS, es = Stor<ST>::kBytes;
  constexpr int kRes = FR;
  const int64_t units = a.E * div_up(a.D, kCols);
  if (a.T <= 4) return launch_serial(gated_serial_kernel<ST>, a, sm, s);
  const int share = row_share(units, div_up(a.T, L), sm);
  if (units * share > INT32_MAX) return launch_serial(gated_serial_kernel<ST>, a, sm, s);
  GatedMaps maps = {};
  if (rows_aligned({a.x, a.gate}, {a.x_stride, a.gate_stride}, es, 16) && rows_aligned({a.h}, {a.D}, es, 2 * es) &&
      encode_steps_map(&maps.in[0], a.x, es, a.D, a.T, a.E, a.x_stride * a.step_t, a.x_stride * a.step_e, kCols, L) &&
      encode_steps_map(&maps.in[1], a.gate, es, a.D, a.T, a.E, a.gate_stride * a.step_t, a.gate_stride * a.step_e, kCols, L)) {
    const auto kernel = gated_tile_kernel<ST, kChunk, W, kStages, true, kRes>;
    const size_t smem = (size_t)kStages * 2 * TileRows<ST, true, L>::kTile;
    static std::atomic<uint64_t> allowed;
    const cudaError_t e = allow_smem(kernel, smem, allowed);
    return e != cudaSuccess ? e : launch_tiles(kernel, units * share, 32 * W, smem, share, s, a, maps);
  }
  const auto kernel = gated_tile_kernel<ST, kChunk, W, kStages, false, kRes>;
  const size_t smem = (size_t)kStages * 2 * TileRows<ST, false, L>::kTile;
  static std::atomic<uint64_t> allowed;
  const cudaError_t e = allow_smem(kernel, smem, allowed);
  return e != cudaSuccess ? e : launch_tiles(kernel, units * share, 32 * W, smem, share, s, a, maps);
}

template <class ST>
cudaError_t grad_typed(const GatedArgs& a, int sm, cudaStream_t s) {
#ifndef HC
#define HC 8
#define HW 8
#define HR 2
#define HS 3
#endif
  constexpr int kChunk = Stor<ST>::kBytes == 2 ? HC : 8, W = Stor<ST>::kBytes == 2 ? HW : 4, L = kChunk * W, kStages = HS, es = Stor<ST>::kBytes;
  constexpr int kRes = HR;
  const int64_t units = a.E * div_up(a.D, kCols);
  if (a.T <= 4) return launch_serial(gated_grad_serial_kernel<ST>, a, sm, s);
  const int share = row_share(units, div_up(a.T, L), sm);
  if (units * share > INT32_MAX) return launch_serial(gated_grad_serial_kernel<ST>, a, sm, s);
  GatedMaps maps = {};
  const float* in[4] = {a.x, a.gate, a.dh, a.in_h};
  const int64_t stride[4] = {a.x_stride, a.gate_stride, a.dh_stride, a.h_stride};
  bool bulk = rows_aligned({a.x, a.gate, a.dh, a.in_h}, {a.x_stride, a.gate_stride, a.dh_stride, a.h_stride}, es, 16) &&
              rows_aligned({a.dx, a.dgate}, {a.D, a.dx_stride, a.dgate_stride}, es, 2 * es);
  for (int i = 0; bulk && i < 4; ++i)
    bulk = encode_steps_map(&maps.in[i], in[i], es, a.D, a.T, a.E, stride[i] * a.step_t, stride[i] * a.step_e, kCols, L);
  if (bulk) {
    const auto kernel = gated_grad_tile_kernel<ST, kChunk, W, kStages, true, kRes>;
    const size_t smem = (size_t)kStages * 4 * TileRows<ST, true, L>::kTile;
    static std::atomic<uint64_t> allowed;
    const cudaError_t e = allow_smem(kernel, smem, allowed);
    return e != cudaSuccess ? e : launch_tiles(kernel, units * share, 32 * W, smem, share, s, a, maps);
  }
  const auto kernel = gated_grad_tile_kernel<ST, kChunk, W, kStages, false, kRes>;
  const size_t smem = (size_t)kStages * 4 * TileRows<ST, false, L>::kTile;
  static std::atomic<uint64_t> allowed;
  const cudaError_t e = allow_smem(kernel, smem, allowed);
  return e != cudaSuccess ? e : launch_tiles(kernel, units * share, 32 * W, smem, share, s, a, maps);
}

}  // namespace

cudaError_t run_gated_scan(const GatedArgs& a, int sm, cudaStream_t s) {
  return a.bf16_io ? scan_typed<bf16>(a, sm, s) : scan_typed<float>(a, sm, s);
}

cudaError_t run_gated_scan_backward(const GatedArgs& a, int sm, cudaStream_t s) {
  return a.bf16_io ? grad_typed<bf16>(a, sm, s) : grad_typed<float>(a, sm, s);
}

cudaError_t status_gated(unsigned int* word, bool clear) { return unit_status(word, clear); }

}  // namespace rlca
