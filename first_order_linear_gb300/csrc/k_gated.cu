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
// 6000 steps came out 2e-5 off.)  bfloat16 gates take the short exponential: its
// error, 2^-22 of the value at |g| = 4, is far below the gate's own rounding.
struct Gate {
  float a, na;
};
template <class ST>
__device__ __forceinline__ Gate gate_of(float g) {
  const float e = Stor<ST>::kBytes == 4 ? expf(-fabsf(g)) : __expf(-fabsf(g)), less = e * __fdividef(1.f, 1.f + e), more = 1.f - less;
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
      const Gate g = gate_of<ST>(load1<ST>(a.gate, row * a.gate_stride + c, n * a.gate_stride));
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
      const Gate g = gate_of<ST>(load1<ST>(a.gate, row * a.gate_stride + c, n * a.gate_stride));
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
// Tiles: a CTA walks the steps of 64 channels of a row in tiles of 8 steps a
// warp, a lane two channels.  A thread scans its 8 steps from 0 and keeps,
// for each, the value and the product of gates that the state before them
// still meets; the warps' maps (product, value) meet in shared memory, and one
// multiply-add a step brings the state in.  Behind a flagged step nothing of
// the state before it arrives, whatever it holds: flags are the same for all
// channels, so that is a matter of branches and not of products with 0.
//
// Where the rows alone leave SMs idle, a cluster of CTAs shares a row: its
// CTAs take the tiles of a round side by side, leave their maps in each
// other's shared memory and meet once a round.
// ---------------------------------------------------------------------------
constexpr int kChunk = 8, kCols = 64, kMaxShare = 8;

// two channels' maps of a run of steps: h -> q + p h, a severed one marked by
// p = -0 (products of gates are never negative)
using Map2 = float4;  // p0, q0, p1, q1
__device__ __forceinline__ bool severed(float p) { return __float_as_uint(p) == 0x80000000u; }
__device__ __forceinline__ float through(float p, float q, float h) { return severed(p) ? q : fmaf(p, h, q); }
__device__ __forceinline__ void pass(const Map2& m, float* h) {
  h[0] = through(m.x, m.y, h[0]);
  h[1] = through(m.z, m.w, h[1]);
}
// `then` behind `first`
__device__ __forceinline__ Map2 chain(const Map2& then, const Map2& first) {
  Map2 r;
  r.x = severed(then.x) ? then.x : then.x * first.x;
  r.y = through(then.x, then.y, first.y);
  r.z = severed(then.z) ? then.z : then.z * first.z;
  r.w = through(then.z, then.w, first.w);
  return r;
}

__device__ __forceinline__ void store_peer(void* mine, int rank, const Map2& m) {
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(mine)), "r"(rank));
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(at), "f"(m.x), "f"(m.y), "f"(m.z), "f"(m.w)
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

// a lane's two channels of a step
template <class ST>
__device__ __forceinline__ void open2(const unsigned char* at, float* v);
template <>
__device__ __forceinline__ void open2<float>(const unsigned char* at, float* v) {
  const float2 f = *reinterpret_cast<const float2*>(at);
  v[0] = f.x, v[1] = f.y;
}
template <>
__device__ __forceinline__ void open2<bf16>(const unsigned char* at, float* v) {
  const uint32_t w = *reinterpret_cast<const uint32_t*>(at);
  v[0] = __uint_as_float(w << 16), v[1] = __uint_as_float(w & 0xffff0000u);
}

// What a CTA works on, and where a lane's channels lie: next to each other
// (kPairs, rows on 2-element boundaries), or 32 apart.
template <class ST, bool kPairs>
struct Cols {
  int64_t c0;
  int lane;
  int64_t D;
  __device__ int64_t ch(int k) const { return kPairs ? c0 + 2 * lane + k : c0 + lane + 32 * k; }
  __device__ bool on(int k) const { return ch(k) < D; }
  __device__ void load(const float* p, int64_t row, int64_t n, float* v) const {
#pragma unroll
    for (int k = 0; k < 2; ++k) v[k] = on(k) ? load1<ST>(p, row + ch(k), n) : 0.f;
  }
  __device__ void store(float* p, int64_t row, int64_t n, const float* v) const {
    if constexpr (kPairs) {
      if (on(0) && span_in_range(row + ch(0), 2, n)) {
        if constexpr (Stor<ST>::kBytes == 4)
          *reinterpret_cast<float2*>(p + row + ch(0)) = make_float2(v[0], v[1]);
        else
          *reinterpret_cast<uint32_t*>(reinterpret_cast<uint16_t*>(p) + row + ch(0)) = Stor<bf16>::pack2(v[0], v[1]);
      }
    } else {
#pragma unroll
      for (int k = 0; k < 2; ++k)
        if (on(k)) store1<ST>(p, row + ch(k), n, v[k]);
    }
  }
};

// the two channels' states in float32 [E, D]
template <class C>
__device__ __forceinline__ void load_state(const C& cols, const float* p, int64_t e, int64_t E, float* v) {
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int64_t i = e * cols.D + cols.ch(k);
    v[k] = p != nullptr && cols.on(k) && in_range(i, E * cols.D) ? p[i] : 0.f;
  }
}
template <class C>
__device__ __forceinline__ void store_state(const C& cols, float* p, int64_t e, int64_t E, const float* v) {
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int64_t i = e * cols.D + cols.ch(k);
    if (p != nullptr && cols.on(k) && in_range(i, E * cols.D)) p[i] = v[k];
  }
}

// bit i: the state before step t0 + i counts as 0 (steps in front of `len` only; lane i looks)
__device__ __forceinline__ bool cut_before(const GatedArgs& a, int64_t e, int64_t t, int len) {
  return t > 0 && t < len && flagged(a, e * a.step_e + (t - 1) * a.step_t);
}

// shared memory of a tile kernel beside its ring
template <int W>
struct GatedShared {
  Map2 warp_map[2][W][32];
  Map2 cta_map[2][kMaxShare][32];
  uint64_t full[4];
};

template <class ST, int W, int STAGES, bool kBulk>
__global__ void __launch_bounds__(32 * W, kBulk ? 3 : 2) gated_tile_kernel(GatedArgs a, const __grid_constant__ GatedMaps maps, int share) {
  constexpr int L = kChunk * W, kTile = L * kCols * Stor<ST>::kBytes;
  extern __shared__ __align__(128) unsigned char ring_tiles[];  // [STAGES][x, gate][L][64]
  __shared__ GatedShared<W> sh;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rank = share > 1 ? blockIdx.x % share : 0;
  const int64_t blocks = (a.D + kCols - 1) / kCols, unit = blockIdx.x / share, e = unit / blocks;
  const Cols<ST, kBulk> cols{(unit % blocks) * kCols, lane, a.D};
  const int64_t n = a.E * a.T;
  pdl_trigger();
  if (kBulk && threadIdx.x == 0) {
    for (int i = 0; i < STAGES; ++i) mbar_init(&sh.full[i], 1);
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
    unsigned char* to = ring_tiles + (size_t)stage * 2 * kTile;
    const int t = (rank + j * share) * L;
    mbar_arrive_expect_tx(&sh.full[stage], 2 * kTile);
    tile_load(to, &maps.in[0], (int)cols.c0, t, (int)e, &sh.full[stage]);
    tile_load(to + kTile, &maps.in[1], (int)cols.c0, t, (int)e, &sh.full[stage]);
  };
  if (kBulk && threadIdx.x == 0)
    for (int j = 0; j < STAGES - 1 && j < mine; ++j) fill(j, j);

  float carry[2];
  load_state(cols, a.state, e, a.E, carry);
  FillRing<STAGES> ring;
  const bool flags = a.terminated != nullptr || a.truncated != nullptr;
  bool cut_next = flags && lane < kChunk && cut_before(a, e, (int64_t)rank * L + warp * kChunk + lane, len);
  for (int k = 0; k < rounds; ++k) {
    const int buf = k & 1;
    const int64_t t0 = ((int64_t)rank + (int64_t)k * share) * L + warp * kChunk;  // the warp's first step
    const int real = min(max(len - t0, (int64_t)0), (int64_t)kChunk);
    const uint32_t cut = __ballot_sync(kFullMask, cut_next);
    if (flags && lane < kChunk) cut_next = cut_before(a, e, t0 + (int64_t)share * L + lane, len);
    float p[kChunk][2], q[kChunk][2];
    Map2 m = make_float4(1.f, 0.f, 1.f, 0.f);
    if (k < mine) {
      const unsigned char* at = nullptr;
      if constexpr (kBulk) {
        if (threadIdx.x == 0 && ring.ok && k + STAGES - 1 < mine) fill(ring.fill_stage(), k + STAGES - 1);
        if (ring.ok) ring.ok = mbar_wait_bounded(&sh.full[ring.stage], ring.phase);
        at = ring_tiles + (size_t)ring.stage * 2 * kTile + ((size_t)warp * kChunk * kCols + 2 * lane) * Stor<ST>::kBytes;
        ring.next();
      }
      float x[kChunk][2], g[kChunk][2];
#pragma unroll
      for (int i = 0; i < kChunk; ++i) {
        if constexpr (kBulk) {
          open2<ST>(at + (size_t)i * kCols * Stor<ST>::kBytes, x[i]);
          open2<ST>(at + kTile + (size_t)i * kCols * Stor<ST>::kBytes, g[i]);
        } else {
          x[i][0] = x[i][1] = g[i][0] = g[i][1] = 0.f;
          if (i < real) {
            const int64_t row = e * a.step_e + (t0 + i) * a.step_t;
            cols.load(a.x, row * a.x_stride, n * a.x_stride, x[i]);
            cols.load(a.gate, row * a.gate_stride, n * a.gate_stride, g[i]);
          }
        }
      }
      float P[2] = {1.f, 1.f}, Q[2] = {0.f, 0.f};
      if (cut == 0 && real == kChunk) {
#pragma unroll
        for (int i = 0; i < kChunk; ++i)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const Gate s = gate_of<ST>(g[i][c]);
            q[i][c] = Q[c] = fmaf(s.a, Q[c], s.na * x[i][c]);
            p[i][c] = P[c] = P[c] * s.a;
          }
      } else {
#pragma unroll
        for (int i = 0; i < kChunk; ++i)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const Gate s = gate_of<ST>(g[i][c]);
            const bool here = (cut >> i) & 1;
            if (i < real) {
              Q[c] = here ? s.na * x[i][c] : fmaf(s.a, Q[c], s.na * x[i][c]);
              P[c] = here ? 0.f : P[c] * s.a;
            }
            q[i][c] = Q[c];
            p[i][c] = P[c];
          }
        if (cut != 0) P[0] = P[1] = -0.f;
      }
      m = make_float4(P[0], Q[0], P[1], Q[1]);
    }
    sh.warp_map[buf][warp][lane] = m;
    __syncthreads();
    float h[2] = {carry[0], carry[1]};
    if (share > 1) {
      if (warp == 0) {
        Map2 all = sh.warp_map[buf][0][lane];
#pragma unroll
        for (int w = 1; w < W; ++w) all = chain(sh.warp_map[buf][w][lane], all);
        for (int r = 0; r < share; ++r) store_peer(&sh.cta_map[buf][rank][lane], r, all);
      }
      cluster_meet();
      for (int r = 0; r < share; ++r) {
        pass(sh.cta_map[buf][r][lane], carry);
        if (r + 1 == rank) h[0] = carry[0], h[1] = carry[1];
      }
      for (int w = 0; w < warp; ++w) pass(sh.warp_map[buf][w][lane], h);
    } else {
#pragma unroll
      for (int w = 0; w < W; ++w) {
        if (w == warp) h[0] = carry[0], h[1] = carry[1];
        pass(sh.warp_map[buf][w][lane], carry);
      }
    }
    const int reached = cut != 0 ? __ffs(cut) - 1 : kChunk;  // steps that the state reaches
    const int64_t row0 = e * a.step_e + t0 * a.step_t;
    if (k < mine && real == kChunk && cut == 0) {
#pragma unroll
      for (int i = 0; i < kChunk; ++i) {
        const float v[2] = {fmaf(p[i][0], h[0], q[i][0]), fmaf(p[i][1], h[1], q[i][1])};
        cols.store(a.h, (row0 + i * a.step_t) * a.D, n * a.D, v);
      }
    } else {
#pragma unroll
      for (int i = 0; i < kChunk; ++i) {
        if (t0 + i >= a.T) continue;
        float v[2] = {0.f, 0.f};
        if (k < mine && i < real) {
#pragma unroll
          for (int c = 0; c < 2; ++c) v[c] = i < reached ? fmaf(p[i][c], h[c], q[i][c]) : q[i][c];
        }
        cols.store(a.h, (row0 + i * a.step_t) * a.D, n * a.D, v);
      }
    }
  }
  // behind the row's last tile
  const float zero[2] = {0.f, 0.f};
  for (int64_t t = ((int64_t)rounds * share + rank) * L; t < a.T; t += (int64_t)share * L)
    for (int i = 0; i < kChunk && t + warp * kChunk + i < a.T; ++i)
      cols.store(a.h, (e * a.step_e + (t + warp * kChunk + i) * a.step_t) * a.D, n * a.D, zero);
  if (rank == 0 && warp == 0 && a.last != nullptr) {
    if (len > 0 && flagged(a, e * a.step_e + (int64_t)(len - 1) * a.step_t)) carry[0] = carry[1] = 0.f;
    store_state(cols, a.last, e, a.E, carry);
  }
  if constexpr (kBulk) {
    // (copies still on their way after a wait gave up land before the CTA ends)
    if (!ring.ok && threadIdx.x == 0)
      for (int i = 0; i < STAGES; ++i) mbar_wait_bounded(&sh.full[i], ring.last_fill(i));
  }
  if (share > 1) cluster_meet();  // no CTA ends while a peer may still write to it
}

template <class ST, int W, int STAGES, bool kBulk>
__global__ void __launch_bounds__(32 * W, 2) gated_grad_tile_kernel(GatedArgs a, const __grid_constant__ GatedMaps maps, int share) {
  constexpr int L = kChunk * W, kTile = L * kCols * Stor<ST>::kBytes;
  extern __shared__ __align__(128) unsigned char ring_tiles[];  // [STAGES][x, gate, dh, h one step earlier][L][64]
  __shared__ GatedShared<W> sh;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rank = share > 1 ? blockIdx.x % share : 0;
  const int64_t blocks = (a.D + kCols - 1) / kCols, unit = blockIdx.x / share, e = unit / blocks;
  const Cols<ST, kBulk> cols{(unit % blocks) * kCols, lane, a.D};
  const int64_t n = a.E * a.T;
  pdl_trigger();
  if (kBulk && threadIdx.x == 0) {
    for (int i = 0; i < STAGES; ++i) mbar_init(&sh.full[i], 1);
    mbar_fence_init();
  }
  if (share > 1) cluster_meet();  // (a peer's memory is written only once it runs)
  else __syncthreads();
  pdl_wait();

  const int len = row_length(a, e);
  const int ntiles = (len + L - 1) / L, rounds = (ntiles + share - 1) / share;
  const int mine = ntiles > rank ? (ntiles - rank + share - 1) / share : 0;
  // the row's last tile first
  const auto fill = [&](int stage, int j) {
    if (!in_range(stage, STAGES)) return;
    unsigned char* to = ring_tiles + (size_t)stage * 4 * kTile;
    const int t = (rank + (mine - 1 - j) * share) * L;
    mbar_arrive_expect_tx(&sh.full[stage], 4 * kTile);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      tile_load(to + i * kTile, &maps.in[i], (int)cols.c0, i == 3 ? t - 1 : t, (int)e, &sh.full[stage]);
  };
  if (kBulk && threadIdx.x == 0)
    for (int j = 0; j < STAGES - 1 && j < mine; ++j) fill(j, j);

  const float zero[2] = {0.f, 0.f};
  float carry[2];
  load_state(cols, a.d_last, e, a.E, carry);
  if (len > 0 && flagged(a, e * a.step_e + (int64_t)(len - 1) * a.step_t)) carry[0] = carry[1] = 0.f;
  FillRing<STAGES> ring;
  int j = 0;
  const bool flags = a.terminated != nullptr || a.truncated != nullptr;
  const int64_t last0 = ((int64_t)rank + (int64_t)(rounds - 1) * share) * L + warp * kChunk;
  bool cut_next = flags && lane < kChunk && cut_before(a, e, last0 + lane, len);
  for (int k = rounds - 1; k >= 0; --k) {
    const int buf = k & 1;
    const int64_t t0 = ((int64_t)rank + (int64_t)k * share) * L + warp * kChunk;
    const int real = min(max(len - t0, (int64_t)0), (int64_t)kChunk);
    const uint32_t cut = __ballot_sync(kFullMask, cut_next);
    if (flags && lane < kChunk) cut_next = cut_before(a, e, t0 - (int64_t)share * L + lane, len);
    // a step's G is g + p u, u from behind the chunk; dx = na G, dgate = w G
    float p[kChunk][2], g[kChunk][2], na[kChunk][2], w[kChunk][2];
    Map2 m = make_float4(1.f, 0.f, 1.f, 0.f);
    if (k < mine) {
      const unsigned char* at = nullptr;
      if constexpr (kBulk) {
        if (threadIdx.x == 0 && ring.ok && j + STAGES - 1 < mine) fill(ring.fill_stage(), j + STAGES - 1);
        if (ring.ok) ring.ok = mbar_wait_bounded(&sh.full[ring.stage], ring.phase);
        at = ring_tiles + (size_t)ring.stage * 4 * kTile + ((size_t)warp * kChunk * kCols + 2 * lane) * Stor<ST>::kBytes;
        ring.next();
        ++j;
      }
      const int64_t row0 = e * a.step_e + t0 * a.step_t;
      float P[2] = {1.f, 1.f}, Q[2] = {0.f, 0.f};
      const auto read = [&](int i, float* x, float* gate, float* dh, float* before) {
        if constexpr (kBulk) {
          const unsigned char* r = at + (size_t)i * kCols * Stor<ST>::kBytes;
          open2<ST>(r, x);
          open2<ST>(r + kTile, gate);
          open2<ST>(r + 2 * kTile, dh);
          open2<ST>(r + 3 * kTile, before);
        } else {
          const int64_t row = row0 + i * a.step_t;
          x[0] = x[1] = gate[0] = gate[1] = dh[0] = dh[1] = before[0] = before[1] = 0.f;
          if (i < real) {
            cols.load(a.x, row * a.x_stride, n * a.x_stride, x);
            cols.load(a.gate, row * a.gate_stride, n * a.gate_stride, gate);
            cols.load(a.dh, row * a.dh_stride, n * a.dh_stride, dh);
            if (t0 + i > 0) cols.load(a.in_h, (row - a.step_t) * a.h_stride, n * a.h_stride, before);
          }
        }
      };
      if (cut == 0 && real == kChunk && t0 > 0) {
#pragma unroll
        for (int i = kChunk - 1; i >= 0; --i) {
          float x[2], gate[2], dh[2], before[2];
          read(i, x, gate, dh, before);
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const Gate s = gate_of<ST>(gate[c]);
            p[i][c] = P[c];
            g[i][c] = dh[c] + Q[c];
            na[i][c] = s.na;
            w[i][c] = s.a * s.na * (before[c] - x[c]);
            Q[c] = s.a * g[i][c];
            P[c] *= s.a;
          }
        }
      } else {
        float first[2] = {0.f, 0.f};
        if (t0 == 0) load_state(cols, a.state, e, a.E, first);
#pragma unroll
        for (int i = kChunk - 1; i >= 0; --i) {
          float x[2], gate[2], dh[2], before[2];
          read(i, x, gate, dh, before);
          const bool here = (cut >> i) & 1;
          if (t0 + i == 0) before[0] = first[0], before[1] = first[1];
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const Gate s = gate_of<ST>(gate[c]);
            p[i][c] = P[c];
            g[i][c] = Q[c];
            na[i][c] = w[i][c] = 0.f;
            if (i < real) {
              g[i][c] += dh[c];
              na[i][c] = s.na;
              w[i][c] = s.a * s.na * ((here ? 0.f : before[c]) - x[c]);
              Q[c] = here ? 0.f : s.a * g[i][c];
              P[c] = here ? 0.f : P[c] * s.a;
            }
          }
        }
        if (cut != 0) P[0] = P[1] = -0.f;
      }
      m = make_float4(P[0], Q[0], P[1], Q[1]);
    }
    sh.warp_map[buf][warp][lane] = m;
    __syncthreads();
    float u[2] = {carry[0], carry[1]};
    if (share > 1) {
      if (warp == 0) {
        Map2 all = sh.warp_map[buf][W - 1][lane];
#pragma unroll
        for (int v = W - 2; v >= 0; --v) all = chain(sh.warp_map[buf][v][lane], all);
        for (int r = 0; r < share; ++r) store_peer(&sh.cta_map[buf][rank][lane], r, all);
      }
      cluster_meet();
      for (int r = share - 1; r >= 0; --r) {
        pass(sh.cta_map[buf][r][lane], carry);
        if (r - 1 == rank) u[0] = carry[0], u[1] = carry[1];
      }
      for (int v = W - 1; v > warp; --v) pass(sh.warp_map[buf][v][lane], u);
    } else {
#pragma unroll
      for (int v = W - 1; v >= 0; --v) {
        if (v == warp) u[0] = carry[0], u[1] = carry[1];
        pass(sh.warp_map[buf][v][lane], carry);
      }
    }
    const int64_t row0 = e * a.step_e + t0 * a.step_t;
    const int reached = cut != 0 ? 31 - __clz(cut) : 0;  // the first step that u reaches
    if (k < mine && real == kChunk && cut == 0) {
#pragma unroll
      for (int i = 0; i < kChunk; ++i) {
        float dx[2], dg[2];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const float G = fmaf(p[i][c], u[c], g[i][c]);
          dx[c] = na[i][c] * G;
          dg[c] = w[i][c] * G;
        }
        cols.store(a.dx, (row0 + i * a.step_t) * a.dx_stride, n * a.dx_stride, dx);
        cols.store(a.dgate, (row0 + i * a.step_t) * a.dgate_stride, n * a.dgate_stride, dg);
      }
    } else {
#pragma unroll
      for (int i = 0; i < kChunk; ++i) {
        if (t0 + i >= a.T) continue;
        float dx[2] = {0.f, 0.f}, dg[2] = {0.f, 0.f};
        if (k < mine && i < real) {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const float G = i >= reached ? fmaf(p[i][c], u[c], g[i][c]) : g[i][c];
            dx[c] = na[i][c] * G;
            dg[c] = w[i][c] * G;
          }
        }
        cols.store(a.dx, (row0 + i * a.step_t) * a.dx_stride, n * a.dx_stride, dx);
        cols.store(a.dgate, (row0 + i * a.step_t) * a.dgate_stride, n * a.dgate_stride, dg);
      }
    }
  }
  for (int64_t t = ((int64_t)rounds * share + rank) * L; t < a.T; t += (int64_t)share * L)
    for (int i = 0; i < kChunk && t + warp * kChunk + i < a.T; ++i) {
      const int64_t row = e * a.step_e + (t + warp * kChunk + i) * a.step_t;
      cols.store(a.dx, row * a.dx_stride, n * a.dx_stride, zero);
      cols.store(a.dgate, row * a.dgate_stride, n * a.dgate_stride, zero);
    }
  if (rank == 0 && warp == 0 && a.d_state != nullptr) store_state(cols, a.d_state, e, a.E, carry);
  if constexpr (kBulk) {
    if (!ring.ok && threadIdx.x == 0)
      for (int i = 0; i < STAGES; ++i) mbar_wait_bounded(&sh.full[i], ring.last_fill(i));
  }
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
  constexpr int W = Stor<ST>::kBytes == 2 ? 8 : 4, L = kChunk * W, kStages = 3, es = Stor<ST>::kBytes;
  const int64_t units = a.E * div_up(a.D, kCols);
  if (a.T <= 4) return launch_serial(gated_serial_kernel<ST>, a, sm, s);
  const int share = row_share(units, div_up(a.T, L), sm);
  if (units * share > INT32_MAX) return launch_serial(gated_serial_kernel<ST>, a, sm, s);
  GatedMaps maps = {};
  if (rows_aligned({a.x, a.gate}, {a.x_stride, a.gate_stride}, es, 16) && rows_aligned({a.h}, {a.D}, es, 2 * es) &&
      encode_steps_map(&maps.in[0], a.x, es, a.D, a.T, a.E, a.x_stride * a.step_t, a.x_stride * a.step_e, kCols, L) &&
      encode_steps_map(&maps.in[1], a.gate, es, a.D, a.T, a.E, a.gate_stride * a.step_t, a.gate_stride * a.step_e, kCols, L)) {
    const auto kernel = gated_tile_kernel<ST, W, kStages, true>;
    const size_t smem = (size_t)kStages * 2 * L * kCols * es;
    static std::atomic<uint64_t> allowed;
    const cudaError_t e = allow_smem(kernel, smem, allowed);
    return e != cudaSuccess ? e : launch_tiles(kernel, units * share, 32 * W, smem, share, s, a, maps);
  }
  return launch_tiles(gated_tile_kernel<ST, W, 1, false>, units * share, 32 * W, 0, share, s, a, maps);
}

template <class ST>
cudaError_t grad_typed(const GatedArgs& a, int sm, cudaStream_t s) {
  constexpr int W = Stor<ST>::kBytes == 2 ? 8 : 4, L = kChunk * W, kStages = 3, es = Stor<ST>::kBytes;
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
    const auto kernel = gated_grad_tile_kernel<ST, W, kStages, true>;
    const size_t smem = (size_t)kStages * 4 * L * kCols * es;
    static std::atomic<uint64_t> allowed;
    const cudaError_t e = allow_smem(kernel, smem, allowed);
    return e != cudaSuccess ? e : launch_tiles(kernel, units * share, 32 * W, smem, share, s, a, maps);
  }
  return launch_tiles(gated_grad_tile_kernel<ST, W, 1, false>, units * share, 32 * W, 0, share, s, a, maps);
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
