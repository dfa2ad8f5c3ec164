// Token log-probabilities and entropies of a policy head, and their gradient.
//
// Three matrix products carry the work, all on the tensor cores (tc.cuh):
// the logits' tiles, whose epilogue keeps per half tile of 128 tokens a
// running (max, sum e^z, sum e^z z) -- or, in the gradient, turns the logits
// into dz --, and the two products of dz with the weight and with the hidden
// rows.  The logits exist in TMEM only; dz exists for one piece of the
// vocabulary at a time.
//
// Measured (device time of a whole call): 8192 x 4096 x 131072 bfloat16
// log-probabilities 5.37 to 5.45 ms, 1614 to 1638 TFLOP/s under the power cap (0.94 to
// 0.95 of the library product's sustained rate); 8192 x 4096 x 32768 alone 1.23 ms,
// 1788 TFLOP/s; the gradient at 4096 x 4096 x 32768 1.94 ms, 1700 TFLOP/s.
#include <algorithm>
#include <type_traits>

#include "policy.h"
#include "reduce.cuh"
#include "tc.cuh"

namespace rlca {

namespace {

// ---------------------------------------------------------------------------
// Workspace.  Rows that take part are numbered in order ("parts"); rows[]
// maps a part to its row, and count[0] is how many there are -- known on the
// device only, so launches are sized for all N rows and tiles past count[0]
// do not exist.  The parts' hidden rows are packed next to each other, so rows
// that take no part cost nothing and their contents (NaN included) reach no
// sum.  float32 operands are packed as three bfloat16 planes (tc.cuh); a
// weight that the copies cannot read in place -- float32, or rows that do not
// start on 16-byte boundaries -- is packed too, a piece at a time.
// ---------------------------------------------------------------------------
constexpr int64_t kPieceBytes = int64_t(1) << 30;    // dz of one piece of the vocabulary
constexpr int64_t kPackBytes = int64_t(256) << 20;   // packed weight of one piece
constexpr int64_t kSplitBytes = int64_t(64) << 20;   // d_hidden's partial sums beyond the first
constexpr int64_t kWholeStages = 24;                  // k stages (times terms) of a d_hidden sum that is not split
constexpr int64_t kSplitStages = 8;                   // ... and at least this many a split
constexpr int64_t kBandBytes = int64_t(48) << 20;    // hidden rows walked together (well inside L2)
constexpr float kLog2e = 1.4426950408889634f;

constexpr int64_t round_up(int64_t a, int64_t b) { return div_up(a, b) * b; }

// most pieces of the vocabulary that head_few_kernel leaves statistics of
constexpr int kFewCtasPerSm = 2;
int64_t few_pieces(int sm_count) { return kFewCtasPerSm * (int64_t)sm_count; }

struct HeadPlan {
  int planes;       // bfloat16 planes of an operand
  bool packed;      // the weight is packed
  int64_t Np;       // parts, rounded up to whole tiles
  int64_t Dp;       // pitch of packed rows
  int64_t Dh;       // pitch of d_hidden's float32 sums
  int64_t piece;    // tokens per piece (whole tiles unless it is the whole vocabulary)
  int64_t pitch;    // of dz and of the column of partial statistics: piece in whole tiles
  int row_tiles, d_tiles, splits;
  bool two_dz;      // dz as two bfloat16 values (their sum), the second's rows after the first's
  size_t count, rows, tok, info, hidden, weight, part, taken, dz, dh;  // byte offsets
  int64_t part_size, dh_size;  // elements
  size_t bytes;
};

HeadPlan plan_head(int64_t N, int64_t D, int64_t V, bool bf16_io, bool backward, bool packed, int sm_count) {
  HeadPlan p = {};
  p.planes = bf16_io ? 1 : 3;
  p.packed = packed;
  p.Np = round_up(N, kTcM);
  p.Dp = round_up(D, 8);
  p.Dh = round_up(D, 32);
  p.row_tiles = (int)(p.Np / kTcM);
  p.d_tiles = (int)div_up(D, kTcN);
  p.two_dz = backward && bf16_io && N <= kTcRows;
  const int64_t tiles = div_up(V, kTcN);
  int64_t piece_tiles = tiles;
  if (packed) piece_tiles = std::min(piece_tiles, std::max<int64_t>(1, kPackBytes / (2 * p.planes * p.Dp * kTcN)));
  if (backward) piece_tiles = std::min(piece_tiles, std::max<int64_t>(1, kPieceBytes / (2 * p.planes * p.Np * kTcN)));
  p.pitch = piece_tiles * kTcN;
  p.piece = std::min(p.pitch, V);
  // (offsets count from the workspace's first 256-byte boundary: the kernels
  // write 32 bytes at a time)
  size_t at = 0;
  const auto take = [&](size_t n) {
    const size_t here = at;
    at += (n + 255) & ~size_t(255);
    return here;
  };
  p.count = take(4);
  p.rows = take((size_t)N * 4);
  p.tok = take((size_t)N * 4);
  p.hidden = take((size_t)p.planes * p.Np * p.Dp * 2);
  if (packed) p.weight = take((size_t)p.planes * p.pitch * p.Dp * 2);
  if (backward) {
    p.info = take((size_t)N * sizeof(float4));
    p.dz = take((size_t)p.planes * p.Np * p.pitch * 2);
    // d_hidden has few tiles when there are few rows: its sum over tokens is
    // then split until the tiles fill the CTA pairs -- unless a whole sum is
    // hardly longer than the kernel that joins the splits (0.27 us a stage
    // against 5 to 6 us)
    const int64_t out_tiles = (int64_t)p.row_tiles * p.d_tiles, out_bytes = p.Np * p.Dh * 4;
    const int64_t stages = div_up(p.piece, kTcK);
    p.splits = 1;
    if ((p.two_dz ? 2 : 1) * stages > kWholeStages || piece_tiles < tiles)
      p.splits = (int)std::max<int64_t>(
          1, std::min({(int64_t)sm_count / 2 / out_tiles, 1 + kSplitBytes / out_bytes, div_up(stages, kSplitStages)}));
    // (one piece, not split: the product writes d_hidden itself)
    if (p.splits > 1 || piece_tiles < tiles) {
      p.dh_size = (p.two_dz ? 2 : 1) * p.splits * p.Np * p.Dh;
      p.dh = take((size_t)p.dh_size * sizeof(float));
    }
  } else {
    // (head_few_kernel: one piece a CTA, of at most 16 rows)
    p.part_size = std::max(tiles * 2 * p.Np, few_pieces(sm_count) * 16);
    p.part = take((size_t)p.part_size * sizeof(float4));
    p.taken = take((size_t)p.Np * 4);
  }
  p.bytes = at + 255;
  return p;
}

struct HeadView {  // the workspace's arrays on the device
  int* count;
  int* rows;
  int* tok;
  float4* info;  // per part: d_logp, d_entropy, lse, entropy
  void *hidden, *weight;
  float4* part;
  float* taken;
  uint16_t* dz;
  float* dh;
  // elements of part, hidden, weight (planes and all) and dh
  int64_t part_size, hidden_size, weight_size, dh_size;
  HeadView(const HeadPlan& p, void* ws) {
    unsigned char* b = reinterpret_cast<unsigned char*>(((uintptr_t)ws + 255) & ~(uintptr_t)255);
    count = reinterpret_cast<int*>(b + p.count);
    rows = reinterpret_cast<int*>(b + p.rows);
    tok = reinterpret_cast<int*>(b + p.tok);
    info = reinterpret_cast<float4*>(b + p.info);
    hidden = b + p.hidden;
    weight = b + p.weight;
    part = reinterpret_cast<float4*>(b + p.part);
    taken = reinterpret_cast<float*>(b + p.taken);
    dz = reinterpret_cast<uint16_t*>(b + p.dz);
    dh = reinterpret_cast<float*>(b + p.dh);
    part_size = p.part_size, dh_size = p.dh_size;
    hidden_size = p.planes * p.Np * p.Dp;
    weight_size = p.packed ? p.planes * p.pitch * p.Dp : 0;
  }
};

// ---------------------------------------------------------------------------
// Packing
// ---------------------------------------------------------------------------

// v as the sum of three bfloat16 values, each the rounding of the remainder:
// exact to 24 bits (the remainders are exact in float32)
__device__ __forceinline__ void split3(float v, float& hi, float& mid, float& lo) {
  hi = __bfloat162float(__float2bfloat16_rn(v));
  const float r = v - hi;
  mid = __bfloat162float(__float2bfloat16_rn(r));
  lo = r - mid;
}

// Eight elements from column c of a row that starts at element `at`, as they
// lie in memory, zeros from `width` on.  `size`: elements from src to the end
// of the matrix.  A row that starts off a 16-byte boundary is read as the
// aligned vectors around the eight elements, shifted into place, where those
// vectors lie inside the matrix; otherwise element by element.
template <class ST>
struct Eight {
  static constexpr int ES = Stor<ST>::kBytes, NV = 8 * ES / 16;  // vectors that eight elements fill
  uint32_t w[4 * NV + 4];

  __device__ __forceinline__ void load(const float* src, int64_t size, int64_t at, int64_t c, int64_t width) {
    const uintptr_t p = (uintptr_t)src + (uintptr_t)(at + c) * ES;
    const uint32_t off = (uint32_t)(p & 15);
    const uintptr_t lo = p - off, hi = lo + 16 * (NV + (off ? 1 : 0));
    if (lo >= (uintptr_t)src && hi <= (uintptr_t)src + (uintptr_t)size * ES) {
      const uint4* q = reinterpret_cast<const uint4*>(lo);
#pragma unroll
      for (int i = 0; i <= NV; ++i) {
        const uint4 x = i < NV || off ? __ldg(q + i) : make_uint4(0u, 0u, 0u, 0u);
        w[4 * i] = x.x, w[4 * i + 1] = x.y, w[4 * i + 2] = x.z, w[4 * i + 3] = x.w;
      }
      if (off) {
#pragma unroll
        for (int i = 0; i + 2 < 4 * NV + 4; ++i) w[i] = off & 8 ? w[i + 2] : w[i];
#pragma unroll
        for (int i = 0; i + 3 < 4 * NV + 4; ++i) w[i] = off & 4 ? w[i + 1] : w[i];
        if (ES == 2 && (off & 2)) {
#pragma unroll
          for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 16);
        }
      }
      if (c + 8 > width) {
#pragma unroll
        for (int i = 0; i < 4 * NV; ++i) {
          if (ES == 4) w[i] = c + i < width ? w[i] : 0u;
          else w[i] = c + 2 * i + 1 < width ? w[i] : c + 2 * i < width ? w[i] & 0xffffu : 0u;
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4 * NV; ++i) {
        if constexpr (ES == 4) {
          w[i] = c + i < width && in_range(at + c + i, size) ? __float_as_uint(Stor<ST>::ld(src, at + c + i)) : 0u;
        } else {
          const int64_t k = c + 2 * i;
          const uint16_t* e = reinterpret_cast<const uint16_t*>(src) + at + k;
          w[i] = (k < width && in_range(at + k, size) ? (uint32_t)__ldg(e) : 0u) |
                 (k + 1 < width && in_range(at + k + 1, size) ? (uint32_t)__ldg(e + 1) << 16 : 0u);
        }
      }
    }
  }
  // ... to element `to` of the packed planes, `plane` elements apart, `size` in all
  __device__ __forceinline__ void pack(void* planes, int64_t to, int64_t plane, int64_t size) const {
    if (!span_in_range(to, 8 + (ES == 2 ? 0 : 2 * plane), size)) return;
    if constexpr (ES == 2) {
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(planes) + to) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
      float* dst = static_cast<float*>(planes);  // Stor<bf16> counts in elements of two bytes
      float h[8], m[8], l[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) split3(__uint_as_float(w[i]), h[i], m[i], l[i]);
      Stor<bf16>::st8(dst, to, h);
      Stor<bf16>::st8(dst, to + plane, m);
      Stor<bf16>::st8(dst, to + 2 * plane, l);
    }
  }
};

constexpr int kPackThreads = 256;

// (8192 rows of 4096: 8 us when they stay where they are; packing moves 128
// MB.  A pass of one CTA over the tokens and a packing pass took 34 us.)
// Numbers the rows that take part, in order, gathers their tokens and factors,
// packs their hidden rows (unless all take part and can be read in place), and
// clears the results of the other rows.  A CTA
// takes rows_per_cta rows and counts the parts before them (and in all) by
// itself: N tokens from L2 instead of a pass of its own and a wait.  With
// pad, the packed rows are zeroed to the next whole stage of k: the gradient's
// product over parts reads them.
template <class ST>
__global__ void __launch_bounds__(kPackThreads)
    head_begin_kernel(HeadArgs a, HeadView w, int64_t rows_per_cta, int64_t Dp, int64_t Np, bool pad,
                      bool in_place) {
  pdl_trigger();
  pdl_wait();
  __shared__ int scratch[32], list[kPackThreads];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t r0 = blockIdx.x * rows_per_cta, r1 = min(a.N, r0 + rows_per_cta);
  int before = 0, all = 0;
#pragma unroll 8
  for (int64_t i = threadIdx.x; i < a.N; i += kPackThreads) {
    const int on = (unsigned)__ldg(a.tokens + i) < (unsigned)a.V;
    all += on;
    before += i < r0 ? on : 0;
  }
  before = cta_sum(before, scratch);
  all = cta_sum(all, scratch);
  if (blockIdx.x == 0 && threadIdx.x == 0) w.count[0] = all;

  // all rows take part and the copies can read them where they lie
  const bool pack = !(in_place && all == a.N);
  const int groups = (int)(Dp / 8);
  const int64_t plane = Np * Dp;
  const int64_t size = (a.N - 1) * a.hidden_stride + a.D;
  for (int64_t i0 = r0; i0 < r1; i0 += kPackThreads) {
    const int64_t i = i0 + threadIdx.x;
    const int tok = i < r1 ? a.tokens[i] : -1;
    const bool on = (unsigned)tok < (unsigned)a.V;
    const unsigned vote = __ballot_sync(0xffffffffu, on);
    if (lane == 0) scratch[warp] = __popc(vote);
    __syncthreads();
    int at = __popc(vote & ((1u << lane) - 1u)), n = 0;
#pragma unroll
    for (int k = 0; k < kPackThreads / 32; ++k) {
      at += k < warp ? scratch[k] : 0;
      n += scratch[k];
    }
    if (on && in_range(before + at, a.N) && in_range(at, kPackThreads)) {
      list[at] = (int)i;
      w.rows[before + at] = (int)i;
      w.tok[before + at] = tok;
      if (a.d_logp != nullptr)
        w.info[before + at] = make_float4(a.d_logp[i], a.d_entropy ? a.d_entropy[i] : 0.f, a.in_lse[i],
                                          a.d_entropy ? a.in_entropy[i] : 0.f);
    } else if (!on && i < r1 && in_range((i - i0) - at, kPackThreads)) {
      list[kPackThreads - 1 - ((int)(i - i0) - at)] = (int)i;  // from the end: those that do not
      if (a.logp != nullptr) {
        a.logp[i] = 0.f;
        a.lse[i] = 0.f;
        if (a.entropy) a.entropy[i] = 0.f;
      }
    }
    __syncthreads();
    if (a.d_hidden != nullptr) {
      const int off = (int)min((int64_t)kPackThreads, r1 - i0) - n;
      for (int r = 0; r < off; ++r) {
        const int64_t to = list[kPackThreads - 1 - r] * a.D;
        for (int64_t c = threadIdx.x; c < a.D; c += kPackThreads)
          if (in_range(to + c, a.N * a.D)) Stor<ST>::st(a.d_hidden, to + c, 0.f);
      }
    }
    constexpr int B = 4;  // groups a thread has in flight
    for (int t0 = threadIdx.x; pack && t0 < n * groups; t0 += B * kPackThreads) {
      Eight<ST> v[B];
      int64_t to[B];
#pragma unroll
      for (int u = 0; u < B; ++u) {
        const int t = min(t0 + u * kPackThreads, n * groups - 1);
        const int r = t / groups, c = (t - r * groups) * 8;
        v[u].load(a.hidden, size, list[r] * a.hidden_stride, c, a.D);
        to[u] = (int64_t)(before + r) * Dp + c;
      }
#pragma unroll
      for (int u = 0; u < B; ++u)
        if (t0 + u * kPackThreads < n * groups) v[u].pack(w.hidden, to[u], plane, w.hidden_size);
    }
    before += n;
    __syncthreads();
  }
  if (!pad || !pack) return;
  const int64_t end = min(Np, ((int64_t)all + kTcK - 1) / kTcK * kTcK);
  for (int64_t r = all + blockIdx.x; r < end; r += gridDim.x)
    for (int c = threadIdx.x; c < groups; c += kPackThreads) {
      Eight<ST> zero = {};
      zero.pack(w.hidden, r * Dp + c * 8, plane, w.hidden_size);
    }
}

// the weight's rows [r0, r0 + rows) packed, zeros past the width (float32:
// 89 MB to 134 MB in 33 us; bfloat16 rows of 2999: 268 MB to 268 MB in 108 us,
// 5 TB/s -- with a division a vector and a detour through float32 149 us)
struct PackArgs {
  const float* src;
  int64_t size;  // elements from src to the end of the matrix
  int64_t r0, rows, width, stride;
  void* dst;  // planes x [dst_rows, pitch]
  int64_t pitch, dst_rows, dst_size;
};
template <class ST>
__global__ void __launch_bounds__(kPackThreads) head_pack_kernel(PackArgs a) {
  pdl_trigger();
  pdl_wait();
  // a warp's lanes side by side on a row, or on several narrow ones
  const int groups = (int)(a.pitch / 8);
  int lanes = 32;
  while (lanes > 1 && lanes / 2 >= groups) lanes /= 2;
  const int lane = threadIdx.x & 31, sub = lane & (lanes - 1), rows = 32 / lanes;
  const int64_t warp = (int64_t)blockIdx.x * (kPackThreads / 32) + (threadIdx.x >> 5);
  const int64_t step = (int64_t)gridDim.x * (kPackThreads / 32) * rows;
  constexpr int B = 4;
  for (int64_t r = warp * rows + lane / lanes; r < a.rows; r += step) {
    const int64_t at = (a.r0 + r) * a.stride, to = r * a.pitch;
    for (int g0 = sub; g0 < groups; g0 += B * lanes) {
      Eight<ST> v[B];
#pragma unroll
      for (int u = 0; u < B; ++u)
        if (g0 + u * lanes < groups) v[u].load(a.src, a.size, at, (g0 + u * lanes) * 8, a.width);
#pragma unroll
      for (int u = 0; u < B; ++u)
        if (g0 + u * lanes < groups) v[u].pack(a.dst, to + (g0 + u * lanes) * 8, a.dst_rows * a.pitch, a.dst_size);
    }
  }
}

// ---------------------------------------------------------------------------
// Epilogues (one row of C a thread, 32 columns at a time)
// ---------------------------------------------------------------------------
__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// two float32 values in one 64-bit register: one instruction for both
__device__ __forceinline__ uint64_t pair_of(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void pair_open(uint64_t p, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(p));
}
__device__ __forceinline__ uint64_t pair_fma(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t pair_add(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t pair_mul(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
// 32 bytes at p (32-byte aligned): a whole sector from one thread
__device__ __forceinline__ void store32(void* p, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}
// sixteen values as bfloat16
__device__ __forceinline__ void store16(uint16_t* p, const float* v) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = Stor<bf16>::pack2(v[2 * i], v[2 * i + 1]);
  store32(p, w);
}

// Partial statistics over some of a part's tokens: top, the largest logit
// (before the temperature); s, the sum of e = 2^(c2 d); t, the sum of e d, with
// d = z - top and c2 = log2(e) / temperature.  The difference comes first: a z c2
// and a top c2 rounded apart, or a sum of e z, would put errors of the size of
// the logits, not of their spread, into the sums.
struct Stats {
  float top, s, t;
  // moves the sums to a top that is no lower
  __device__ __forceinline__ void rebase(float to, float c2) {
    const float down = s == 0.f ? 0.f : top - to, f = exp2_approx(down * c2);  // (no sums: off inf - inf)
    s *= f;  // (first: where f is 0, down may be of any size)
    t = fmaf(s, down, t * f);
    top = to;
  }
  __device__ __forceinline__ void add(Stats o, float c2) {
    const float m = fmaxf(top, o.top);
    rebase(m, c2);
    o.rebase(m, c2);
    s += o.s;
    t += o.t;
  }
  // ... those of the warp's other lanes
  __device__ __forceinline__ void add_lanes(float c2) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      add({__shfl_xor_sync(0xffffffffu, top, o), __shfl_xor_sync(0xffffffffu, s, o), __shfl_xor_sync(0xffffffffu, t, o)}, c2);
  }
};
constexpr float kNoTop = -INFINITY;  // of no logits

// part[half tile][part] = its statistics.  The product runs at 79% of the
// tensor pipe with partial sums every 512 k (2048 x 4096 x 32768: 320 us, 1717
// TFLOP/s); without their TMEM reads 7% less time.  At k = 256 the epilogue is the
// limit (2048 x 256 x 131072: 127 us, the tensor pipe at 48%): 4500 cycles a tile,
// 2048 of them for its 32768 exponentials, 16 an SM and cycle.
struct StatsEpi {
  float4* part;
  float* taken;
  const int* tok;
  int64_t Np, halves;
  int v0, v_end;  // tokens of this piece
  float c2;

  struct State {
    Stats sums;
    int m, at, col0;
    bool live;
  };
  __device__ __forceinline__ void begin(State& st, const TcWalk& w, const TcTile&, int row, int col0) const {
    st.m = row;
    st.live = row < w.m;
    st.at = st.live ? tok[row] - v0 : -1;
    st.col0 = col0;
    st.sums = {kNoTop, 0.f, 0.f};
  }
  __device__ __forceinline__ void chunk(State& st, int col, float (&v)[32], float* block) const {
    const int n = v_end - v0 - col;  // columns that exist
    if (n <= 0) return;
    const int k = st.at - col;
    if (k >= 0 && k < 32) {
      float z = v[0];
#pragma unroll
      for (int i = 1; i < 32; ++i) z = i == k ? v[i] : z;
      if (in_range(st.m, Np)) taken[st.m] = z;
    }
    if (n < 32) {  // the others take the first one's place for now
#pragma unroll
      for (int i = 1; i < 32; ++i) v[i] = i < n ? v[i] : v[0];
    }
    Stats q = st.sums;
    float top = q.top;
#pragma unroll
    for (int i = 0; i < 32; i += 2) asm("max.f32 %0, %0, %1, %2;" : "+f"(top) : "f"(v[i]), "f"(v[i + 1]));
    if (n < 32) {  // ... and one that is far below the largest, whatever its size: d finite, e = 0
      const float low = top - fmaxf(fabsf(top), 2000.f / c2);
#pragma unroll
      for (int i = 1; i < 32; ++i) v[i] = i < n ? v[i] : low;
    }
    q.rebase(top, c2);
    const uint64_t c22 = pair_of(c2, c2), off2 = pair_of(-top, -top);
    uint64_t s2 = pair_of(q.s, 0.f), t2 = pair_of(q.t, 0.f);
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
      const uint64_t d2 = pair_add(pair_of(v[i], v[i + 1]), off2);
      float x0, x1;
      pair_open(pair_mul(d2, c22), x0, x1);
      const uint64_t e2 = pair_of(exp2_approx(x0), exp2_approx(x1));
      s2 = pair_add(s2, e2);
      t2 = pair_fma(e2, d2, t2);
    }
    float s, t, hi;
    pair_open(s2, s, hi);
    s += hi;
    pair_open(t2, t, hi);
    t += hi;
    st.sums = {top, s, t};
  }
  __device__ __forceinline__ void end(State& st) const {
    const int64_t at = (int64_t)((v0 + st.col0) / (kTcN / 2)) * Np + st.m;
    if (st.live && in_range(at, halves * Np)) part[at] = make_float4(st.sums.top, st.sums.s, st.sums.t, 0.f);
  }
};

// (2048 x 4096 x 16384: 162 us, 82% of the tensor pipe.)
// dz = p (a0 + a1 log p), plus g / temperature for the token taken, with
// log p = acc / temperature - lse rounded once, for the exponent and the factor
// alike: terms of the size of the logits or of lse would leave their rounding
// in either.  As three planes where the operands are float32; for bfloat16
// operands as one bfloat16, rounded once because the two products that read it
// run on bfloat16 -- its error of 2^-9 a term is as large as the rounding of the
// gradients themselves, and adds to it (2.4e-3 off in the 2-norm where results
// rounded once are 1.7e-3 off).  A second bfloat16 for what the first left over
// would make two of the three products twice as long.  Up to 128 rows half of
// each 256-row tile is empty otherwise, and it takes that half, in rows 128
// further on: 1.7e-3 off, for 84 instead of 73 us (128 x 1024 x 32768; 202
// instead of 192 at 4096 columns).
template <int PLANES>
struct DzEpi {
  uint16_t* dz;
  int64_t pitch, plane, size;  // size: of all planes
  const float4* info;
  const int* tok;
  int v0;
  float inv_t;
  bool two;

  struct State {
    float lse, a0, a1, g;
    int at;
    bool live, skip;
    uint16_t* row;
  };
  __device__ __forceinline__ void begin(State& st, const TcWalk& w, const TcTile&, int row, int) const {
    st.live = row < w.m;
    st.skip = two && row >= kTcRows;  // the second values' rows
    st.row = dz + (int64_t)row * pitch;
    st.at = -1;
    st.lse = st.a0 = st.a1 = st.g = 0.f;
    if (st.live) {
      const float4 f = info[row];
      st.at = tok[row] - v0;
      st.g = f.x * inv_t;
      st.a0 = -fmaf(f.y, f.w, f.x) * inv_t;
      st.a1 = -f.y * inv_t;
      st.lse = f.z;
    }
  }
  __device__ __forceinline__ void chunk(State& st, int col, float (&v)[32], float* block) const {
    if (st.skip) return;
    const int k = st.at - col;
    const uint64_t t2 = pair_of(inv_t, inv_t), l2 = pair_of(-st.lse, -st.lse), e2 = pair_of(kLog2e, kLog2e);
    const uint64_t a02 = pair_of(st.a0, st.a0), a12 = pair_of(st.a1, st.a1);
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
      const uint64_t logp = pair_fma(pair_of(v[i], v[i + 1]), t2, l2);
      float x0, x1;
      pair_open(pair_mul(logp, e2), x0, x1);
      const uint64_t p = pair_of(exp2_approx(x0), exp2_approx(x1));
      pair_open(pair_mul(p, pair_fma(a12, logp, a02)), v[i], v[i + 1]);
    }
    if (k >= 0 && k < 32) {
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] += i == k ? st.g : 0.f;
    }
    if (!st.live) {  // whatever the packed row holds
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = 0.f;
    }
    const int64_t at = (st.row - dz) + col;
    if (!span_in_range(at, 32 + (two ? kTcRows * pitch : (PLANES - 1) * plane), size)) return;
    if constexpr (PLANES == 1) {
      store16(st.row + col, v);
      store16(st.row + col + 16, v + 16);
      if (two) {
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] -= __bfloat162float(__float2bfloat16_rn(v[i]));
        store16(st.row + kTcRows * pitch + col, v);
        store16(st.row + kTcRows * pitch + col + 16, v + 16);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 32; i += 16) {
        float h[16], m[16], l[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) split3(v[i + j], h[j], m[j], l[j]);
        store16(st.row + col + i, h);
        store16(st.row + plane + col + i, m);
        store16(st.row + 2 * plane + col + i, l);
      }
    }
  }
  __device__ __forceinline__ void end(State&) const {}
};

// 32 values a lane from column `col` on, each lane's to its row that starts
// at element `at` of a matrix of `width` columns (rows that are not `live`
// excepted), rounded once.  align: what the rows' starts are multiples of, in
// bytes.  On 16-byte boundaries each lane writes its own row; elsewhere that
// would be 32 rows an instruction, one element each (20 x 1001 x 30000: 291 us
// for 60 MB), so the block goes through shared memory and the warp writes row
// by row.
template <class ST>
__device__ __forceinline__ void store_rows32(float* out, bool live, int64_t at, int64_t col, int64_t width, int align,
                                             const float* v, float* block) {
  if (align < 16) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < 32; ++i) block[lane * 33 + i] = v[i];
    __syncwarp();
    const unsigned rows = __ballot_sync(0xffffffffu, live);
    const bool on = col + lane < width;
#pragma unroll 4
    for (int r = 0; r < 32; ++r) {
      const int64_t to = __shfl_sync(0xffffffffu, at, r) + col + lane;
      if (on && (rows >> r & 1u)) Stor<ST>::st(out, to, block[r * 33 + lane]);
    }
    __syncwarp();
    return;
  }
  if (!live) return;
  if (align >= 32 && col + 32 <= width) {
    unsigned char* p = reinterpret_cast<unsigned char*>(out) + (at + col) * Stor<ST>::kBytes;
    if constexpr (Stor<ST>::kBytes == 2) {
      store16(reinterpret_cast<uint16_t*>(p), v);
      store16(reinterpret_cast<uint16_t*>(p) + 16, v + 16);
    } else {
#pragma unroll
      for (int i = 0; i < 32; i += 8) {
        uint32_t r[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) r[j] = __float_as_uint(v[i + j]);
        store32(p + 4 * i, r);
      }
    }
  } else {
    // (a width of whole 16-byte vectors: none is cut)
    constexpr int E = 16 / Stor<ST>::kBytes;
#pragma unroll
    for (int i = 0; i < 32; i += E) {
      if (col + i < width) {
        if constexpr (E == 8) Stor<ST>::st8(out, at + col + i, v + i);
        else Stor<ST>::st4(out, at + col + i, v + i);
      }
    }
  }
}

// (d_hidden and d_weight in one launch at 2048 x 4096 x 16384: 329 us, 84% of
// the tensor pipe; float32 at 768 x 1024 x 16384, six products: 192 us, 83%.)
// d_hidden.  The sum over the pieces of the vocabulary is kept in float32
// (`sums`, one plane a split), set by the first piece and added to by the
// others; without splits the last piece writes the result itself, to the
// part's row.  halves: rows 128 on are the sums with dz's second values, a
// plane of their own.
template <class ST>
struct DhEpi {
  float* sums;  // planes x [rows, pitch], `size` in all
  int64_t pitch, plane, size;
  bool first, last;
  float* out;  // [N, width], type ST
  const int* rows;
  int64_t N, width;
  int align;
  bool halves;

  struct State {
    float* sum;
    int64_t at;
    bool live;
  };
  __device__ __forceinline__ void begin(State& st, const TcWalk& w, const TcTile& t, int row, int) const {
    const int part = halves ? row % kTcRows : row;
    st.live = part < w.count;
    st.sum = sums + (halves ? 2 * t.split + row / kTcRows : t.split) * plane + (int64_t)part * pitch;
    st.at = last && st.live ? rows[part] * width : 0;
  }
  __device__ __forceinline__ void chunk(State& st, int col, float (&v)[32], float* block) const {
    if (col >= pitch) return;
    if (!first && st.live && span_in_range(st.sum - sums + col, 32, size)) {
#pragma unroll
      for (int i = 0; i < 32; i += 4) {
        const float4 o = *reinterpret_cast<const float4*>(st.sum + col + i);
        v[i] += o.x, v[i + 1] += o.y, v[i + 2] += o.z, v[i + 3] += o.w;
      }
    }
    if (last) {
      store_rows32<ST>(out, st.live && in_range(st.at, N * width), st.at, col, width, align, v, block);
    } else if (st.live && span_in_range(st.sum - sums + col, 32, size)) {
#pragma unroll
      for (int i = 0; i < 32; i += 8) {
        uint32_t r[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) r[j] = __float_as_uint(v[i + j]);
        store32(st.sum + col + i, r);
      }
    }
  }
  __device__ __forceinline__ void end(State&) const {}
};

// d_weight, rounded once
template <class ST>
struct OutEpi {
  float* out;  // [V, width], element type ST
  int64_t row0, width, V;
  int align;

  struct State {
    int64_t at;
    bool live;
  };
  __device__ __forceinline__ void begin(State& st, const TcWalk& w, const TcTile&, int row, int) const {
    st.live = row < w.m;
    st.at = (row0 + row) * width;
  }
  __device__ __forceinline__ void chunk(State& st, int col, float (&v)[32], float* block) const {
    store_rows32<ST>(out, st.live && in_range(st.at, V * width), st.at, col, width, align, v, block);
  }
  __device__ __forceinline__ void end(State&) const {}
};

// ---------------------------------------------------------------------------
constexpr int kJoinThreads = 256;

__device__ __forceinline__ Stats part_at(const HeadView& w, int64_t i, bool on) {
  if (!on || !in_range(i, w.part_size)) return {kNoTop, 0.f, 0.f};
  const float4 p = __ldg(w.part + i);
  return {p.x, p.y, p.z};
}

// the results of part m, from all its statistics
__device__ __forceinline__ void finish(const HeadArgs& a, const HeadView& w, int64_t m, int64_t row, const Stats& st) {
  if (!in_range(row, a.N) || !in_range(m, a.N)) return;
  const float inv_t = a.inv_temperature, log_s = logf(st.s);
  a.lse[row] = fmaf(st.top, inv_t, log_s);
  a.logp[row] = fmaf(w.taken[m] - st.top, inv_t, -log_s);
  if (a.entropy) a.entropy[row] = fmaf(-st.t / st.s, inv_t, log_s);
}

// (33 MB of statistics at 8192 parts x 256 half tiles: 17 us cold, 1.4% of
// the product they come from.)
// Joins the statistics of `pieces` pieces of the vocabulary: 32 parts a CTA,
// neighbouring lanes on neighbouring parts; warp k takes the pieces k, k + 32,
// ... four at a time, and the warps' results are joined in order.
constexpr int kJoinWarps = 32;
__global__ void __launch_bounds__(32 * kJoinWarps)
    head_join_kernel(HeadArgs a, HeadView w, int64_t pieces, int64_t pitch, float c2) {
  pdl_trigger();
  pdl_wait();
  __shared__ Stats acc[kJoinWarps][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t m = (int64_t)blockIdx.x * 32 + lane;
  if ((int64_t)blockIdx.x * 32 >= w.count[0]) return;
  const bool on = m < w.count[0];
  Stats st = {kNoTop, 0.f, 0.f};
  if (on) {
    for (int64_t k = warp; k < pieces; k += 4 * kJoinWarps) {
      Stats p[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) p[u] = part_at(w, (k + u * kJoinWarps) * pitch + m, k + u * kJoinWarps < pieces);
#pragma unroll
      for (int u = 0; u < 4; ++u) st.add(p[u], c2);
    }
  }
  acc[warp][lane] = st;
  __syncthreads();
  if (warp != 0 || !on) return;
  for (int k = 1; k < kJoinWarps; ++k) st.add(acc[k][lane], c2);
  finish(a, w, m, w.rows[m], st);
}

// ... with few parts: one CTA a part, its threads on the pieces.  identity:
// part m is row m, whether it takes part or not.
__global__ void __launch_bounds__(kJoinThreads)
    head_join_few_kernel(HeadArgs a, HeadView w, int64_t pieces, int64_t pitch, float c2, bool identity) {
  pdl_trigger();
  pdl_wait();
  constexpr int W = kJoinThreads / 32;
  __shared__ Stats acc[W];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t m = blockIdx.x;
  if (!identity && m >= w.count[0]) return;
  Stats st = {kNoTop, 0.f, 0.f};
  for (int64_t k = threadIdx.x; k < pieces; k += 4 * kJoinThreads) {
    Stats p[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) p[u] = part_at(w, (k + u * kJoinThreads) * pitch + m, k + u * kJoinThreads < pieces);
#pragma unroll
    for (int u = 0; u < 4; ++u) st.add(p[u], c2);
  }
  st.add_lanes(c2);
  if (lane == 0) acc[warp] = st;
  __syncthreads();
  if (threadIdx.x != 0) return;
#pragma unroll
  for (int k = 1; k < W; ++k) st.add(acc[k], c2);
  const int64_t row = identity ? m : w.rows[m];
  if (!in_range(row, a.N)) return;
  const bool on = (unsigned)a.tokens[row] < (unsigned)a.V;
  if (on) {
    finish(a, w, m, row, st);
  } else {
    a.lse[row] = a.logp[row] = 0.f;
    if (a.entropy) a.entropy[row] = 0.f;
  }
}

// ---------------------------------------------------------------------------
// A few rows (serving: one new token a sequence).  The weight is read once at
// the rate of HBM, so nothing is to be gained from the tensor cores, whose
// tiles of 256 rows would be almost empty: each warp forms the logits of R
// tokens x NT rows at a time in float32, its lanes side by side on the width,
// the hidden rows in shared memory.  The 32-lane sums of the R x NT logits
// share their shuffles (each step halves the values a lane carries), which
// leaves each lane with one logit, whose running statistics it keeps.
// ---------------------------------------------------------------------------
constexpr int kFewThreads = 256;
constexpr size_t kFewSmem = 96 * 1024;

template <class ST, int VE, int NT, int R>
__global__ void __launch_bounds__(kFewThreads, kFewCtasPerSm)
    head_few_kernel(HeadArgs a, HeadView w, int64_t Ds, float c2) {
  extern __shared__ __align__(16) float few_hidden[];  // [NT][Ds], zeros past D
  constexpr int C = R * NT, W = kFewThreads / 32;
  constexpr int kUnroll = VE == 1 ? (Stor<ST>::kBytes == 2 ? 6 : 8) : NT <= 2 ? 16 / R : 2;
  constexpr int kLog = C == 4 ? 2 : C == 8 ? 3 : C == 16 ? 4 : 5;  // log2 C
  __shared__ Stats acc[W][C];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_trigger();
  pdl_wait();
  for (int64_t t = threadIdx.x; t < NT * Ds; t += kFewThreads) {
    const int64_t r = t / Ds, c = t - r * Ds;
    few_hidden[t] = r < a.N && c < a.D && in_range(r * a.hidden_stride + c, (a.N - 1) * a.hidden_stride + a.D)
                        ? Stor<ST>::ld(a.hidden, r * a.hidden_stride + c)
                        : 0.f;
  }
  __syncthreads();
  const int mine = lane >> (5 - kLog);           // the logit this lane ends up with:
  const int my_tok = mine / NT, my_row = mine % NT;  // token my_tok of the R, row my_row
  const int64_t taken_tok = my_row < a.N ? a.tokens[my_row] : -1;
  Stats st = {kNoTop, 0.f, 0.f};
  const int64_t nv = a.D / VE, w_size = (a.V - 1) * a.weight_stride + a.D;
  for (int64_t v0 = ((int64_t)blockIdx.x * W + warp) * R; v0 < a.V; v0 += (int64_t)gridDim.x * W * R) {
    float z[C];
    // vectors: sums of the even and of the odd columns, two to an instruction
    uint64_t zz[VE >= 4 ? C : 1];
#pragma unroll
    for (int i = 0; i < C; ++i) z[i] = 0.f;
#pragma unroll
    for (int i = 0; i < (VE >= 4 ? C : 1); ++i) zz[i] = 0;
    const float* base[R];
#pragma unroll
    for (int r = 0; r < R; ++r)
      base[r] = reinterpret_cast<const float*>(reinterpret_cast<const unsigned char*>(a.weight) +
                                               min(v0 + r, a.V - 1) * a.weight_stride * Stor<ST>::kBytes);
#pragma unroll kUnroll
    for (int64_t j = lane; j < nv; j += 32) {
      float x[R][VE];
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const bool in = span_in_range(min(v0 + r, a.V - 1) * a.weight_stride + j * VE, VE, w_size) && span_in_range(j * VE, VE, Ds);
        if constexpr (VE == 8) Stor<ST>::ld8(base[r], j * VE, in, x[r]);
        else if constexpr (VE == 4) Stor<ST>::ld4(base[r], j * VE, in, x[r]);
        else x[r][0] = in ? Stor<ST>::ld(base[r], j) : 0.f;
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        if constexpr (VE >= 4) {
#pragma unroll
          for (int e = 0; e < VE; e += 4) {
            const ulonglong2 h = *reinterpret_cast<const ulonglong2*>(few_hidden + n * Ds + j * VE + e);
#pragma unroll
            for (int r = 0; r < R; ++r) {
              zz[r * NT + n] = pair_fma(pair_of(x[r][e], x[r][e + 1]), h.x, zz[r * NT + n]);
              zz[r * NT + n] = pair_fma(pair_of(x[r][e + 2], x[r][e + 3]), h.y, zz[r * NT + n]);
            }
          }
        } else {
          const float h = few_hidden[n * Ds + j];
#pragma unroll
          for (int r = 0; r < R; ++r) z[r * NT + n] = fmaf(x[r][0], h, z[r * NT + n]);
        }
      }
    }
    if constexpr (VE >= 4) {
#pragma unroll
      for (int i = 0; i < C; ++i) {
        float even, odd;
        pair_open(zz[i], even, odd);
        z[i] = even + odd;
      }
    }
    int n = C;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      if (n > 1) {
        n /= 2;
        const bool up = (lane & o) != 0;
#pragma unroll
        for (int i = 0; i < C / 2; ++i)
          if (i < n) {
            const float give = up ? z[i] : z[i + n], keep = up ? z[i + n] : z[i];
            z[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
          }
      } else {
        z[0] += __shfl_xor_sync(0xffffffffu, z[0], o);
      }
    }
    if (v0 + my_tok < a.V) {
      st.add({z[0], 1.f, 0.f}, c2);
      if (v0 + my_tok == taken_tok && (lane & ((32 >> kLog) - 1)) == 0 && in_range(my_row, a.N)) w.taken[my_row] = z[0];
    }
  }
  if ((lane & ((32 >> kLog) - 1)) == 0) acc[warp][mine] = st;
  __syncthreads();
  // the CTA's statistics of row n, by a warp
  for (int n = warp; n < NT; n += W) {
    Stats all = {kNoTop, 0.f, 0.f};
    for (int i = lane; i < W * R; i += 32) all.add(acc[i / R][i % R * NT + n], c2);
    all.add_lanes(c2);
    const int64_t at = (int64_t)blockIdx.x * NT + n;
    if (lane == 0 && in_range(at, w.part_size)) w.part[at] = make_float4(all.top, all.s, all.t, 0.f);
  }
}

// d_hidden where its sum was split: the splits' sums in order, rounded once.
// One thread four columns of a part.
template <class ST>
__global__ void __launch_bounds__(kJoinThreads)
    head_dh_out_kernel(HeadArgs a, HeadView w, int64_t Dh, int64_t plane, int splits, bool vec) {
  pdl_trigger();
  pdl_wait();
  const int groups = (int)((a.D + 3) / 4);
  const int64_t total = (int64_t)w.count[0] * groups;
  for (int64_t t = (int64_t)blockIdx.x * kJoinThreads + threadIdx.x; t < total; t += (int64_t)gridDim.x * kJoinThreads) {
    const int64_t b = t / groups, c = (t - b * groups) * 4;
    const float* src = w.dh + b * Dh + c;
    const int64_t to = w.rows[b] * a.D + c;
    if (!span_in_range(b * Dh + c, (splits - 1) * plane + 4, w.dh_size) ||
        !span_in_range(to, min((int64_t)4, a.D - c), a.N * a.D))
      continue;
    float4 v = *reinterpret_cast<const float4*>(src);
    for (int k0 = 1; k0 < splits; k0 += 8) {
      float4 q[8];
#pragma unroll
      for (int u = 0; u < 8; ++u)
        q[u] = k0 + u < splits ? *reinterpret_cast<const float4*>(src + (k0 + u) * plane) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int u = 0; u < 8; ++u) v.x += q[u].x, v.y += q[u].y, v.z += q[u].z, v.w += q[u].w;
    }
    const float f[4] = {v.x, v.y, v.z, v.w};
    if (vec) {
      Stor<ST>::st4(a.d_hidden, to, f);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (c + i < a.D) Stor<ST>::st(a.d_hidden, to + i, f[i]);
    }
  }
}

// ---------------------------------------------------------------------------
TcTerms terms_of(int planes) {
  TcTerms t = {};
  if (planes == 1) {
    t.n = 1;
    return t;
  }
  const unsigned char a[6] = {0, 2, 1, 0, 1, 0}, b[6] = {2, 0, 1, 1, 0, 0};
  t.n = 6;
  std::copy(a, a + 6, t.a);
  std::copy(b, b + 6, t.b);
  return t;
}

// Rows that head_few_kernel takes, if their float32 copies fit two CTAs' shared
// memory an SM: bfloat16 up to 4 (32768 x 1024: 1 row 25 against 36 us on the
// tensor cores, 4 rows 35 against 33, 8 rows 54 against 32), float32, which
// the tensor cores take as planes that have to be packed first, up to 16 (87
// against 137 us).
bool few(int64_t N, int64_t D, bool bf16_io) {
  const int64_t nt = N <= 1 ? 1 : N <= 2 ? 2 : N <= 4 ? 4 : N <= 8 ? 8 : 16;
  return N <= (bf16_io ? 4 : 16) && (size_t)(nt * round_up(D, 4) * 4) <= kFewSmem;
}
int64_t tiles_of(const TcShape& s) { return div_up(s.m, kTcM) * div_up(s.n, kTcN) * s.splits; }

template <class Job1, class Job2>
cudaError_t launch_product(const Job1& j1, const Job2& j2, int64_t tiles, int sm_count, cudaStream_t st, bool blocks) {
  void (*const kernel)(const Job1, const Job2) = tc_product_kernel<Job1, Job2>;
  static std::atomic<uint64_t> allowed;
  cudaError_t e = allow_smem(kernel, kTcSmemBlocks, allowed);
  if (e != cudaSuccess) return e;
  if (kTcShares<Job1, Job2>) {
    // the warpgroups' register shares are taken from the launch's registers:
    // a kernel built with fewer would wait for the rest for ever
    static const bool enough = [&] {
      cudaFuncAttributes f;
      return cudaFuncGetAttributes(&f, kernel) == cudaSuccess &&
             f.numRegs * kTcThreads >= 32 * (kTcEpiWarps * kTcEpiRegs + 4 * kTcIssueRegs);
    }();
    if (!enough) return cudaErrorInvalidConfiguration;
  }
  return launch_pdl(kernel, 2 * std::min<int64_t>(tiles, sm_count / 2), kTcThreads, blocks ? kTcSmemBlocks : kTcSmem, st, j1,
                    j2);
}
template <class Job>
cudaError_t launch_product(const Job& j, int sm_count, cudaStream_t st, bool blocks = false) {
  return launch_product(j, TcNoJob{}, tiles_of(j.s), sm_count, st, blocks);
}

// Whether two products run faster dealt out together than one after the
// other: stages of the busiest cluster either way (the first product's tiles
// take k1 stages, the second's k2), a launch costing as much as kLaunchStages.
constexpr int64_t kLaunchStages = 24;
bool together(int64_t tiles1, int64_t k1, int64_t tiles2, int64_t k2, int64_t clusters) {
  const int64_t apart = div_up(tiles1, clusters) * k1 + div_up(tiles2, clusters) * k2 + kLaunchStages;
  int64_t most = 0;
  for (int64_t c = 0; c < clusters; ++c) {
    const int64_t n1 = c < tiles1 ? div_up(tiles1 - c, clusters) : 0;
    const int64_t n = c < tiles1 + tiles2 ? div_up(tiles1 + tiles2 - c, clusters) : 0;
    most = std::max(most, n1 * k1 + (n - n1) * k2);
  }
  return most <= apart;
}

// rows of A walked together: as many as keep their `width` values in L2
int band_of(int64_t width, int planes) {
  return (int)std::max<int64_t>(1, kBandBytes / (2 * planes * kTcM * std::max<int64_t>(width, 1)));
}

// a weight that the copies read in place
bool in_place(const HeadArgs& a) {
  return a.bf16_io && ((uintptr_t)a.weight & 15) == 0 && a.weight_stride % 8 == 0;
}

// Stages summed by the tensor cores alone (tc.cuh).
//
// Statistics: 512 values of k.  The error grows with the group and not with the
// width: 512 x 1024 to 8192 x 4001, bfloat16, log-probabilities 1.8e-7 to 2.1e-7
// off in groups of 512 (a plain float32 form 1.6e-7 to 6.1e-7), 3.9e-7 to 4.3e-7 in
// groups of 1024, which take 3 to 5% less time.  float32 operands take 128, and
// so does their dz, whose relative error is the gradients' (of the leading
// product only: 2 to 4% of the time; gradients at 2 x 4000 x 20000 4.1e-7 off
// instead of 1.9e-6).  Their gradients' sums take 512.
//
// bfloat16 gradients: 4096 terms, over rows or tokens of which there may be
// millions.  A sum of one sign stays within 3e-5, a hundredth of the result's
// rounding (unbounded, d_weight of 3 million such rows came out 1.8% too small).
// The logits of their dz: an error in the exponent of p has to stay well below
// dz's own rounding, 2^-9.  In groups of 1024 a logit of 16 of one sign is 1e-4 off
// (in one sum 4e-4 at 4096 columns, 0.5% at 65536); the whole gradient takes 2%
// longer for them (2048 x 4096 x 16384: 487 us, in one sum 478).
constexpr int kLogitsGroup = 8, kLogitsGroupF32 = 2, kGradGroupBf16 = 64, kDzGroupBf16 = 16;

// f(the group), or f(0) where no sum is of more than ONE steps: the whole sum
// in one accumulator, worked on straight from TMEM (tc.cuh).  The bfloat16
// gradients take up to 128 steps that way, 8192 terms, at most 5e-5 off
// (128 x 4096 x 32768: 201 us; in groups of 64 219).  float32 products are of six
// terms, of which the leading one has sums of its own.
template <class ST, int GROUP, int ONE, class F>
cudaError_t with_group(int64_t steps, F&& f) {
  if constexpr (Stor<ST>::kBytes == 2) {
    if (steps <= ONE) return f(std::integral_constant<int, 0>{});
  }
  return f(std::integral_constant<int, GROUP>{});
}

template <class ST>
struct HeadRun {
  static constexpr bool kF32 = Stor<ST>::kBytes == 4;
  static constexpr int kGradGroup = kF32 ? kLogitsGroup : kGradGroupBf16, kDzGroup = kF32 ? kLogitsGroupF32 : kDzGroupBf16,
                       kStatsGroup = kF32 ? kLogitsGroupF32 : kLogitsGroup;
  const HeadArgs& a;
  const HeadPlan p;
  const HeadView w;
  const int sm;
  const cudaStream_t s;
  const TcTerms terms;
  // the parts' rows as a K-major and an MN-major operand: packed, and where
  // they lie (for when all rows take part)
  CUtensorMap hidden_k, hidden_mn, in_place_k, in_place_mn;
  bool hidden_ok = false;  // the copies can read the hidden rows where they lie

  HeadRun(const HeadArgs& args, const HeadPlan& plan, int sm_count, cudaStream_t st)
      : a(args), p(plan), w(plan, args.ws), sm(sm_count), s(st), terms(terms_of(plan.planes)) {}

  cudaError_t rows() {
    if (!encode_matrix_map(&hidden_k, w.hidden, p.Dp, p.Np, p.planes, p.Dp, p.Np * p.Dp, kTcRows) ||
        !encode_matrix_map(&hidden_mn, w.hidden, p.Dp, p.Np, p.planes, p.Dp, p.Np * p.Dp, kTcK))
      return cudaErrorNotSupported;
    hidden_ok = a.bf16_io && ((uintptr_t)a.hidden & 15) == 0 && a.hidden_stride % 8 == 0;
    in_place_k = hidden_k, in_place_mn = hidden_mn;
    if (hidden_ok &&
        (!encode_matrix_map(&in_place_k, a.hidden, a.D, a.N, 1, a.hidden_stride, a.N * a.hidden_stride, kTcRows) ||
         !encode_matrix_map(&in_place_mn, a.hidden, a.D, a.N, 1, a.hidden_stride, a.N * a.hidden_stride, kTcK)))
      return cudaErrorNotSupported;
    const int64_t rows_per_cta = std::max<int64_t>(2, div_up(a.N, 4 * (int64_t)sm));
    return launch_pdl(head_begin_kernel<ST>, div_up(a.N, rows_per_cta), kPackThreads, 0, s, a, w, rows_per_cta, p.Dp,
                      p.Np, a.d_logp != nullptr, hidden_ok);
  }
  // the weight's rows from v0 on, packed where the copies cannot read them in place
  cudaError_t weight_piece(int64_t v0, int64_t len) {
    if (!p.packed) return cudaSuccess;
    PackArgs k = {};
    k.src = a.weight; k.size = (a.V - 1) * a.weight_stride + a.D; k.r0 = v0; k.rows = len; k.width = a.D; k.stride = a.weight_stride;
    k.dst = w.weight; k.pitch = p.Dp; k.dst_rows = p.pitch; k.dst_size = w.weight_size;
    return launch_pdl(head_pack_kernel<ST>, std::min<int64_t>(div_up(len * (p.Dp / 8), 4 * kPackThreads), 8 * (int64_t)sm), kPackThreads, 0, s, k);
  }
  bool weight_map(CUtensorMap* m, int64_t len, int box_rows) {
    if (p.packed) return encode_matrix_map(m, w.weight, p.Dp, len, p.planes, p.Dp, p.pitch * p.Dp, box_rows);
    return encode_matrix_map(m, a.weight, a.D, a.V, 1, a.weight_stride, a.V * a.weight_stride, box_rows);
  }
  TcShape logits_shape(int64_t v0, int64_t len) {
    TcShape t = {};
    t.count = w.count; t.count_axis = 1;
    t.m = (int)a.N; t.n = (int)len; t.k = (int)a.D;
    t.b_n0 = p.packed ? 0 : (int)v0;
    t.other = hidden_ok ? 1 : 0; t.full = (int)a.N;
    t.splits = 1; t.band = band_of(p.Dp, p.planes); t.terms = terms;
    return t;
  }

  cudaError_t forward() {
    cudaError_t e = rows();
    const float c2 = a.inv_temperature * kLog2e;
    for (int64_t v0 = 0; v0 < a.V && e == cudaSuccess; v0 += p.piece) {
      const int64_t len = std::min(p.piece, a.V - v0);
      e = weight_piece(v0, len);
      if (e != cudaSuccess) break;
      CUtensorMap wk;
      if (!weight_map(&wk, len, kTcN / 2)) return cudaErrorNotSupported;
      const StatsEpi epi{w.part, w.taken, w.tok, p.Np, div_up(a.V, kTcN) * 2, (int)v0, (int)(v0 + len), c2};
      const TcShape t = logits_shape(v0, len);
      e = with_group<ST, kStatsGroup, kStatsGroup>(div_up(a.D, kTcK), [&](auto g) {
        return launch_product(TcJob<false, false, g.value, StatsEpi>{hidden_k, wk, in_place_k, t, epi}, sm, s);
      });
    }
    return e == cudaSuccess ? join(div_up(a.V, kTcN) * 2, p.Np, false) : e;
  }
  // (at few parts, few CTAs would run the whole column of pieces each)
  cudaError_t join(int64_t pieces, int64_t pitch, bool identity) {
    const float c2 = a.inv_temperature * kLog2e;
    if (identity || a.N <= 256)
      return launch_pdl(head_join_few_kernel, a.N, kJoinThreads, 0, s, a, w, pieces, pitch, c2, identity);
    return launch_pdl(head_join_kernel, div_up(a.N, 32), 32 * kJoinWarps, 0, s, a, w, pieces, pitch, c2);
  }

  // 16 loads of a lane in flight: 4 tokens at a time, or 8 of up to 64 vectors
  // (512 x 131072 bfloat16); 16 rows hold 32 sums at 2 tokens
  template <int VE, int NT>
  cudaError_t few_rows() {
    if (VE > 1 && NT <= 2 && a.D / VE <= 64) return few_launch<VE, NT, (NT <= 2 ? 8 : 4)>();
    return few_launch<VE, NT, (NT > 8 ? 2 : 4)>();
  }
  template <int VE, int NT, int R>
  cudaError_t few_launch() {
    const auto kernel = head_few_kernel<ST, VE, NT, R>;
    const int64_t Ds = round_up(a.D, 4);
    const size_t smem = (size_t)NT * Ds * 4;
    static std::atomic<uint64_t> allowed;
    cudaError_t e = allow_smem(kernel, kFewSmem, allowed);
    if (e != cudaSuccess) return e;
    const int64_t grid = std::min(div_up(a.V, R * (kFewThreads / 32)), few_pieces(sm));
    e = launch_pdl(kernel, grid, kFewThreads, smem, s, a, w, Ds, a.inv_temperature * kLog2e);
    return e == cudaSuccess ? join(grid, NT, true) : e;
  }
  template <int VE>
  cudaError_t few_rows() {
    if (a.N <= 1) return few_rows<VE, 1>();
    if (a.N <= 2) return few_rows<VE, 2>();
    if constexpr (Stor<ST>::kBytes == 2) return few_rows<VE, 4>();
    else return a.N <= 4 ? few_rows<VE, 4>() : a.N <= 8 ? few_rows<VE, 8>() : few_rows<VE, 16>();
  }
  cudaError_t forward_few() {
    constexpr int VE = 16 / Stor<ST>::kBytes;
    const bool vec = ((uintptr_t)a.weight & 15) == 0 && (a.weight_stride * Stor<ST>::kBytes) % 16 == 0 && a.D % VE == 0;
    return vec ? few_rows<VE>() : few_rows<1>();
  }

  // what the starts of an output's rows are multiples of (32, 16, or neither: 1)
  int align_of(const float* out) const {
    const uintptr_t rows = (uintptr_t)out | (uintptr_t)(a.D * Stor<ST>::kBytes);
    return rows % 32 == 0 ? 32 : rows % 16 == 0 ? 16 : 1;
  }

  cudaError_t backward() {
    cudaError_t e = rows();
    // (with two values: planes of kTcRows rows in one tile)
    const int64_t dz_rows = p.two_dz ? kTcRows : p.Np, dz_plane = dz_rows * p.pitch, dh_plane = p.Np * p.Dh;
    const int dz_planes = p.two_dz ? 2 : p.planes;
    // d_hidden's sum takes the second values as rows of their own where the
    // splits' sums are joined anyway, else as a second term; d_weight as a
    // second term
    const bool halves = p.two_dz && p.splits > 1;
    TcTerms dz_terms = terms;
    if (p.two_dz) dz_terms.n = 2, dz_terms.a[0] = 1, dz_terms.a[1] = 0;
    for (int64_t v0 = 0; v0 < a.V && e == cudaSuccess; v0 += p.piece) {
      const int64_t len = std::min(p.piece, a.V - v0);
      e = weight_piece(v0, len);
      if (e != cudaSuccess) break;
      CUtensorMap wk, wmn, dz_k, dz_mn;
      if (!weight_map(&wk, len, kTcN / 2) || !weight_map(&wmn, len, kTcK) ||
          !encode_matrix_map(&dz_k, w.dz, len, halves ? p.Np : dz_rows, halves ? 1 : dz_planes, p.pitch, dz_plane, kTcRows) ||
          !encode_matrix_map(&dz_mn, w.dz, len, dz_rows, dz_planes, p.pitch, dz_plane, kTcK))
        return cudaErrorNotSupported;
      using Dz = DzEpi<Stor<ST>::kBytes == 2 ? 1 : 3>;
      const Dz dz{w.dz, p.pitch, dz_plane, dz_planes * dz_plane, w.info, w.tok, (int)v0, a.inv_temperature, p.two_dz};
      e = with_group<ST, kDzGroup, kDzGroup>(div_up(a.D, kTcK), [&](auto g) {
        return launch_product(TcJob<false, false, g.value, Dz>{hidden_k, wk, in_place_k, logits_shape(v0, len), dz}, sm, s);
      });
      if (e != cudaSuccess) break;
      // d_hidden's sum over this piece's tokens, and its tokens' d_weight
      TcShape sh = {}, sw = {};
      sh.count = sw.count = w.count;
      sw.terms = dz_terms;
      sh.terms = halves ? terms : dz_terms;
      sh.band = sw.band = 16;
      sh.count_axis = halves ? 0 : 1;
      sh.m = halves ? kTcM : (int)a.N; sh.n = (int)a.D; sh.k = (int)len;
      sh.b_k0 = p.packed ? 0 : (int)v0;
      sh.splits = p.splits;
      sw.count_axis = 2;
      sw.m = (int)len; sw.n = (int)a.D; sw.k = (int)a.N;
      sw.splits = 1;
      sw.other = hidden_ok ? 2 : 0; sw.full = (int)a.N;
      const DhEpi<ST> eh{w.dh, p.Dh, dh_plane, (halves ? 2 : 1) * p.splits * dh_plane, v0 == 0, p.splits == 1 && v0 + len == a.V,
                         a.d_hidden, w.rows, a.N, a.D, align_of(a.d_hidden), halves};
      const OutEpi<ST> ew{a.d_weight, v0, a.D, a.V, align_of(a.d_weight)};
      const int64_t kh = div_up(div_up(len, kTcK), p.splits) * sh.terms.n, kw = div_up(a.N, kTcK) * sw.terms.n;
      const bool rows_h = eh.align < 16, rows_w = ew.align < 16;
      const auto hidden_grad = [&](auto g) { return TcJob<false, true, g.value, DhEpi<ST>>{dz_k, wmn, wmn, sh, eh}; };
      const auto weight_grad = [&](auto g) { return TcJob<true, true, g.value, OutEpi<ST>>{dz_mn, hidden_mn, in_place_mn, sw, ew}; };
      if (a.d_hidden && a.d_weight && together(tiles_of(sh), kh, tiles_of(sw), kw, sm / 2)) {
        e = with_group<ST, kGradGroup, kTcLead>(kh, [&](auto g) {
          return with_group<ST, kGradGroup, kTcLead>(kw, [&](auto g2) {
            return launch_product(hidden_grad(g), weight_grad(g2), tiles_of(sh) + tiles_of(sw), sm, s, rows_h || rows_w);
          });
        });
      } else {
        if (a.d_hidden)
          e = with_group<ST, kGradGroup, kTcLead>(kh, [&](auto g) { return launch_product(hidden_grad(g), sm, s, rows_h); });
        if (e == cudaSuccess && a.d_weight)
          e = with_group<ST, kGradGroup, kTcLead>(kw, [&](auto g) { return launch_product(weight_grad(g), sm, s, rows_w); });
      }
    }
    if (e == cudaSuccess && a.d_hidden && p.splits > 1) {
      const bool vec = a.D % 4 == 0 && ((uintptr_t)a.d_hidden & 15) == 0;
      const int64_t grid = std::min<int64_t>(div_up(a.N * div_up(a.D, 4), kJoinThreads), 16 * (int64_t)sm);
      e = launch_pdl(head_dh_out_kernel<ST>, grid, kJoinThreads, 0, s, a, w, p.Dh, dh_plane, (halves ? 2 : 1) * p.splits, vec);
    }
    return e;
  }
};

}  // namespace

size_t head_workspace(int64_t N, int64_t D, int64_t V, bool bf16_io, bool backward, int sm_count) {
  // the call reads the weight in place or packs it by its alignment, which
  // the query cannot see: the larger of the two needs
  const size_t pk = plan_head(N, D, V, bf16_io, backward, true, sm_count).bytes;
  return bf16_io ? std::max(pk, plan_head(N, D, V, bf16_io, backward, false, sm_count).bytes) : pk;
}

cudaError_t run_token_logprob(const HeadArgs& a, int sm_count, cudaStream_t s) {
  const HeadPlan p = plan_head(a.N, a.D, a.V, a.bf16_io, false, !in_place(a), sm_count);
  if (few(a.N, a.D, a.bf16_io)) return a.bf16_io ? HeadRun<bf16>(a, p, sm_count, s).forward_few() : HeadRun<float>(a, p, sm_count, s).forward_few();
  return a.bf16_io ? HeadRun<bf16>(a, p, sm_count, s).forward() : HeadRun<float>(a, p, sm_count, s).forward();
}

cudaError_t run_token_logprob_backward(const HeadArgs& a, int sm_count, cudaStream_t s) {
  const HeadPlan p = plan_head(a.N, a.D, a.V, a.bf16_io, true, !in_place(a), sm_count);
  return a.bf16_io ? HeadRun<bf16>(a, p, sm_count, s).backward() : HeadRun<float>(a, p, sm_count, s).backward();
}

cudaError_t status_head(unsigned int* word, bool clear) { return unit_status(word, clear); }

}  // namespace rlca
