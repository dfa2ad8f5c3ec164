// Token log-probabilities and entropies of a policy head, and their gradient.
//
// Three matrix products carry the work, all on the tensor cores (tc.cuh):
// the logits' tiles, whose epilogue keeps per half tile of 128 tokens a
// running (max, sum e^z, sum e^z z) -- or, in the gradient, turns the logits
// into dz --, and the two products of dz with the weight and with the hidden
// rows.  The logits exist in TMEM only; dz exists for one piece of the
// vocabulary at a time.
#include <algorithm>

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
constexpr int64_t kPieceBytes = int64_t(256) << 20;  // dz of one piece of the vocabulary
constexpr int64_t kPackBytes = int64_t(128) << 20;   // packed weight of one piece
constexpr int64_t kSplitBytes = int64_t(64) << 20;   // d_hidden's partial sums beyond the first
constexpr int64_t kBandBytes = int64_t(48) << 20;    // hidden rows walked together (well inside L2)
constexpr float kLog2e = 1.4426950408889634f;

constexpr int64_t round_up(int64_t a, int64_t b) { return div_up(a, b) * b; }

struct HeadPlan {
  int planes;       // bfloat16 planes of an operand
  bool packed;      // the weight is packed
  int64_t Np;       // parts, rounded up to whole tiles
  int64_t Dp;       // pitch of packed rows
  int64_t Dh;       // pitch of d_hidden's float32 sums
  int64_t piece;    // tokens per piece (whole tiles unless it is the whole vocabulary)
  int64_t pitch;    // of dz and of the column of partial statistics: piece in whole tiles
  int row_tiles, d_tiles, splits;
  size_t count, rows, tok, info, hidden, weight, part, taken, dz, dh;  // byte offsets
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
  const int64_t tiles = div_up(V, kTcN);
  int64_t piece_tiles = tiles;
  if (packed) piece_tiles = std::min(piece_tiles, std::max<int64_t>(1, kPackBytes / (2 * p.planes * p.Dp * kTcN)));
  if (backward) piece_tiles = std::min(piece_tiles, std::max<int64_t>(1, kPieceBytes / (2 * p.planes * p.Np * kTcN)));
  p.pitch = piece_tiles * kTcN;
  p.piece = std::min(p.pitch, V);
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
    // then split until the tiles fill the SMs
    const int64_t out_tiles = (int64_t)p.row_tiles * p.d_tiles, out_bytes = p.Np * p.Dh * 4;
    p.splits = (int)std::max<int64_t>(
        1, std::min({(int64_t)sm_count / out_tiles, 1 + kSplitBytes / out_bytes, div_up(p.piece, kTcK)}));
    p.dh = take((size_t)p.splits * out_bytes);
  } else {
    p.part = take((size_t)tiles * 2 * p.Np * sizeof(float4));
    p.taken = take((size_t)p.Np * 4);
  }
  p.bytes = at;
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
  HeadView(const HeadPlan& p, void* ws) {
    unsigned char* b = static_cast<unsigned char*>(ws);
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
  }
};

// Numbers the rows that take part, in order (one CTA: a running count over
// blocks of rows), and clears the results of those that do not.
constexpr int kRowsThreads = 1024;
__global__ void __launch_bounds__(kRowsThreads) head_rows_kernel(HeadArgs a, HeadView w) {
  pdl_trigger();
  pdl_wait();
  __shared__ int warps[32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int base = 0;
  for (int64_t i0 = 0; i0 < a.N; i0 += kRowsThreads) {
    const int64_t i = i0 + threadIdx.x;
    const int tok = i < a.N ? a.tokens[i] : -1;
    const bool on = tok >= 0 && tok < a.V;
    const unsigned vote = __ballot_sync(0xffffffffu, on);
    if (lane == 0) warps[warp] = __popc(vote);
    __syncthreads();
    int before = base, total = base;
    for (int k = 0; k < 32; ++k) {
      before += k < warp ? warps[k] : 0;
      total += warps[k];
    }
    if (on) {
      const int at = before + __popc(vote & ((1u << lane) - 1u));
      w.rows[at] = (int)i;
      w.tok[at] = tok;
      if (a.d_logp != nullptr)
        w.info[at] = make_float4(a.d_logp[i], a.d_entropy ? a.d_entropy[i] : 0.f, a.in_lse[i],
                                 a.d_entropy ? a.in_entropy[i] : 0.f);
    }
    if (!on && i < a.N && a.logp != nullptr) {
      a.logp[i] = 0.f;
      a.lse[i] = 0.f;
      if (a.entropy) a.entropy[i] = 0.f;
    }
    base = total;
    __syncthreads();
  }
  if (threadIdx.x == 0) w.count[0] = base;
}

// ---------------------------------------------------------------------------
// Packing: rows of 8-element groups, zeros past the width and from row
// `valid` to the next whole tile.
// ---------------------------------------------------------------------------
constexpr int kPackThreads = 256;

struct PackArgs {
  const float* src;  // element type by the kernel
  const int* map;    // row of src, or null: r0 + r
  const int* valid;  // rows that exist, or null: `rows`
  int64_t r0, rows, width, stride;
  void* dst;  // planes x [dst_rows, pitch]
  int64_t pitch, dst_rows;
};

// v as the sum of three bfloat16 values, each the rounding of the remainder:
// exact to 24 bits (the remainders are exact in float32)
__device__ __forceinline__ void split3(float v, float& hi, float& mid, float& lo) {
  hi = __bfloat162float(__float2bfloat16_rn(v));
  const float r = v - hi;
  mid = __bfloat162float(__float2bfloat16_rn(r));
  lo = r - mid;
}

template <class ST>
__global__ void __launch_bounds__(kPackThreads) head_pack_kernel(PackArgs a) {
  pdl_trigger();
  pdl_wait();
  const int64_t groups = a.pitch / 8;
  const int64_t valid = a.valid ? min((int64_t)*a.valid, a.rows) : a.rows;
  const int64_t rows = min(a.dst_rows, (valid + kTcM - 1) / kTcM * kTcM);
  const bool vec = ((uintptr_t)a.src & 15) == 0 && (a.stride * Stor<ST>::kBytes) % 16 == 0;
  for (int64_t t = (int64_t)blockIdx.x * kPackThreads + threadIdx.x; t < rows * groups;
       t += (int64_t)gridDim.x * kPackThreads) {
    const int64_t r = t / groups, c = (t % groups) * 8;
    float v[8];
    if (r < valid && vec && c + 8 <= a.width) {
      const int64_t at = (a.map ? (int64_t)a.map[r] : a.r0 + r) * a.stride + c;
      if constexpr (Stor<ST>::kBytes == 2) {
        Stor<ST>::ld8(a.src, at, true, v);
      } else {
        float (&lo)[4] = reinterpret_cast<float (&)[4]>(v[0]);
        float (&hi)[4] = reinterpret_cast<float (&)[4]>(v[4]);
        Stor<ST>::ld4(a.src, at, true, lo);
        Stor<ST>::ld4(a.src, at + 4, true, hi);
      }
    } else {
      const int64_t at = r < valid ? (a.map ? (int64_t)a.map[r] : a.r0 + r) * a.stride : 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = r < valid && c + i < a.width ? Stor<ST>::ld(a.src, at + c + i) : 0.f;
    }
    float* dst = static_cast<float*>(a.dst);  // Stor<bf16> counts in elements of two bytes
    const int64_t to = r * a.pitch + c;
    if constexpr (Stor<ST>::kBytes == 2) {
      Stor<bf16>::st8(dst, to, v);
    } else {
      float h[8], m[8], l[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) split3(v[i], h[i], m[i], l[i]);
      const int64_t plane = a.dst_rows * a.pitch;
      Stor<bf16>::st8(dst, to, h);
      Stor<bf16>::st8(dst, to + plane, m);
      Stor<bf16>::st8(dst, to + 2 * plane, l);
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

// part[half tile][part] = (max of acc, sum e, sum e acc) with
// e = 2^(c2 (acc - max)), c2 = log2(e) / temperature
struct StatsEpi {
  float4* part;
  float* taken;
  const int* tok;
  int64_t Np;
  int v0, v_end;  // tokens of this piece
  float c2;

  struct State {
    float top, s, t;
    int m, at, col0;
    bool live;
  };
  __device__ __forceinline__ void begin(State& st, const TcWalk& w, const TcTile&, int row, int col0) const {
    st.m = row;
    st.live = row < w.m;
    st.at = st.live ? tok[row] - v0 : -1;
    st.col0 = col0;
    st.top = -INFINITY;
    st.s = st.t = 0.f;
  }
  __device__ __forceinline__ void chunk(State& st, int col, float (&v)[32]) const {
    const int n = v_end - v0 - col;  // columns that exist
    if (n <= 0) return;
    if (n < 32) {
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = i < n ? v[i] : -3.402823466e38f;
    }
    float top = v[0];
#pragma unroll
    for (int i = 1; i < 32; ++i) top = fmaxf(top, v[i]);
    top = fmaxf(top, st.top);
    // the first chunk: 2^-inf = 0 drops the empty sums (kept off inf - inf)
    const float f = st.top == -INFINITY ? 0.f : exp2_approx((st.top - top) * c2);
    float s = st.s * f, t = st.t * f;
    const float off = -top * c2;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      const float e = exp2_approx(fmaf(v[i], c2, off));
      s += e;
      t = fmaf(e, v[i], t);
    }
    st.top = top;
    st.s = s;
    st.t = t;
    const int k = st.at - col;
    if (k >= 0 && k < 32) {
      float z = v[0];
#pragma unroll
      for (int i = 1; i < 32; ++i) z = i == k ? v[i] : z;
      taken[st.m] = z;
    }
  }
  __device__ __forceinline__ void end(State& st) const {
    if (st.live) part[(int64_t)((v0 + st.col0) / (kTcN / 2)) * Np + st.m] = make_float4(st.top, st.s, st.t, 0.f);
  }
};

// eight values as bfloat16 at p (16-byte aligned)
__device__ __forceinline__ void store8(uint16_t* p, const float* v) {
  Stor<bf16>::st8(reinterpret_cast<float*>(p), 0, v);
}

// dz = p (a0 + a1 acc), plus g / temperature for the token taken, as one
// bfloat16 (rounded once: the two products that read it run on bfloat16) or
// as three planes
template <int PLANES>
struct DzEpi {
  uint16_t* dz;
  int64_t pitch, plane;
  const float4* info;
  const int* tok;
  int v0;
  float inv_t;

  struct State {
    float lse2, a0, a1, g;
    int at;
    bool live;
    uint16_t* row;
  };
  __device__ __forceinline__ void begin(State& st, const TcWalk& w, const TcTile&, int row, int) const {
    st.live = row < w.m;
    st.row = dz + (int64_t)row * pitch;
    st.at = -1;
    st.lse2 = st.a0 = st.a1 = st.g = 0.f;
    if (st.live) {
      const float4 f = info[row];
      st.at = tok[row] - v0;
      st.g = f.x * inv_t;
      st.a0 = -(f.x + f.y * (f.w - f.z)) * inv_t;
      st.a1 = -f.y * inv_t * inv_t;
      st.lse2 = -f.z * kLog2e;
    }
  }
  __device__ __forceinline__ void chunk(State& st, int col, float (&v)[32]) const {
    const float c2 = inv_t * kLog2e;
    const int k = st.at - col;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      const float p = exp2_approx(fmaf(v[i], c2, st.lse2));
      v[i] = st.live ? p * fmaf(st.a1, v[i], st.a0) : 0.f;
    }
    if (k >= 0 && k < 32) {
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] += i == k ? st.g : 0.f;
    }
    if constexpr (PLANES == 1) {
#pragma unroll
      for (int i = 0; i < 32; i += 8) store8(st.row + col + i, v + i);
    } else {
#pragma unroll
      for (int i = 0; i < 32; i += 8) {
        float h[8], m[8], l[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) split3(v[i + j], h[j], m[j], l[j]);
        store8(st.row + col + i, h);
        store8(st.row + plane + col + i, m);
        store8(st.row + 2 * plane + col + i, l);
      }
    }
  }
  __device__ __forceinline__ void end(State&) const {}
};

// float32 sums, set by the first piece and added to by the others
struct SumEpi {
  float* out;  // splits x [rows, pitch]
  int64_t pitch, plane;
  bool add;

  struct State {
    float* row;
    bool live;
  };
  __device__ __forceinline__ void begin(State& st, const TcWalk& w, const TcTile& t, int row, int) const {
    st.live = row < w.m;
    st.row = out + t.split * plane + (int64_t)row * pitch;
  }
  __device__ __forceinline__ void chunk(State& st, int col, float (&v)[32]) const {
    if (!st.live || col >= pitch) return;
#pragma unroll
    for (int i = 0; i < 32; i += 4) {
      float4* p = reinterpret_cast<float4*>(st.row + col + i);
      float4 r = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
      if (add) {
        const float4 o = *p;
        r.x += o.x, r.y += o.y, r.z += o.z, r.w += o.w;
      }
      *p = r;
    }
  }
  __device__ __forceinline__ void end(State&) const {}
};

// the result, rounded once
template <class ST>
struct OutEpi {
  float* out;  // [.., width], element type ST
  int64_t row0, width;
  bool vec;  // rows start on 16-byte boundaries

  struct State {
    int64_t at;
    bool live;
  };
  __device__ __forceinline__ void begin(State& st, const TcWalk& w, const TcTile&, int row, int) const {
    st.live = row < w.m;
    st.at = (row0 + row) * width;
  }
  __device__ __forceinline__ void chunk(State& st, int col, float (&v)[32]) const {
    if (!st.live) return;
    if (vec && col + 32 <= width) {
      if constexpr (Stor<ST>::kBytes == 2) {
#pragma unroll
        for (int i = 0; i < 32; i += 8) Stor<ST>::st8(out, st.at + col + i, v + i);
      } else {
#pragma unroll
        for (int i = 0; i < 32; i += 4) Stor<ST>::st4(out, st.at + col + i, v + i);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (col + i < width) Stor<ST>::st(out, st.at + col + i, v[i]);
    }
  }
  __device__ __forceinline__ void end(State&) const {}
};

// ---------------------------------------------------------------------------
constexpr int kJoinThreads = 256;

// joins a part's half tiles, one warp a part
__global__ void __launch_bounds__(kJoinThreads)
    head_join_kernel(HeadArgs a, HeadView w, int64_t halves, int64_t Np, float c2) {
  pdl_trigger();
  pdl_wait();
  const int64_t m = (int64_t)blockIdx.x * (kJoinThreads / 32) + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (m >= w.count[0]) return;
  float top = -INFINITY;
  for (int64_t k = lane; k < halves; k += 32) top = fmaxf(top, w.part[k * Np + m].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  float s = 0.f, t = 0.f;
  for (int64_t k = lane; k < halves; k += 32) {
    const float4 p = w.part[k * Np + m];
    const float f = exp2_approx((p.x - top) * c2);
    s += p.y * f;
    t += p.z * f;
  }
  s = warp_sum(s);
  t = warp_sum(t);
  if (lane != 0) return;
  const float inv_t = a.inv_temperature;
  const float log_s = logf(s);
  const int64_t i = w.rows[m];
  a.lse[i] = fmaf(top, inv_t, log_s);
  a.logp[i] = fmaf(w.taken[m] - top, inv_t, -log_s);
  if (a.entropy) a.entropy[i] = fmaf(top - t / s, inv_t, log_s);
}

// d_hidden: the parts' rows rounded once, zeros for rows that take no part
template <class ST>
__global__ void __launch_bounds__(kJoinThreads) head_dh_out_kernel(HeadArgs a, HeadView w, int64_t Dh, int64_t plane, int splits) {
  pdl_trigger();
  pdl_wait();
  const int64_t b = blockIdx.x;
  if (b < w.count[0]) {
    const int64_t row = w.rows[b];
    for (int64_t c = threadIdx.x; c < a.D; c += kJoinThreads) {
      float v = w.dh[b * Dh + c];
      for (int k = 1; k < splits; ++k) v += w.dh[k * plane + b * Dh + c];
      Stor<ST>::st(a.d_hidden, row * a.D + c, v);
    }
  }
  const int tok = a.tokens[b];
  if (tok < 0 || tok >= a.V)
    for (int64_t c = threadIdx.x; c < a.D; c += kJoinThreads) Stor<ST>::st(a.d_hidden, b * a.D + c, 0.f);
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

template <bool A_MN, bool B_MN, int GROUP, class Epi>
cudaError_t launch_product(const CUtensorMap& ma, const CUtensorMap& mb, const TcShape& s, const Epi& epi, int sm_count,
                           cudaStream_t st) {
  const auto kernel = tc_product_kernel<A_MN, B_MN, GROUP, Epi>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kTcSmem);
  if (e != cudaSuccess) return e;
  const int64_t tiles = div_up(s.m, kTcM) * div_up(s.n, kTcN) * s.splits;
  return launch_pdl(kernel, 2 * std::min<int64_t>(tiles, sm_count / 2), kTcThreads, kTcSmem, st, ma, mb, s, epi);
}

// rows of A walked together: as many as keep their `width` values in L2
int band_of(int64_t width, int planes) {
  return (int)std::max<int64_t>(1, kBandBytes / (2 * planes * kTcM * std::max<int64_t>(width, 1)));
}

// a weight that the copies read in place
bool in_place(const HeadArgs& a) {
  return a.bf16_io && ((uintptr_t)a.weight & 15) == 0 && a.weight_stride % 8 == 0;
}

// Stages summed by the tensor cores alone (tc.cuh): 512 values of k for
// results that leave in float32; the bfloat16 gradients' own rounding is
// larger than the whole sum's error.
constexpr int kLogitsGroup = 8;

template <class ST>
struct HeadRun {
  static constexpr int kGradGroup = Stor<ST>::kBytes == 4 ? kLogitsGroup : 0;
  const HeadArgs& a;
  const HeadPlan p;
  const HeadView w;
  const int sm;
  const cudaStream_t s;
  const TcTerms terms;
  CUtensorMap hidden_k, hidden_mn;  // the parts' rows as a K-major and an MN-major operand

  HeadRun(const HeadArgs& args, const HeadPlan& plan, int sm_count, cudaStream_t st)
      : a(args), p(plan), w(plan, args.ws), sm(sm_count), s(st), terms(terms_of(plan.planes)) {}

  cudaError_t rows() {
    if (!encode_matrix_map(&hidden_k, w.hidden, p.Dp, p.Np, p.planes, p.Dp, p.Np * p.Dp, kTcRows) ||
        !encode_matrix_map(&hidden_mn, w.hidden, p.Dp, p.Np, p.planes, p.Dp, p.Np * p.Dp, kTcK))
      return cudaErrorNotSupported;
    cudaError_t e = launch_pdl(head_rows_kernel, 1, kRowsThreads, 0, s, a, w);
    if (e != cudaSuccess) return e;
    PackArgs k = {};
    k.src = a.hidden; k.map = w.rows; k.valid = w.count; k.rows = a.N; k.width = a.D; k.stride = a.hidden_stride;
    k.dst = w.hidden; k.pitch = p.Dp; k.dst_rows = p.Np;
    return pack(k);
  }
  cudaError_t pack(const PackArgs& k) {
    const int64_t grid = std::min<int64_t>(div_up(k.dst_rows * (k.pitch / 8), kPackThreads), 8 * (int64_t)sm);
    return launch_pdl(head_pack_kernel<ST>, grid, kPackThreads, 0, s, k);
  }
  // the weight's rows from v0 on, as an operand with boxes of box_rows; rows and columns of it in *y0
  cudaError_t weight_piece(int64_t v0, int64_t len) {
    if (!p.packed) return cudaSuccess;
    PackArgs k = {};
    k.src = a.weight; k.r0 = v0; k.rows = len; k.width = a.D; k.stride = a.weight_stride;
    k.dst = w.weight; k.pitch = p.Dp; k.dst_rows = p.pitch;
    return pack(k);
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
      const StatsEpi epi{w.part, w.taken, w.tok, p.Np, (int)v0, (int)(v0 + len), c2};
      e = launch_product<false, false, kLogitsGroup>(hidden_k, wk, logits_shape(v0, len), epi, sm, s);
    }
    if (e == cudaSuccess)
      e = launch_pdl(head_join_kernel, div_up(a.N, kJoinThreads / 32), kJoinThreads, 0, s, a, w, div_up(a.V, kTcN) * 2,
                     p.Np, c2);
    return e;
  }

  cudaError_t backward() {
    cudaError_t e = rows();
    const int64_t dz_plane = p.Np * p.pitch, dh_plane = p.Np * p.Dh;
    for (int64_t v0 = 0; v0 < a.V && e == cudaSuccess; v0 += p.piece) {
      const int64_t len = std::min(p.piece, a.V - v0);
      e = weight_piece(v0, len);
      if (e != cudaSuccess) break;
      CUtensorMap wk, wmn, dz_k, dz_mn;
      if (!weight_map(&wk, len, kTcN / 2) || !weight_map(&wmn, len, kTcK) ||
          !encode_matrix_map(&dz_k, w.dz, len, p.Np, p.planes, p.pitch, dz_plane, kTcRows) ||
          !encode_matrix_map(&dz_mn, w.dz, len, p.Np, p.planes, p.pitch, dz_plane, kTcK))
        return cudaErrorNotSupported;
      if constexpr (Stor<ST>::kBytes == 2) {
        const DzEpi<1> epi{w.dz, p.pitch, dz_plane, w.info, w.tok, (int)v0, a.inv_temperature};
        e = launch_product<false, false, kGradGroup>(hidden_k, wk, logits_shape(v0, len), epi, sm, s);
      } else {
        const DzEpi<3> epi{w.dz, p.pitch, dz_plane, w.info, w.tok, (int)v0, a.inv_temperature};
        e = launch_product<false, false, kGradGroup>(hidden_k, wk, logits_shape(v0, len), epi, sm, s);
      }
      if (e == cudaSuccess && a.d_hidden) {
        TcShape t = {};
        t.count = w.count; t.count_axis = 1;
        t.m = (int)a.N; t.n = (int)a.D; t.k = (int)len;
        t.b_k0 = p.packed ? 0 : (int)v0;
        t.splits = p.splits; t.band = 16; t.terms = terms;
        e = launch_product<false, true, kGradGroup>(dz_k, wmn, t, SumEpi{w.dh, p.Dh, dh_plane, v0 > 0}, sm, s);
      }
      if (e == cudaSuccess && a.d_weight) {
        TcShape t = {};
        t.count = w.count; t.count_axis = 2;
        t.m = (int)len; t.n = (int)a.D; t.k = (int)a.N;
        t.splits = 1; t.band = 16; t.terms = terms;
        const bool vec = (a.D * Stor<ST>::kBytes) % 16 == 0 && ((uintptr_t)a.d_weight & 15) == 0;
        e = launch_product<true, true, kGradGroup>(dz_mn, hidden_mn, t, OutEpi<ST>{a.d_weight, v0, a.D, vec}, sm, s);
      }
    }
    if (e == cudaSuccess && a.d_hidden)
      e = launch_pdl(head_dh_out_kernel<ST>, a.N, kJoinThreads, 0, s, a, w, p.Dh, dh_plane, p.splits);
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
  return a.bf16_io ? HeadRun<bf16>(a, p, sm_count, s).forward() : HeadRun<float>(a, p, sm_count, s).forward();
}

cudaError_t run_token_logprob_backward(const HeadArgs& a, int sm_count, cudaStream_t s) {
  const HeadPlan p = plan_head(a.N, a.D, a.V, a.bf16_io, true, !in_place(a), sm_count);
  return a.bf16_io ? HeadRun<bf16>(a, p, sm_count, s).backward() : HeadRun<float>(a, p, sm_count, s).backward();
}

cudaError_t status_head(unsigned int* word, bool clear) { return unit_status(word, clear); }

}  // namespace rlca
