// Token log-probabilities and entropies of a policy head, and their gradient.
#include <algorithm>

#include "policy.h"
#include "reduce.cuh"

namespace rlca {

namespace {

// ---------------------------------------------------------------------------
// Workspace.  Rows that take part are numbered in order ("parts"); `rows`
// maps a part to its row, and count[0] is how many there are -- known on the
// device only, so grids cover all N rows and what lies past count[0] leaves.
// ---------------------------------------------------------------------------
constexpr int kTile = 64;  // logits tiles are kTile parts x kTile tokens
constexpr int64_t kPieceBytes = int64_t(256) << 20;  // dz of one piece of the vocabulary

struct HeadPlan {
  int64_t row_tiles, col_tiles;
  int64_t piece;  // backward: tokens per piece of the vocabulary (whole tiles)
  size_t count, rows, part, taken, dz, dh;  // byte offsets
  size_t bytes;
};

HeadPlan plan_head(int64_t N, int64_t D, int64_t V, bool backward) {
  HeadPlan p = {};
  p.row_tiles = div_up(N, kTile);
  p.col_tiles = div_up(V, kTile);
  size_t at = 0;
  const auto take = [&](size_t n) {
    const size_t here = at;
    at += (n + 255) & ~size_t(255);
    return here;
  };
  p.count = take(4);
  p.rows = take((size_t)N * 4);
  if (backward) {
    p.piece = std::min(p.col_tiles, std::max<int64_t>(1, kPieceBytes / (4 * N * kTile))) * kTile;
    p.dz = take((size_t)N * p.piece * 4);
    p.dh = take((size_t)N * D * 4);
  } else {
    p.part = take((size_t)p.col_tiles * N * sizeof(float4));
    p.taken = take((size_t)N * 4);
  }
  p.bytes = at;
  return p;
}

struct HeadView {  // the workspace's arrays on the device
  int* count;
  int* rows;
  float4* part;
  float* taken;
  float* dz;
  float* dh;
  HeadView(const HeadPlan& p, void* ws) {
    unsigned char* b = static_cast<unsigned char*>(ws);
    count = reinterpret_cast<int*>(b + p.count);
    rows = reinterpret_cast<int*>(b + p.rows);
    part = reinterpret_cast<float4*>(b + p.part);
    taken = reinterpret_cast<float*>(b + p.taken);
    dz = reinterpret_cast<float*>(b + p.dz);
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
    if (on) w.rows[before + __popc(vote & ((1u << lane) - 1u))] = (int)i;
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
// One kTile x kTile tile of sum_k A(m, k) B(n, k) in float32, 4 x 4 values a
// thread; A and B are loaders that return 0 outside their arrays.
// ---------------------------------------------------------------------------
constexpr int kTileThreads = 256;
constexpr int kTileK = 16;

template <class LA, class LB>
__device__ __forceinline__ void tile_product(const LA& A, const LB& B, int64_t m0, int64_t n0, int64_t K,
                                             float (&acc)[4][4]) {
  __shared__ float sa[kTileK][kTile + 1], sb[kTileK][kTile + 1];
  const int tm = (threadIdx.x >> 4) * 4, tn = (threadIdx.x & 15) * 4;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
  for (int64_t k0 = 0; k0 < K; k0 += kTileK) {
    for (int t = threadIdx.x; t < kTile * kTileK; t += kTileThreads) {
      A.stage(sa, m0, k0, t);
      B.stage(sb, n0, k0, t);
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kTileK; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(sa[k][tm + i], sb[k][tn + j], acc[i][j]);
    __syncthreads();
  }
}

// element (m, k) of a matrix with k contiguous: row `map[m]` (or m) of p
template <class ST>
struct RowMajor {
  const float* p;
  const int* map;
  int64_t stride, M, K;
  __device__ __forceinline__ void stage(float (&s)[kTileK][kTile + 1], int64_t m0, int64_t k0, int t) const {
    const int k = t % kTileK, m = t / kTileK;
    float v = 0.f;
    if (m0 + m < M && k0 + k < K) v = Stor<ST>::ld(p, (map ? (int64_t)map[m0 + m] : m0 + m) * stride + k0 + k);
    s[k][m] = v;
  }
};
// ... and with m contiguous: row `map[k]` (or k) of p
template <class ST>
struct ColMajor {
  const float* p;
  const int* map;
  int64_t stride, M, K;
  __device__ __forceinline__ void stage(float (&s)[kTileK][kTile + 1], int64_t m0, int64_t k0, int t) const {
    const int m = t % kTile, k = t / kTile;
    float v = 0.f;
    if (m0 + m < M && k0 + k < K) v = Stor<ST>::ld(p, (map ? (int64_t)map[k0 + k] : k0 + k) * stride + m0 + m);
    s[k][m] = v;
  }
};

// a tile of logits: part[tile][part] = (max, sum e^{z - max}, sum e^{z - max} z)
template <class ST>
__global__ void __launch_bounds__(kTileThreads) head_stats_kernel(HeadArgs a, HeadView w, int64_t row_tiles) {
  pdl_trigger();
  pdl_wait();
  const int64_t m0 = (blockIdx.x % row_tiles) * kTile, n0 = (blockIdx.x / row_tiles) * kTile;
  const int64_t count = w.count[0];
  if (m0 >= count) return;
  float acc[4][4];
  tile_product(RowMajor<ST>{a.hidden, w.rows, a.hidden_stride, count, a.D},
               RowMajor<ST>{a.weight, nullptr, a.weight_stride, a.V, a.D}, m0, n0, a.D, acc);
  __shared__ float z[kTile][kTile + 1];
  const int tm = (threadIdx.x >> 4) * 4, tn = (threadIdx.x & 15) * 4;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) z[tm + i][tn + j] = acc[i][j] * a.inv_temperature;
  __syncthreads();
  const int64_t m = m0 + threadIdx.x;
  if (threadIdx.x >= kTile || m >= count) return;
  const float* row = z[threadIdx.x];
  const int n = (int)min((int64_t)kTile, a.V - n0);
  float top = row[0];
  for (int j = 1; j < n; ++j) top = fmaxf(top, row[j]);
  float s = 0.f, t = 0.f;
  for (int j = 0; j < n; ++j) {
    const float e = __expf(row[j] - top);
    s += e;
    t += e * row[j];
  }
  w.part[(n0 / kTile) * a.N + m] = make_float4(top, s, t, 0.f);
  const int64_t at = a.tokens[w.rows[m]] - n0;
  if (at >= 0 && at < n) w.taken[m] = row[at];
}

// joins a part's tiles, one warp a part
__global__ void __launch_bounds__(kTileThreads) head_join_kernel(HeadArgs a, HeadView w, int64_t col_tiles) {
  pdl_trigger();
  pdl_wait();
  const int64_t m = (int64_t)blockIdx.x * (kTileThreads / 32) + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (m >= w.count[0]) return;
  float top = -INFINITY;
  for (int64_t k = lane; k < col_tiles; k += 32) top = fmaxf(top, w.part[k * a.N + m].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  float s = 0.f, t = 0.f;
  for (int64_t k = lane; k < col_tiles; k += 32) {
    const float4 p = w.part[k * a.N + m];
    const float f = __expf(p.x - top);
    s += p.y * f;
    t += p.z * f;
  }
  s = warp_sum(s);
  t = warp_sum(t);
  if (lane != 0) return;
  const float lse = top + logf(s);
  const int64_t i = w.rows[m];
  a.lse[i] = lse;
  a.logp[i] = w.taken[m] - lse;
  if (a.entropy) a.entropy[i] = lse - t / s;
}

// a tile of dz for the piece of the vocabulary that starts at token v0
template <class ST>
__global__ void __launch_bounds__(kTileThreads)
    head_dz_kernel(HeadArgs a, HeadView w, int64_t row_tiles, int64_t piece, int64_t v0) {
  pdl_trigger();
  pdl_wait();
  const int64_t m0 = (blockIdx.x % row_tiles) * kTile, n0 = v0 + (blockIdx.x / row_tiles) * kTile;
  const int64_t count = w.count[0];
  if (m0 >= count) return;
  float acc[4][4];
  tile_product(RowMajor<ST>{a.hidden, w.rows, a.hidden_stride, count, a.D},
               RowMajor<ST>{a.weight, nullptr, a.weight_stride, a.V, a.D}, m0, n0, a.D, acc);
  const int tm = (threadIdx.x >> 4) * 4, tn = (threadIdx.x & 15) * 4;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t m = m0 + tm + i;
    if (m >= count) continue;
    const int64_t row = w.rows[m];
    const float g = a.d_logp[row], e = a.d_entropy ? a.d_entropy[row] : 0.f;
    const float lse = a.in_lse[row], ent = a.d_entropy ? a.in_entropy[row] : 0.f;
    const int64_t at = a.tokens[row];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t v = n0 + tn + j;
      const float logq = acc[i][j] * a.inv_temperature - lse;
      const float dz = -__expf(logq) * (g + e * (logq + ent)) + (v == at ? g : 0.f);
      if (v < a.V) w.dz[m * piece + (v - v0)] = dz * a.inv_temperature;
    }
  }
}

// dh[part] += dz weight over one piece (or = for the first)
template <class ST>
__global__ void __launch_bounds__(kTileThreads)
    head_dh_kernel(HeadArgs a, HeadView w, int64_t row_tiles, int64_t piece, int64_t v0) {
  pdl_trigger();
  pdl_wait();
  const int64_t m0 = (blockIdx.x % row_tiles) * kTile, n0 = (blockIdx.x / row_tiles) * kTile;
  const int64_t count = w.count[0], K = min(piece, a.V - v0);
  if (m0 >= count) return;
  float acc[4][4];
  tile_product(RowMajor<float>{w.dz, nullptr, piece, count, K},
               ColMajor<ST>{reinterpret_cast<const float*>(reinterpret_cast<const unsigned char*>(a.weight) +
                                                           v0 * a.weight_stride * Stor<ST>::kBytes),
                            nullptr, a.weight_stride, a.D, K},
               m0, n0, K, acc);
  const int tm = (threadIdx.x >> 4) * 4, tn = (threadIdx.x & 15) * 4;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t m = m0 + tm + i, c = n0 + tn + j;
      if (m < count && c < a.D) w.dh[m * a.D + c] = acc[i][j] + (v0 > 0 ? w.dh[m * a.D + c] : 0.f);
    }
}

// d_weight = dz^T hidden over one piece
template <class ST>
__global__ void __launch_bounds__(kTileThreads)
    head_dw_kernel(HeadArgs a, HeadView w, int64_t tok_tiles, int64_t piece, int64_t v0) {
  pdl_trigger();
  pdl_wait();
  const int64_t m0 = (blockIdx.x % tok_tiles) * kTile, n0 = (blockIdx.x / tok_tiles) * kTile;
  const int64_t count = w.count[0], M = min(piece, a.V - v0);
  float acc[4][4];
  tile_product(ColMajor<float>{w.dz, nullptr, piece, M, count},
               ColMajor<ST>{a.hidden, w.rows, a.hidden_stride, a.D, count}, m0, n0, count, acc);
  const int tm = (threadIdx.x >> 4) * 4, tn = (threadIdx.x & 15) * 4;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t m = m0 + tm + i, c = n0 + tn + j;
      if (m < M && c < a.D) Stor<ST>::st(a.d_weight, (v0 + m) * a.D + c, acc[i][j]);
    }
}

// d_hidden: the parts' rows rounded once, zeros for rows that take no part
template <class ST>
__global__ void __launch_bounds__(kTileThreads) head_dh_out_kernel(HeadArgs a, HeadView w) {
  pdl_trigger();
  pdl_wait();
  const int64_t b = blockIdx.x;
  if (b < w.count[0]) {
    const int64_t row = w.rows[b];
    for (int64_t c = threadIdx.x; c < a.D; c += kTileThreads) Stor<ST>::st(a.d_hidden, row * a.D + c, w.dh[b * a.D + c]);
  }
  const int tok = a.tokens[b];
  if (tok < 0 || tok >= a.V)
    for (int64_t c = threadIdx.x; c < a.D; c += kTileThreads) Stor<ST>::st(a.d_hidden, b * a.D + c, 0.f);
}

template <class ST>
cudaError_t forward_typed(const HeadArgs& a, const HeadPlan& p, cudaStream_t s) {
  const HeadView w(p, a.ws);
  cudaError_t e = launch_pdl(head_rows_kernel, 1, kRowsThreads, 0, s, a, w);
  if (e == cudaSuccess)
    e = launch_pdl(head_stats_kernel<ST>, p.row_tiles * p.col_tiles, kTileThreads, 0, s, a, w, p.row_tiles);
  if (e == cudaSuccess)
    e = launch_pdl(head_join_kernel, div_up(a.N, kTileThreads / 32), kTileThreads, 0, s, a, w, p.col_tiles);
  return e;
}

template <class ST>
cudaError_t backward_typed(const HeadArgs& a, const HeadPlan& p, cudaStream_t s) {
  const HeadView w(p, a.ws);
  cudaError_t e = launch_pdl(head_rows_kernel, 1, kRowsThreads, 0, s, a, w);
  const int64_t d_tiles = div_up(a.D, kTile);
  for (int64_t v0 = 0; v0 < a.V && e == cudaSuccess; v0 += p.piece) {
    const int64_t tok_tiles = div_up(std::min(p.piece, a.V - v0), kTile);
    e = launch_pdl(head_dz_kernel<ST>, p.row_tiles * tok_tiles, kTileThreads, 0, s, a, w, p.row_tiles, p.piece, v0);
    if (e == cudaSuccess && a.d_hidden)
      e = launch_pdl(head_dh_kernel<ST>, p.row_tiles * d_tiles, kTileThreads, 0, s, a, w, p.row_tiles, p.piece, v0);
    if (e == cudaSuccess && a.d_weight)
      e = launch_pdl(head_dw_kernel<ST>, tok_tiles * d_tiles, kTileThreads, 0, s, a, w, tok_tiles, p.piece, v0);
  }
  if (e == cudaSuccess && a.d_hidden) e = launch_pdl(head_dh_out_kernel<ST>, a.N, kTileThreads, 0, s, a, w);
  return e;
}

}  // namespace

size_t head_workspace(int64_t N, int64_t D, int64_t V, bool, bool backward, int) {
  return plan_head(N, D, V, backward).bytes;
}

cudaError_t run_token_logprob(const HeadArgs& a, int, cudaStream_t s) {
  const HeadPlan p = plan_head(a.N, a.D, a.V, false);
  return a.bf16_io ? forward_typed<bf16>(a, p, s) : forward_typed<float>(a, p, s);
}

cudaError_t run_token_logprob_backward(const HeadArgs& a, int, cudaStream_t s) {
  const HeadPlan p = plan_head(a.N, a.D, a.V, true);
  return a.bf16_io ? backward_typed<bf16>(a, p, s) : backward_typed<float>(a, p, s);
}

cudaError_t status_head(unsigned int* word, bool clear) { return unit_status(word, clear); }

}  // namespace rlca
