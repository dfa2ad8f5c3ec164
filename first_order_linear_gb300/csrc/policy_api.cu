// policy_api.cu -- the extern "C" entry points of the policy-update
// operators declared in include/rlca.h: argument checks on the host, then
// the launches.  Nothing here allocates or synchronises.
#include <algorithm>
#include <cmath>

#include "host_checks.h"
#include "policy.h"
#include "policy_checks.h"
#include "rlca.h"

namespace rlca {

namespace {

// bytes from the first to the last element of n rows of `width` elements
size_t matrix_bytes(int64_t n, int64_t width, int64_t stride, size_t elem) {
  return n == 0 ? 0 : ((size_t)(n - 1) * (size_t)stride + (size_t)width) * elem;
}

bool stride_ok(int64_t stride, int64_t width) { return stride >= width && stride <= kMaxStride; }

// head sizes: RLCA_OK, or the status to return
int head_sizes(int64_t N, int64_t D, int64_t V) {
  if (N < 0 || D < 1 || V < 1) return RLCA_ERR_INVALID_ARG;
  if (D > RLCA_MAX_HEAD_DIM || N > RLCA_MAX_HEAD_ROWS || V > RLCA_MAX_HEAD_ROWS) return RLCA_ERR_UNSUPPORTED;
  return RLCA_OK;
}

bool temperature_ok(float inv) { return inv > 0.f && std::isfinite(inv); }

}  // namespace

bool policy_estimator(int estimator) {
  return estimator >= RLCA_EST_TOKEN_LOGPROB && estimator <= RLCA_EST_GATED_SCAN_BACKWARD;
}

int policy_workspace_size(int estimator, int64_t E, int64_t T, int32_t num_actions, uint32_t flags, size_t* bytes) {
  const bool scan = estimator == RLCA_EST_GATED_SCAN || estimator == RLCA_EST_GATED_SCAN_BACKWARD;
  if (!flags_ok(flags, scan ? RLCA_BF16 | RLCA_TIME_MAJOR : RLCA_BF16)) return RLCA_ERR_INVALID_ARG;
  const bool head = estimator == RLCA_EST_TOKEN_LOGPROB || estimator == RLCA_EST_TOKEN_LOGPROB_BACKWARD;
  if (head) {
    const int st = head_sizes(E, T, num_actions);
    if (st != RLCA_OK) return st;
  } else if (E < 0 || T < 0 || E > kMaxRows || T > kMaxWidth) {
    return RLCA_ERR_INVALID_ARG;
  } else if (scan && (num_actions < 0 || num_actions > kMaxWidth || (num_actions > 0 && E * T > kMaxRows))) {
    return RLCA_ERR_INVALID_ARG;
  }
  if (E == 0 || T == 0) return RLCA_OK;
  int sm = 0;
  if (sm_count_of_current_device(&sm) != cudaSuccess) return RLCA_ERR_CUDA;
  if (head)
    *bytes = head_workspace(E, T, num_actions, (flags & RLCA_BF16) != 0, estimator == RLCA_EST_TOKEN_LOGPROB_BACKWARD, sm);
  else if (estimator == RLCA_EST_LAYER_NORM_BACKWARD)
    *bytes = layer_norm_backward_workspace(E, T, sm);
  else if (scan)
    *bytes = gated_scan_workspace(E, T, num_actions, (flags & RLCA_BF16) != 0, estimator == RLCA_EST_GATED_SCAN_BACKWARD, sm);
  else if (estimator == RLCA_EST_RMS_NORM_BACKWARD)
    *bytes = rms_norm_backward_workspace(E, T, sm);
  else
    *bytes = clip_workspace(E, sm);
  return RLCA_OK;
}

}  // namespace rlca

using namespace rlca;

extern "C" {

int rlca_layer_norm(const float* x, const float* weight, const float* bias, float* y, float* mean, float* rstd,
                    int64_t N, int64_t D, int64_t x_stride, float eps, uint32_t flags, rlca_stream_t stream) {
  if (N < 0 || D < 0 || N > kMaxRows || D > kMaxWidth || !flags_ok(flags, RLCA_BF16)) return RLCA_ERR_INVALID_ARG;
  if (!(eps >= 0.f) || std::isinf(eps)) return RLCA_ERR_INVALID_ARG;
  if (N == 0 || D == 0) return RLCA_OK;
  if (!x || !weight || !y || !stride_ok(x_stride, D)) return RLCA_ERR_INVALID_ARG;
  const size_t es = ebytes(flags), nd = (size_t)N * (size_t)D * es, d = (size_t)D * es, n = (size_t)N * 4;
  if (any_overlap({{x, matrix_bytes(N, D, x_stride, es)}, {weight, d}, {bias, d}}, {{y, nd}, {mean, n}, {rstd, n}}))
    return RLCA_ERR_INVALID_ARG;
  int sm = 0;
  if (sm_count_of_current_device(&sm) != cudaSuccess) return RLCA_ERR_CUDA;
  NormArgs a = {};
  a.x = x; a.weight = weight; a.bias = bias; a.y = y; a.mean = mean; a.rstd = rstd;
  a.N = N; a.D = D; a.x_stride = x_stride; a.eps = eps; a.bf16_io = (flags & RLCA_BF16) != 0;
  return launched(run_layer_norm(a, sm, stream), stream);
}

int rlca_layer_norm_backward(const float* dy, const float* x, const float* weight, const float* mean,
                             const float* rstd, float* dx, float* dweight, float* dbias, int64_t N, int64_t D,
                             int64_t dy_stride, int64_t x_stride, uint32_t flags, void* workspace,
                             size_t workspace_bytes, rlca_stream_t stream) {
  if (N < 0 || D < 0 || N > kMaxRows || D > kMaxWidth || !flags_ok(flags, RLCA_BF16)) return RLCA_ERR_INVALID_ARG;
  if (D == 0) return RLCA_OK;
  if (!dx && !dweight && !dbias) return RLCA_ERR_INVALID_ARG;
  if (N > 0 && (!dy || !x || !weight || !mean || !rstd || !stride_ok(dy_stride, D) || !stride_ok(x_stride, D)))
    return RLCA_ERR_INVALID_ARG;
  const size_t es = ebytes(flags), nd = (size_t)N * (size_t)D * es, d = (size_t)D * es, n = (size_t)N * 4;
  if (any_overlap({{dy, matrix_bytes(N, D, dy_stride, es)}, {x, matrix_bytes(N, D, x_stride, es)}, {weight, d},
                   {mean, n}, {rstd, n}, {workspace, workspace_bytes}},
                  {{dx, nd}, {dweight, d}, {dbias, d}}))
    return RLCA_ERR_INVALID_ARG;
  int sm = 0;
  if (sm_count_of_current_device(&sm) != cudaSuccess) return RLCA_ERR_CUDA;
  if (N > 0 && !workspace_ok(workspace, workspace_bytes, layer_norm_backward_workspace(N, D, sm)))
    return RLCA_ERR_INVALID_ARG;
  NormGradArgs a = {};
  a.dy = dy; a.x = x; a.weight = weight; a.mean = mean; a.rstd = rstd;
  a.dx = dx; a.dweight = dweight; a.dbias = dbias;
  a.N = N; a.D = D; a.dy_stride = dy_stride; a.x_stride = x_stride; a.bf16_io = (flags & RLCA_BF16) != 0;
  a.ws = static_cast<float*>(workspace);
  return launched(run_layer_norm_backward(a, sm, stream), stream);
}

int rlca_token_logprob(const float* hidden, const float* weight, const int32_t* tokens, float* logp, float* lse,
                       float* entropy, int64_t N, int64_t D, int64_t V, int64_t hidden_stride, int64_t weight_stride,
                       float inv_temperature, uint32_t flags, void* workspace, size_t workspace_bytes,
                       rlca_stream_t stream) {
  const int st = head_sizes(N, D, V);
  if (st != RLCA_OK) return st;
  if (!flags_ok(flags, RLCA_BF16) || !temperature_ok(inv_temperature)) return RLCA_ERR_INVALID_ARG;
  if (N == 0) return RLCA_OK;
  if (!hidden || !weight || !tokens || !logp || !lse || !stride_ok(hidden_stride, D) || !stride_ok(weight_stride, D))
    return RLCA_ERR_INVALID_ARG;
  const size_t es = ebytes(flags), n = (size_t)N * 4;
  if (any_overlap({{hidden, matrix_bytes(N, D, hidden_stride, es)}, {weight, matrix_bytes(V, D, weight_stride, es)},
                   {tokens, n}, {workspace, workspace_bytes}},
                  {{logp, n}, {lse, n}, {entropy, n}}))
    return RLCA_ERR_INVALID_ARG;
  int sm = 0;
  if (sm_count_of_current_device(&sm) != cudaSuccess) return RLCA_ERR_CUDA;
  const bool bf = (flags & RLCA_BF16) != 0;
  if (!workspace_ok(workspace, workspace_bytes, head_workspace(N, D, V, bf, false, sm))) return RLCA_ERR_INVALID_ARG;
  HeadArgs a = {};
  a.hidden = hidden; a.weight = weight; a.tokens = tokens; a.logp = logp; a.lse = lse; a.entropy = entropy;
  a.N = N; a.D = D; a.V = V; a.hidden_stride = hidden_stride; a.weight_stride = weight_stride;
  a.inv_temperature = inv_temperature; a.bf16_io = bf; a.ws = workspace;
  return launched(run_token_logprob(a, sm, stream), stream);
}

int rlca_token_logprob_backward(const float* hidden, const float* weight, const int32_t* tokens, const float* lse,
                                const float* entropy, const float* d_logp, const float* d_entropy, float* d_hidden,
                                float* d_weight, int64_t N, int64_t D, int64_t V, int64_t hidden_stride,
                                int64_t weight_stride, float inv_temperature, uint32_t flags, void* workspace,
                                size_t workspace_bytes, rlca_stream_t stream) {
  const int st = head_sizes(N, D, V);
  if (st != RLCA_OK) return st;
  if (!flags_ok(flags, RLCA_BF16) || !temperature_ok(inv_temperature)) return RLCA_ERR_INVALID_ARG;
  if (!d_hidden && !d_weight) return RLCA_ERR_INVALID_ARG;
  const size_t es = ebytes(flags), n = (size_t)N * 4;
  if (N == 0) {
    if (d_weight == nullptr) return RLCA_OK;
    const cudaError_t e = cudaMemsetAsync(d_weight, 0, (size_t)V * (size_t)D * es, stream);
    return e == cudaSuccess ? RLCA_OK : RLCA_ERR_CUDA;
  }
  if (!hidden || !weight || !tokens || !lse || !d_logp || (entropy == nullptr) != (d_entropy == nullptr) ||
      !stride_ok(hidden_stride, D) || !stride_ok(weight_stride, D))
    return RLCA_ERR_INVALID_ARG;
  if (any_overlap({{hidden, matrix_bytes(N, D, hidden_stride, es)}, {weight, matrix_bytes(V, D, weight_stride, es)},
                   {tokens, n}, {lse, n}, {entropy, n}, {d_logp, n}, {d_entropy, n}, {workspace, workspace_bytes}},
                  {{d_hidden, (size_t)N * (size_t)D * es}, {d_weight, (size_t)V * (size_t)D * es}}))
    return RLCA_ERR_INVALID_ARG;
  int sm = 0;
  if (sm_count_of_current_device(&sm) != cudaSuccess) return RLCA_ERR_CUDA;
  const bool bf = (flags & RLCA_BF16) != 0;
  if (!workspace_ok(workspace, workspace_bytes, head_workspace(N, D, V, bf, true, sm))) return RLCA_ERR_INVALID_ARG;
  HeadArgs a = {};
  a.hidden = hidden; a.weight = weight; a.tokens = tokens;
  a.in_lse = lse; a.in_entropy = entropy; a.d_logp = d_logp; a.d_entropy = d_entropy;
  a.d_hidden = d_hidden; a.d_weight = d_weight;
  a.N = N; a.D = D; a.V = V; a.hidden_stride = hidden_stride; a.weight_stride = weight_stride;
  a.inv_temperature = inv_temperature; a.bf16_io = bf; a.ws = workspace;
  return launched(run_token_logprob_backward(a, sm, stream), stream);
}

int rlca_clip_grads(const void* const* grads, void* const* outs, const int64_t* sizes, const uint32_t* dtypes,
                    int64_t count, float max_norm, float eps, float* norm, void* workspace, size_t workspace_bytes,
                    rlca_stream_t stream) {
  if (count < 0 || count > kMaxRows || !norm || !(max_norm >= 0.f) || !(eps >= 0.f)) return RLCA_ERR_INVALID_ARG;
  if (count > 0 && (!grads || !sizes || !dtypes)) return RLCA_ERR_INVALID_ARG;
  const Span nspan{norm, 4}, wspan{workspace, workspace_bytes};
  if (overlap(nspan, wspan)) return RLCA_ERR_INVALID_ARG;
  for (int64_t k = 0; k < count; ++k) {
    if (sizes[k] < 0 || sizes[k] > (int64_t(1) << 40) || !flags_ok(dtypes[k], RLCA_BF16)) return RLCA_ERR_INVALID_ARG;
    if (sizes[k] == 0) continue;
    const uintptr_t es = (uintptr_t)ebytes(dtypes[k]);
    if (!grads[k] || !aligned(grads[k], es)) return RLCA_ERR_INVALID_ARG;
    const Span g{grads[k], (size_t)sizes[k] * es};
    if (overlap(g, nspan) || overlap(g, wspan)) return RLCA_ERR_INVALID_ARG;
    if (!outs) continue;
    if (!outs[k] || !aligned(outs[k], es)) return RLCA_ERR_INVALID_ARG;
    const Span o{outs[k], g.bytes};
    if ((outs[k] != grads[k] && overlap(o, g)) || overlap(o, nspan) || overlap(o, wspan)) return RLCA_ERR_INVALID_ARG;
  }
  int sm = 0;
  if (sm_count_of_current_device(&sm) != cudaSuccess) return RLCA_ERR_CUDA;
  if (count > 0 && !workspace_ok(workspace, workspace_bytes, clip_workspace(count, sm))) return RLCA_ERR_INVALID_ARG;
  ClipArgs a = {};
  a.grads = grads; a.outs = outs; a.sizes = sizes; a.dtypes = dtypes; a.count = count;
  a.max_norm = max_norm; a.eps = eps; a.norm = norm; a.ws = static_cast<double*>(workspace);
  return launched(run_clip_grads(a, sm, stream), stream);
}

}  // extern "C"
