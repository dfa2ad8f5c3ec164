// trunk_api.cu -- the extern "C" entry points of a recurrent policy's trunk
// declared in include/rlca.h: argument checks on the host, then the launches.
// Nothing here allocates or synchronises.
#include <cmath>

#include "host_checks.h"
#include "policy.h"
#include "policy_checks.h"
#include "rlca.h"
#include "trunk.h"

namespace rlca {

namespace {

constexpr int64_t kMaxSteps = int64_t(1) << 30;

bool sizes_ok(int64_t n, int64_t width) { return n >= 0 && width >= 0 && n <= kMaxRows && width <= kMaxWidth; }

// n rows of `width` elements at a row stride, all of `elem` bytes
struct Rows {
  const void* p;
  int64_t n, width, stride;
  size_t elem;
  size_t bytes() const { return p == nullptr || n == 0 ? 0 : ((size_t)(n - 1) * (size_t)stride + (size_t)width) * elem; }
  bool ok() const { return p == nullptr || (stride >= width && stride <= kMaxStride && aligned(p, elem)); }
};

// whether two matrices share an element: rows at one stride may lie side by side
bool rows_overlap(const Rows& a, const Rows& b) {
  if (!overlap({a.p, a.bytes()}, {b.p, b.bytes()})) return false;
  if (a.stride != b.stride || a.elem != b.elem || a.n <= 1 || b.n <= 1) return true;
  const int64_t pitch = a.stride * (int64_t)a.elem;
  int64_t at = ((int64_t)((uintptr_t)b.p - (uintptr_t)a.p)) % pitch;  // b's columns in a's rows
  if (at < 0) at += pitch;
  return at < a.width * (int64_t)a.elem || at + b.width * (int64_t)b.elem > pitch;
}

// every output against every input and every other output
bool rows_clash(std::initializer_list<Rows> ins, std::initializer_list<Rows> outs) {
  for (const Rows& o : outs) {
    for (const Rows& i : ins)
      if (rows_overlap(o, i)) return true;
    for (const Rows& o2 : outs)
      if (&o2 != &o && rows_overlap(o, o2)) return true;
  }
  return false;
}

bool rows_ok(std::initializer_list<Rows> all) {
  for (const Rows& r : all)
    if (!r.ok()) return false;
  return true;
}

Rows flat(const void* p, int64_t n, size_t elem) { return {p, 1, n, n > 0 ? n : 1, elem}; }

// sizes and flags of a gated scan: RLCA_OK with *empty where nothing is to be done, or the status to return
int gated_sizes(int64_t E, int64_t T, int64_t D, uint32_t flags, bool* empty) {
  if (!sizes_ok(E, D) || T < 0 || T > kMaxSteps || !flags_ok(flags, RLCA_TIME_MAJOR | RLCA_BF16)) return RLCA_ERR_INVALID_ARG;
  *empty = E == 0 || D == 0;
  if (!*empty && E * T > kMaxRows) return RLCA_ERR_INVALID_ARG;
  return RLCA_OK;
}

}  // namespace

}  // namespace rlca

using namespace rlca;

extern "C" {

int rlca_rms_norm(const float* x, const float* residual, const float* weight, float* total, float* y, uint8_t* y8,
                  float* y8_scale, uint8_t* total8, float* total8_scale, float* rstd, int64_t N, int64_t D,
                  int64_t x_stride, int64_t residual_stride, float eps, uint32_t flags, rlca_stream_t stream) {
  if (!sizes_ok(N, D) || !flags_ok(flags, RLCA_BF16) || !(eps >= 0.f) || std::isinf(eps)) return RLCA_ERR_INVALID_ARG;
  if (N == 0 || D == 0) return RLCA_OK;
  if (!x || !weight || (residual == nullptr) != (total == nullptr) || (y8 == nullptr) != (y8_scale == nullptr) ||
      (total8 == nullptr) != (total8_scale == nullptr) || (!total && !y && !y8 && !total8 && !rstd))
    return RLCA_ERR_INVALID_ARG;
  const size_t es = ebytes(flags);
  const int64_t groups = div_up(D, RLCA_GROUP);
  const Rows rx{x, N, D, x_stride, es}, rr{residual, N, D, residual_stride, es}, rt{total, N, D, D, es};
  const Rows rw = flat(weight, D, es), ry{y, N, D, D, es}, rs = flat(rstd, N, 4);
  const Rows q1{y8, N, D, D, 1}, s1{y8_scale, N, groups, groups, 4}, q2{total8, N, D, D, 1},
      s2{total8_scale, N, groups, groups, 4};
  if (!rows_ok({rx, rr, rt, rw, ry, rs, s1, s2})) return RLCA_ERR_INVALID_ARG;
  const bool in_place = total != nullptr && total == residual && residual_stride == D;
  if (rows_clash({rx, rw}, {rt, ry, q1, s1, q2, s2, rs}) ||
      (residual && rows_clash({rr}, {in_place ? Rows{nullptr, N, D, D, es} : rt, ry, q1, s1, q2, s2, rs})))
    return RLCA_ERR_INVALID_ARG;
  int sm = 0;
  if (sm_count_of_current_device(&sm) != cudaSuccess) return RLCA_ERR_CUDA;
  RmsArgs a = {};
  a.x = x; a.residual = residual; a.weight = weight; a.total = total; a.y = y; a.y8 = y8; a.y8_scale = y8_scale;
  a.total8 = total8; a.total8_scale = total8_scale; a.rstd = rstd;
  a.N = N; a.D = D; a.x_stride = x_stride; a.residual_stride = residual_stride; a.eps = eps;
  a.bf16_io = (flags & RLCA_BF16) != 0;
  return launched(run_rms_norm(a, sm, stream), stream);
}

int rlca_rms_norm_backward(const float* dy, const float* d_total, const float* total, const uint8_t* total8,
                           const float* total8_scale, const float* weight, const float* rstd, float* dx, float* dweight,
                           int64_t N, int64_t D, int64_t dy_stride, int64_t d_total_stride, int64_t total_stride,
                           uint32_t flags, void* workspace, size_t workspace_bytes, rlca_stream_t stream) {
  if (!sizes_ok(N, D) || !flags_ok(flags, RLCA_BF16)) return RLCA_ERR_INVALID_ARG;
  if (D == 0) return RLCA_OK;
  if (!dx && !dweight) return RLCA_ERR_INVALID_ARG;
  const size_t es = ebytes(flags);
  if (N > 0 && (!dy || !weight || !rstd || (total == nullptr) == (total8 == nullptr) ||
                (total8 == nullptr) != (total8_scale == nullptr)))
    return RLCA_ERR_INVALID_ARG;
  const int64_t groups = div_up(D, RLCA_GROUP);
  const Rows rdy{dy, N, D, dy_stride, es}, rdt{d_total, N, D, d_total_stride, es}, rt{total, N, D, total_stride, es};
  const Rows q{total8, N, D, D, 1}, sc{total8_scale, N, groups, groups, 4}, rw = flat(weight, D, es), rs = flat(rstd, N, 4);
  const Rows ws = flat(workspace, (int64_t)workspace_bytes, 1), rdx{dx, N, D, D, es}, rdw = flat(dweight, D, es);
  if ((N > 0 && !rows_ok({rdy, rdt, rt, sc, rw, rs, rdx})) || !rdw.ok()) return RLCA_ERR_INVALID_ARG;
  if (rows_clash({rdy, rdt, rt, q, sc, rw, rs}, {rdx, rdw, ws})) return RLCA_ERR_INVALID_ARG;
  int sm = 0;
  if (sm_count_of_current_device(&sm) != cudaSuccess) return RLCA_ERR_CUDA;
  if (!workspace_ok(workspace, workspace_bytes, N == 0 ? 0 : rms_norm_backward_workspace(N, D, sm))) return RLCA_ERR_INVALID_ARG;
  RmsGradArgs a = {};
  a.dy = dy; a.d_total = d_total; a.total = total; a.total8 = total8; a.total8_scale = total8_scale;
  a.weight = weight; a.rstd = rstd; a.dx = dx; a.dweight = dweight;
  a.N = N; a.D = D; a.dy_stride = dy_stride; a.d_total_stride = d_total_stride; a.total_stride = total_stride;
  a.bf16_io = (flags & RLCA_BF16) != 0; a.ws = static_cast<float*>(workspace);
  return launched(run_rms_norm_backward(a, sm, stream), stream);
}

int rlca_gated_scan(const float* x, const float* gate, const uint8_t* terminated, const uint8_t* truncated,
                    const float* state, const int32_t* lengths, float* h, float* last, int64_t E, int64_t T, int64_t D,
                    int64_t x_stride, int64_t gate_stride, uint32_t flags, void* workspace, size_t workspace_bytes,
                    rlca_stream_t stream) {
  bool empty = false;
  const int st = gated_sizes(E, T, D, flags, &empty);
  if (st != RLCA_OK || empty) return st;
  const size_t es = ebytes(flags);
  const int64_t n = E * T;
  if (n > 0 && (!x || !gate || !h)) return RLCA_ERR_INVALID_ARG;
  if (n == 0 && !last) return RLCA_OK;
  const Rows rx{x, n, D, x_stride, es}, rg{gate, n, D, gate_stride, es}, rh{h, n, D, D, es};
  const Rows t1 = flat(terminated, n, 1), t2 = flat(truncated, n, 1), len = flat(lengths, E, 4);
  const Rows s0 = flat(state, E * D, 4), s1 = flat(last, E * D, 4);
  if ((n > 0 && !rows_ok({rx, rg, rh})) || !rows_ok({len, s0, s1})) return RLCA_ERR_INVALID_ARG;
  const Rows ws = flat(workspace, (int64_t)workspace_bytes, 1);
  if (rows_clash({rx, rg, t1, t2, len}, {rh, s1, ws}) || rows_overlap(rh, s0) || rows_overlap(ws, s0) ||
      (last != state && rows_overlap(s1, s0)))
    return RLCA_ERR_INVALID_ARG;
  int sm = 0;
  if (sm_count_of_current_device(&sm) != cudaSuccess) return RLCA_ERR_CUDA;
  if (!workspace_ok(workspace, workspace_bytes, gated_scan_workspace(E, T, D, (flags & RLCA_BF16) != 0, false, sm)))
    return RLCA_ERR_INVALID_ARG;
  GatedArgs a = {};
  a.ws = workspace;
  a.x = x; a.gate = gate; a.terminated = terminated; a.truncated = truncated; a.state = state; a.lengths = lengths;
  a.h = h; a.last = last;
  a.E = E; a.T = T; a.D = D; a.step_e = (flags & RLCA_TIME_MAJOR) ? 1 : T; a.step_t = (flags & RLCA_TIME_MAJOR) ? E : 1;
  a.x_stride = x_stride; a.gate_stride = gate_stride; a.h_stride = D; a.bf16_io = (flags & RLCA_BF16) != 0;
  return launched(run_gated_scan(a, sm, stream), stream);
}

int rlca_gated_scan_backward(const float* dh, const float* x, const float* gate, const float* h,
                             const uint8_t* terminated, const uint8_t* truncated, const float* state,
                             const int32_t* lengths, const float* d_last, float* dx, float* dgate, float* d_state,
                             int64_t E, int64_t T, int64_t D, int64_t dh_stride, int64_t x_stride, int64_t gate_stride,
                             int64_t h_stride, int64_t dx_stride, int64_t dgate_stride, uint32_t flags,
                             void* workspace, size_t workspace_bytes, rlca_stream_t stream) {
  bool empty = false;
  const int st = gated_sizes(E, T, D, flags, &empty);
  if (st != RLCA_OK || empty) return st;
  const size_t es = ebytes(flags);
  const int64_t n = E * T;
  if (n > 0 && (!dh || !x || !gate || !h || !dx || !dgate)) return RLCA_ERR_INVALID_ARG;
  if (n == 0 && !d_state) return RLCA_OK;
  const Rows rdh{dh, n, D, dh_stride, es}, rx{x, n, D, x_stride, es}, rg{gate, n, D, gate_stride, es},
      rh{h, n, D, h_stride, es}, rdx{dx, n, D, dx_stride, es}, rdg{dgate, n, D, dgate_stride, es};
  const Rows t1 = flat(terminated, n, 1), t2 = flat(truncated, n, 1), len = flat(lengths, E, 4);
  const Rows s0 = flat(state, E * D, 4), dl = flat(d_last, E * D, 4), ds = flat(d_state, E * D, 4);
  if ((n > 0 && !rows_ok({rdh, rx, rg, rh, rdx, rdg})) || !rows_ok({len, s0, dl, ds})) return RLCA_ERR_INVALID_ARG;
  const Rows ws = flat(workspace, (int64_t)workspace_bytes, 1);
  if (rows_clash({rdh, rx, rg, rh, t1, t2, len, s0}, {rdx, rdg, ds, ws}) || rows_overlap(rdx, dl) || rows_overlap(rdg, dl) ||
      rows_overlap(ws, dl) || (d_state != d_last && rows_overlap(ds, dl)))
    return RLCA_ERR_INVALID_ARG;
  int sm = 0;
  if (sm_count_of_current_device(&sm) != cudaSuccess) return RLCA_ERR_CUDA;
  if (!workspace_ok(workspace, workspace_bytes, gated_scan_workspace(E, T, D, (flags & RLCA_BF16) != 0, true, sm)))
    return RLCA_ERR_INVALID_ARG;
  GatedArgs a = {};
  a.ws = workspace;
  a.dh = dh; a.x = x; a.gate = gate; a.in_h = h; a.terminated = terminated; a.truncated = truncated; a.state = state;
  a.lengths = lengths; a.d_last = d_last; a.dx = dx; a.dgate = dgate; a.d_state = d_state;
  a.E = E; a.T = T; a.D = D; a.step_e = (flags & RLCA_TIME_MAJOR) ? 1 : T; a.step_t = (flags & RLCA_TIME_MAJOR) ? E : 1;
  a.dh_stride = dh_stride; a.x_stride = x_stride; a.gate_stride = gate_stride; a.h_stride = h_stride;
  a.dx_stride = dx_stride; a.dgate_stride = dgate_stride; a.bf16_io = (flags & RLCA_BF16) != 0;
  return launched(run_gated_scan_backward(a, sm, stream), stream);
}

}  // extern "C"
