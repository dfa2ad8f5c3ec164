"""PyTorch-facing wrappers of the C ABI, one per entry point, same names.

Each wrapper checks dtypes, devices and contiguity, allocates the outputs
(unless given) and the two-pass workspace, and makes one entry-point call
into ``librlca.so`` on the current CUDA stream (plus, the first time a shape
is seen, a workspace-size query whose answer is kept).  No arithmetic of
the method runs here; a missing library raises (see
:func:`first_order_linear_gb300._lib.load`).

Layout: env-major ``[E, T]`` by default; ``time_major=True`` takes ``[T, E]``
(and ``[T, E, A]`` for Retrace's per-action tensors).  ``inputs_ready=True``
sets RLCA_INPUTS_READY (the inputs were not written by the kernel just before
this call on the stream, so the call may overlap it).  Flags may be uint8 or
bool tensors; ``None`` means "no such flag" for the optional inputs.  Float
tensors are float32, or all bfloat16 (RLCA_BF16: bfloat16 storage, float32
arithmetic, outputs rounded once).
"""
from __future__ import annotations

import ctypes as C
import operator
from array import array

import torch

from . import _lib
from ._lib import check

__all__ = [
    "rlca_gae", "rlca_value_targets", "rlca_discounted_return", "rlca_td_lambda", "rlca_vtrace", "rlca_retrace",
    "rlca_elig_trace", "rlca_episodic_prefix_sum", "rlca_affine_scan", "rlca_workspace_size",
    "rlca_layer_norm", "rlca_layer_norm_backward", "rlca_token_logprob", "rlca_token_logprob_backward",
    "rlca_clip_grads",
]


def _require_cuda(dev):
    """The call's tensors (all on ``dev`` by the checks before) must be on a
    CUDA device: the kernels read device memory and there is no host
    implementation."""
    if dev.type != "cuda":
        raise ValueError(f"tensors are on {dev}: the kernels need tensors on a CUDA device")


def _ptr(t):
    # a plain int: the entry points' argtypes turn it into a void*
    return None if t is None else t.data_ptr()


def _check(t, name, dtypes, shape, device, required=True):
    if t is None:
        if required:
            raise ValueError(f"{name} is required")
        return
    # one combined test on the common path; the detailed checks name the fault
    if (isinstance(t, torch.Tensor) and t.dtype in dtypes and t.shape == shape and t.device == device
            and t.is_contiguous()):
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: dtype {t.dtype}, expected one of {dtypes}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


_F = (torch.float32,)
_U8 = (torch.uint8, torch.bool)
_I32 = (torch.int32,)


def _fdt(t, name):
    """Element type of a call's float arrays, taken from its first float
    input: float32, or bfloat16 (RLCA_BF16: bfloat16 storage, float32
    arithmetic).  Every other float tensor of the call must match."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError(f"{name}: dtype {t.dtype}, expected float32 or bfloat16")
    return t.dtype


def _fflag(fdt):
    return _lib.RLCA_BF16 if fdt == torch.bfloat16 else 0


def _flags(time_major, multipass, extra=0, inputs_ready=False):
    return ((_lib.RLCA_TIME_MAJOR if time_major else 0) | (_lib.RLCA_MULTIPASS if multipass else 0)
            | (_lib.RLCA_INPUTS_READY if inputs_ready else 0) | extra)


def _dims(x, time_major):
    if x.dim() < 2:
        raise ValueError("rollout tensors are 2-D ([E, T] or [T, E])")
    return (x.shape[1], x.shape[0]) if time_major else (x.shape[0], x.shape[1])


# workspace sizes by (estimator, E, T, A, flags, device index): a size
# depends only on these and the device's SM count, so each is asked once
_ws_sizes = {}


def rlca_workspace_size(estimator: int, E: int, T: int, num_actions: int = 0, flags: int = 0,
                        device=None) -> int:
    """Bytes of workspace a call needs on ``device`` (default: current)."""
    dev = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
    index = dev.index if dev.index is not None else torch.cuda.current_device()
    key = (estimator, E, T, num_actions, flags, index)
    need = _ws_sizes.get(key)
    if need is None:
        if len(_ws_sizes) >= 4096:  # many distinct shapes: start over rather than grow without bound
            _ws_sizes.clear()
        lib = _lib.load()
        out = C.c_size_t(0)
        with torch.cuda.device(index):
            check("rlca_workspace_size", lib.rlca_workspace_size(estimator, E, T, num_actions, flags, C.byref(out)))
        need = _ws_sizes[key] = out.value
    return need


def _workspace(estimator, E, T, A, flags, device, workspace):
    need = _ws_sizes.get((estimator, E, T, A, flags, device.index))
    if need is None:
        need = rlca_workspace_size(estimator, E, T, A, flags, device)
    if need == 0:
        return None, 0
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
    if workspace.numel() * workspace.element_size() < need or workspace.device != device:
        raise ValueError(f"workspace needs {need} bytes on {device}")
    return workspace, workspace.numel() * workspace.element_size()


def _stream(device, stream):
    s = stream if stream is not None else torch.cuda.current_stream(device)
    return s.cuda_stream


def _hold(device, stream, *tensors):
    """Marks device tensors the call reads or writes as in use on ``stream``
    when that is not the current stream.  Buffers this module allocates
    (the workspace, outputs not passed in) come from the caching allocator
    on the current stream; without the mark, memory freed there could be
    handed to new work on the current stream while the kernel on ``stream``
    still reads or writes it."""
    if stream is None or stream == torch.cuda.current_stream(device):
        return
    for t in tensors:
        if t is not None:
            t.record_stream(stream)


def _boundaries(shape, dev, terminated, truncated, trunc_value, bootstrap, E, F=_F):
    _check(terminated, "terminated", _U8, shape, dev, required=False)
    _check(truncated, "truncated", _U8, shape, dev, required=False)
    _check(trunc_value, "trunc_value", F, shape, dev, required=truncated is not None)
    _check(bootstrap, "bootstrap", F, (E,), dev, required=False)


def rlca_gae(rewards, values, terminated=None, truncated=None, trunc_value=None, bootstrap=None, *,
             gamma=0.99, lambda_=0.95, advantages=None, returns=None, want_returns=True,
             time_major=False, multipass=False, inputs_ready=False, workspace=None, stream=None):
    """GAE advantages (and returns = advantages + values).  Returns
    ``(advantages, returns)``; returns is None when ``want_returns`` is
    False and no buffer is given."""
    lib = _lib.load()
    dev = rewards.device
    fdt = _fdt(rewards, "rewards")
    F = (fdt,)
    E, T = _dims(rewards, time_major)
    shape = tuple(rewards.shape)
    _check(rewards, "rewards", F, shape, dev)
    _check(values, "values", F, shape, dev)
    _boundaries(shape, dev, terminated, truncated, trunc_value, bootstrap, E, F)
    if advantages is None:
        advantages = torch.empty(shape, dtype=fdt, device=dev)
    if returns is None and want_returns:
        returns = torch.empty(shape, dtype=fdt, device=dev)
    _check(advantages, "advantages", F, shape, dev)
    _check(returns, "returns", F, shape, dev, required=False)
    flags = _flags(time_major, multipass, inputs_ready=inputs_ready) | _fflag(fdt)
    _require_cuda(dev)
    with torch.cuda.device(dev):
        ws, wsb = _workspace(_lib.RLCA_EST_GAE, E, T, 0, flags, dev, workspace)
        check("rlca_gae", lib.rlca_gae(
            _ptr(rewards), _ptr(values), _ptr(terminated), _ptr(truncated), _ptr(trunc_value), _ptr(bootstrap),
            _ptr(advantages), _ptr(returns), E, T, gamma, lambda_, flags, _ptr(ws), wsb, _stream(dev, stream)))
        _hold(dev, stream, ws, advantages, returns)
    return advantages, returns


def rlca_value_targets(rewards, values, terminated=None, truncated=None, trunc_value=None, bootstrap=None, *,
                       gamma=0.99, lambda_=0.95, advantages=None, returns=None, disc_returns=None,
                       td_lambda_returns=None, outputs=("advantages", "returns", "disc_returns", "td_lambda_returns"),
                       time_major=False, multipass=False, inputs_ready=False, workspace=None, stream=None):
    """GAE advantages and returns, discounted returns and TD(lambda) returns
    in one fused pass.  ``outputs`` names the results to compute (buffers
    passed explicitly are always written).  Returns the four tensors (None
    for those not computed) in the order (advantages, returns,
    disc_returns, td_lambda_returns)."""
    lib = _lib.load()
    dev = rewards.device
    fdt = _fdt(rewards, "rewards")
    F = (fdt,)
    E, T = _dims(rewards, time_major)
    shape = tuple(rewards.shape)
    _check(rewards, "rewards", F, shape, dev)
    _check(values, "values", F, shape, dev)
    _boundaries(shape, dev, terminated, truncated, trunc_value, bootstrap, E, F)
    bufs = dict(advantages=advantages, returns=returns, disc_returns=disc_returns,
                td_lambda_returns=td_lambda_returns)
    for name in bufs:
        if bufs[name] is None and name in outputs:
            bufs[name] = torch.empty(shape, dtype=fdt, device=dev)
        _check(bufs[name], name, F, shape, dev, required=False)
    flags = _flags(time_major, multipass, inputs_ready=inputs_ready) | _fflag(fdt)
    _require_cuda(dev)
    with torch.cuda.device(dev):
        ws, wsb = _workspace(_lib.RLCA_EST_VALUE_TARGETS, E, T, 0, flags, dev, workspace)
        check("rlca_value_targets", lib.rlca_value_targets(
            _ptr(rewards), _ptr(values), _ptr(terminated), _ptr(truncated), _ptr(trunc_value), _ptr(bootstrap),
            _ptr(bufs["advantages"]), _ptr(bufs["returns"]), _ptr(bufs["disc_returns"]),
            _ptr(bufs["td_lambda_returns"]), E, T, gamma, lambda_, flags, _ptr(ws), wsb, _stream(dev, stream)))
        _hold(dev, stream, ws, *bufs.values())
    return bufs["advantages"], bufs["returns"], bufs["disc_returns"], bufs["td_lambda_returns"]


def rlca_discounted_return(rewards, terminated=None, truncated=None, trunc_value=None, bootstrap=None, *,
                           gamma=0.99, out=None, time_major=False, multipass=False, inputs_ready=False, workspace=None,
                           stream=None):
    """Discounted returns G_t = r_t + gamma * G_{t+1} with the boundary rules."""
    lib = _lib.load()
    dev = rewards.device
    fdt = _fdt(rewards, "rewards")
    F = (fdt,)
    E, T = _dims(rewards, time_major)
    shape = tuple(rewards.shape)
    _check(rewards, "rewards", F, shape, dev)
    _boundaries(shape, dev, terminated, truncated, trunc_value, bootstrap, E, F)
    if out is None:
        out = torch.empty(shape, dtype=fdt, device=dev)
    _check(out, "out", F, shape, dev)
    flags = _flags(time_major, multipass, inputs_ready=inputs_ready) | _fflag(fdt)
    _require_cuda(dev)
    with torch.cuda.device(dev):
        ws, wsb = _workspace(_lib.RLCA_EST_DISCOUNTED_RETURN, E, T, 0, flags, dev, workspace)
        check("rlca_discounted_return", lib.rlca_discounted_return(
            _ptr(rewards), _ptr(terminated), _ptr(truncated), _ptr(trunc_value), _ptr(bootstrap), _ptr(out),
            E, T, gamma, flags, _ptr(ws), wsb, _stream(dev, stream)))
        _hold(dev, stream, ws, out)
    return out


def rlca_td_lambda(rewards, values, terminated=None, truncated=None, trunc_value=None, bootstrap=None, *,
                   gamma=0.99, lambda_=0.95, out=None, time_major=False, multipass=False, inputs_ready=False, workspace=None,
                   stream=None):
    """TD(lambda) returns."""
    lib = _lib.load()
    dev = rewards.device
    fdt = _fdt(rewards, "rewards")
    F = (fdt,)
    E, T = _dims(rewards, time_major)
    shape = tuple(rewards.shape)
    _check(rewards, "rewards", F, shape, dev)
    _check(values, "values", F, shape, dev)
    _boundaries(shape, dev, terminated, truncated, trunc_value, bootstrap, E, F)
    if out is None:
        out = torch.empty(shape, dtype=fdt, device=dev)
    _check(out, "out", F, shape, dev)
    flags = _flags(time_major, multipass, inputs_ready=inputs_ready) | _fflag(fdt)
    _require_cuda(dev)
    with torch.cuda.device(dev):
        ws, wsb = _workspace(_lib.RLCA_EST_TD_LAMBDA, E, T, 0, flags, dev, workspace)
        check("rlca_td_lambda", lib.rlca_td_lambda(
            _ptr(rewards), _ptr(values), _ptr(terminated), _ptr(truncated), _ptr(trunc_value), _ptr(bootstrap),
            _ptr(out), E, T, gamma, lambda_, flags, _ptr(ws), wsb, _stream(dev, stream)))
        _hold(dev, stream, ws, out)
    return out


def rlca_vtrace(rewards, values, logp_target, logp_behaviour, terminated=None, truncated=None,
                trunc_value=None, bootstrap=None, *, gamma=0.99, rho_bar=1.0, c_bar=1.0, lambda_=1.0,
                vs=None, pg_advantages=None, want_pg=True, time_major=False, multipass=False, inputs_ready=False,
                workspace=None, stream=None):
    """V-Trace targets and policy-gradient advantages: ``(vs, pg_advantages)``."""
    lib = _lib.load()
    dev = rewards.device
    fdt = _fdt(rewards, "rewards")
    F = (fdt,)
    E, T = _dims(rewards, time_major)
    shape = tuple(rewards.shape)
    for name, t in (("rewards", rewards), ("values", values), ("logp_target", logp_target),
                    ("logp_behaviour", logp_behaviour)):
        _check(t, name, F, shape, dev)
    _boundaries(shape, dev, terminated, truncated, trunc_value, bootstrap, E, F)
    if vs is None:
        vs = torch.empty(shape, dtype=fdt, device=dev)
    if pg_advantages is None and want_pg:
        pg_advantages = torch.empty(shape, dtype=fdt, device=dev)
    _check(vs, "vs", F, shape, dev)
    _check(pg_advantages, "pg_advantages", F, shape, dev, required=False)
    flags = _flags(time_major, multipass, inputs_ready=inputs_ready) | _fflag(fdt)
    _require_cuda(dev)
    with torch.cuda.device(dev):
        ws, wsb = _workspace(_lib.RLCA_EST_VTRACE, E, T, 0, flags, dev, workspace)
        check("rlca_vtrace", lib.rlca_vtrace(
            _ptr(rewards), _ptr(values), _ptr(logp_target), _ptr(logp_behaviour), _ptr(terminated),
            _ptr(truncated), _ptr(trunc_value), _ptr(bootstrap), _ptr(vs), _ptr(pg_advantages), E, T,
            gamma, rho_bar, c_bar, lambda_, flags, _ptr(ws), wsb, _stream(dev, stream)))
        _hold(dev, stream, ws, vs, pg_advantages)
    return vs, pg_advantages


def rlca_retrace(q, pi, mu_a, actions, rewards, terminated=None, truncated=None, trunc_value=None,
                 bootstrap=None, *, gamma=0.99, lambda_=0.95, out=None, time_major=False, multipass=False, inputs_ready=False,
                 workspace=None, stream=None):
    """Retrace(lambda) Q targets; q and pi are [E, T, A] ([T, E, A])."""
    lib = _lib.load()
    dev = rewards.device
    fdt = _fdt(rewards, "rewards")
    F = (fdt,)
    E, T = _dims(rewards, time_major)
    shape = tuple(rewards.shape)
    if q.dim() != 3:
        raise ValueError("q must be 3-D")
    A = q.shape[-1]
    _check(q, "q", F, shape + (A,), dev)
    _check(pi, "pi", F, shape + (A,), dev)
    _check(mu_a, "mu_a", F, shape, dev)
    _check(actions, "actions", _I32, shape, dev)
    _check(rewards, "rewards", F, shape, dev)
    _boundaries(shape, dev, terminated, truncated, trunc_value, bootstrap, E, F)
    if out is None:
        out = torch.empty(shape, dtype=fdt, device=dev)
    _check(out, "out", F, shape, dev)
    flags = _flags(time_major, multipass, inputs_ready=inputs_ready) | _fflag(fdt)
    _require_cuda(dev)
    with torch.cuda.device(dev):
        ws, wsb = _workspace(_lib.RLCA_EST_RETRACE, E, T, A, flags, dev, workspace)
        check("rlca_retrace", lib.rlca_retrace(
            _ptr(q), _ptr(pi), _ptr(mu_a), _ptr(actions), _ptr(rewards), _ptr(terminated), _ptr(truncated),
            _ptr(trunc_value), _ptr(bootstrap), _ptr(out), E, T, A, gamma, lambda_, flags, _ptr(ws), wsb,
            _stream(dev, stream)))
        _hold(dev, stream, ws, out)
    return out


def rlca_elig_trace(x, terminated=None, truncated=None, *, gamma=0.99, lambda_=0.95, out=None,
                    time_major=False, multipass=False, inputs_ready=False, workspace=None, stream=None):
    """Accumulating eligibility trace (forward scan)."""
    lib = _lib.load()
    dev = x.device
    fdt = _fdt(x, "x")
    F = (fdt,)
    E, T = _dims(x, time_major)
    shape = tuple(x.shape)
    _check(x, "x", F, shape, dev)
    _check(terminated, "terminated", _U8, shape, dev, required=False)
    _check(truncated, "truncated", _U8, shape, dev, required=False)
    if out is None:
        out = torch.empty(shape, dtype=fdt, device=dev)
    _check(out, "out", F, shape, dev)
    flags = _flags(time_major, multipass, inputs_ready=inputs_ready) | _fflag(fdt)
    _require_cuda(dev)
    with torch.cuda.device(dev):
        ws, wsb = _workspace(_lib.RLCA_EST_ELIG_TRACE, E, T, 0, flags, dev, workspace)
        check("rlca_elig_trace", lib.rlca_elig_trace(
            _ptr(x), _ptr(terminated), _ptr(truncated), _ptr(out), E, T, gamma, lambda_, flags, _ptr(ws), wsb,
            _stream(dev, stream)))
        _hold(dev, stream, ws, out)
    return out


def rlca_episodic_prefix_sum(x, terminated=None, truncated=None, *, exclusive=False, flag_is_start=False,
                             out=None, time_major=False, multipass=False, inputs_ready=False, workspace=None, stream=None):
    """Per-episode running sum of x (int32 wraps; float32 or bfloat16 storage)."""
    lib = _lib.load()
    dev = x.device
    E, T = _dims(x, time_major)
    shape = tuple(x.shape)
    if x.dtype == torch.int32:
        dtype = _lib.RLCA_I32
    elif x.dtype in (torch.float32, torch.bfloat16):
        dtype = _lib.RLCA_F32
    else:
        raise TypeError("x must be int32, float32 or bfloat16")
    _check(x, "x", (x.dtype,), shape, dev)
    _check(terminated, "terminated", _U8, shape, dev, required=False)
    _check(truncated, "truncated", _U8, shape, dev, required=False)
    if out is None:
        out = torch.empty(shape, dtype=x.dtype, device=dev)
    _check(out, "out", (x.dtype,), shape, dev)
    extra = (_lib.RLCA_PSUM_EXCLUSIVE if exclusive else 0) | (_lib.RLCA_PSUM_FLAG_IS_START if flag_is_start else 0)
    flags = _flags(time_major, multipass, extra, inputs_ready=inputs_ready) | (
        _lib.RLCA_BF16 if x.dtype == torch.bfloat16 else 0)
    _require_cuda(dev)
    with torch.cuda.device(dev):
        ws, wsb = _workspace(_lib.RLCA_EST_PREFIX_SUM, E, T, 0, flags, dev, workspace)
        check("rlca_episodic_prefix_sum", lib.rlca_episodic_prefix_sum(
            _ptr(x), dtype, _ptr(terminated), _ptr(truncated), _ptr(out), E, T, flags, _ptr(ws), wsb,
            _stream(dev, stream)))
        _hold(dev, stream, ws, out)
    return out


def rlca_affine_scan(alpha, beta, carry=None, *, reverse=True, out=None, time_major=False, multipass=False, inputs_ready=False,
                     workspace=None, stream=None):
    """Generic A_t = alpha_t + beta_t * A_{t+1} (reverse) or A_{t-1} (forward)."""
    lib = _lib.load()
    dev = alpha.device
    fdt = _fdt(alpha, "alpha")
    F = (fdt,)
    E, T = _dims(alpha, time_major)
    shape = tuple(alpha.shape)
    _check(alpha, "alpha", F, shape, dev)
    _check(beta, "beta", F, shape, dev)
    _check(carry, "carry", F, (E,), dev, required=False)
    if out is None:
        out = torch.empty(shape, dtype=fdt, device=dev)
    _check(out, "out", F, shape, dev)
    flags = _flags(time_major, multipass, inputs_ready=inputs_ready) | _fflag(fdt)
    _require_cuda(dev)
    with torch.cuda.device(dev):
        ws, wsb = _workspace(_lib.RLCA_EST_AFFINE_SCAN, E, T, 0, flags, dev, workspace)
        check("rlca_affine_scan", lib.rlca_affine_scan(
            _ptr(alpha), _ptr(beta), _ptr(carry), _ptr(out), E, T, 1 if reverse else 0, flags, _ptr(ws), wsb,
            _stream(dev, stream)))
        _hold(dev, stream, ws, out)
    return out


# ---- the policy update around the scans ------------------------------------
# Matrices here are 2-D with contiguous rows at any row stride (a slice of a
# wider buffer works); everything else is contiguous as above.  Small calls
# cost more on the host than on the device, so the checks take one combined
# test on the common path and the device is only switched when it is not the
# current one.

def _check_matrix(t, name, dtype, shape, device):
    """Checks a matrix input and returns its row stride in elements."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype}")
    got = t.shape
    if len(got) != 2 or (shape is not None and got != shape):
        raise ValueError(f"{name}: shape {tuple(got)}, expected {tuple(shape) if shape else '2 dimensions'}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    rows, width = got
    row_stride, stride = t.stride()
    if width > 1 and stride != 1:
        raise ValueError(f"{name} must have contiguous rows")
    if rows <= 1:
        return width
    if row_stride < width:
        raise ValueError(f"{name}: rows overlap (row stride {row_stride} below width {width})")
    return row_stride


def _out(t, name, dtype, shape, device, want=True):
    """An output buffer: the one given (checked), a new one, or None."""
    if t is None:
        return torch.empty(shape, dtype=dtype, device=device) if want else None
    _check(t, name, (dtype,), shape, device)
    return t


class _Here:
    """The device guard of a call whose device is the current one already."""
    def __enter__(self):
        return None

    def __exit__(self, *exc):
        return False


_here = _Here()


def _on(device):
    return _here if device.index == torch.cuda.current_device() else torch.cuda.device(device)


def _raw_stream(device, stream):
    # the handle of the current stream without building a Stream object
    return stream.cuda_stream if stream is not None else torch._C._cuda_getCurrentRawStream(device.index)


def rlca_layer_norm(x, weight, bias=None, *, eps=1e-5, y=None, mean=None, rstd=None, stream=None):
    """Layer norm of the rows of ``x`` [N, D]: ``(y, mean, rstd)``, the
    statistics float32 for :func:`rlca_layer_norm_backward`."""
    lib = _lib.load()
    fdt = _fdt(x, "x")
    dev = x.device
    stride = _check_matrix(x, "x", fdt, None, dev)
    N, D = x.shape
    _check(weight, "weight", (fdt,), (D,), dev)
    _check(bias, "bias", (fdt,), (D,), dev, required=False)
    y = _out(y, "y", fdt, (N, D), dev)
    mean = _out(mean, "mean", torch.float32, (N,), dev)
    rstd = _out(rstd, "rstd", torch.float32, (N,), dev)
    _require_cuda(dev)
    with _on(dev):
        check("rlca_layer_norm", lib.rlca_layer_norm(
            x.data_ptr(), weight.data_ptr(), _ptr(bias), y.data_ptr(), mean.data_ptr(), rstd.data_ptr(), N, D, stride,
            eps, _fflag(fdt), _raw_stream(dev, stream)))
        _hold(dev, stream, y, mean, rstd)
    return y, mean, rstd


def rlca_layer_norm_backward(dy, x, weight, mean, rstd, *, dx=None, dweight=None, dbias=None, want_dx=True,
                             want_dweight=True, want_dbias=True, workspace=None, stream=None):
    """Gradient of :func:`rlca_layer_norm`: ``(dx, dweight, dbias)`` (None
    for those not wanted; at least one is)."""
    lib = _lib.load()
    fdt = _fdt(x, "x")
    dev = x.device
    x_stride = _check_matrix(x, "x", fdt, None, dev)
    N, D = x.shape
    dy_stride = _check_matrix(dy, "dy", fdt, (N, D), dev)
    _check(weight, "weight", (fdt,), (D,), dev)
    _check(mean, "mean", _F, (N,), dev)
    _check(rstd, "rstd", _F, (N,), dev)
    dx = _out(dx, "dx", fdt, (N, D), dev, want_dx)
    dweight = _out(dweight, "dweight", fdt, (D,), dev, want_dweight)
    dbias = _out(dbias, "dbias", fdt, (D,), dev, want_dbias)
    if dx is None and dweight is None and dbias is None:
        raise ValueError("no output wanted")
    _require_cuda(dev)
    flags = _fflag(fdt)
    with _on(dev):
        ws, wsb = _workspace(_lib.RLCA_EST_LAYER_NORM_BACKWARD, N, D, 0, flags, dev, workspace)
        check("rlca_layer_norm_backward", lib.rlca_layer_norm_backward(
            dy.data_ptr(), x.data_ptr(), weight.data_ptr(), mean.data_ptr(), rstd.data_ptr(), _ptr(dx), _ptr(dweight),
            _ptr(dbias), N, D, dy_stride, x_stride, flags, _ptr(ws), wsb, _raw_stream(dev, stream)))
        _hold(dev, stream, ws, dx, dweight, dbias)
    return dx, dweight, dbias


def _check_head(hidden, weight, tokens, temperature):
    fdt = _fdt(hidden, "hidden")
    dev = hidden.device
    hidden_stride = _check_matrix(hidden, "hidden", fdt, None, dev)
    N, D = hidden.shape
    weight_stride = _check_matrix(weight, "weight", fdt, None, dev)
    V, width = weight.shape
    if width != D:
        raise ValueError(f"weight: shape {(V, width)}, expected (vocabulary, {D})")
    _check(tokens, "tokens", _I32, (N,), dev)
    if not temperature > 0.0:
        raise ValueError(f"temperature {temperature} must be positive")
    return fdt, dev, N, D, V, hidden_stride, weight_stride


def rlca_token_logprob(hidden, weight, tokens, *, temperature=1.0, logp=None, lse=None, entropy=None,
                       want_entropy=True, workspace=None, stream=None):
    """Log-probabilities of ``tokens`` [N] (int32) under the policy
    softmax(hidden [N, D] weight [V, D]^T / temperature), without storing
    the logits: ``(logp, lse, entropy)``, float32, entropy None when not
    wanted.  -logp is the cross entropy.  A row whose token lies outside
    [0, V) takes no part: its results are 0."""
    lib = _lib.load()
    fdt, dev, N, D, V, hs, wst = _check_head(hidden, weight, tokens, temperature)
    logp = _out(logp, "logp", torch.float32, (N,), dev)
    lse = _out(lse, "lse", torch.float32, (N,), dev)
    entropy = _out(entropy, "entropy", torch.float32, (N,), dev, want_entropy)
    _require_cuda(dev)
    flags = _fflag(fdt)
    with _on(dev):
        ws, wsb = _workspace(_lib.RLCA_EST_TOKEN_LOGPROB, N, D, V, flags, dev, workspace)
        check("rlca_token_logprob", lib.rlca_token_logprob(
            hidden.data_ptr(), weight.data_ptr(), tokens.data_ptr(), logp.data_ptr(), lse.data_ptr(), _ptr(entropy), N,
            D, V, hs, wst, 1.0 / temperature, flags, _ptr(ws), wsb, _raw_stream(dev, stream)))
        _hold(dev, stream, ws, logp, lse, entropy)
    return logp, lse, entropy


def rlca_token_logprob_backward(hidden, weight, tokens, lse, d_logp, *, entropy=None, d_entropy=None,
                                temperature=1.0, d_hidden=None, d_weight=None, want_d_hidden=True,
                                want_d_weight=True, workspace=None, stream=None):
    """Gradient of :func:`rlca_token_logprob` for the factors ``d_logp`` [N]
    and, with the saved ``entropy``, ``d_entropy`` [N] (float32):
    ``(d_hidden, d_weight)``, None for one not wanted (at least one is).
    bfloat16, more than 128 rows: the logits' gradient is rounded to bfloat16
    before its two products."""
    lib = _lib.load()
    fdt, dev, N, D, V, hs, wst = _check_head(hidden, weight, tokens, temperature)
    rows = (N,)
    _check(lse, "lse", _F, rows, dev)
    _check(d_logp, "d_logp", _F, rows, dev)
    if (entropy is None) != (d_entropy is None):
        raise ValueError("entropy and d_entropy come together")
    if entropy is not None:
        _check(entropy, "entropy", _F, rows, dev)
        _check(d_entropy, "d_entropy", _F, rows, dev)
    d_hidden = _out(d_hidden, "d_hidden", fdt, (N, D), dev, want_d_hidden)
    d_weight = _out(d_weight, "d_weight", fdt, (V, D), dev, want_d_weight)
    if d_hidden is None and d_weight is None:
        raise ValueError("no output wanted")
    _require_cuda(dev)
    flags = _fflag(fdt)
    with _on(dev):
        ws, wsb = _workspace(_lib.RLCA_EST_TOKEN_LOGPROB_BACKWARD, N, D, V, flags, dev, workspace)
        check("rlca_token_logprob_backward", lib.rlca_token_logprob_backward(
            hidden.data_ptr(), weight.data_ptr(), tokens.data_ptr(), lse.data_ptr(), _ptr(entropy), d_logp.data_ptr(),
            _ptr(d_entropy), _ptr(d_hidden), _ptr(d_weight), N, D, V, hs, wst, 1.0 / temperature, flags, _ptr(ws), wsb,
            _raw_stream(dev, stream)))
        _hold(dev, stream, ws, d_hidden, d_weight)
    return d_hidden, d_weight


_GRAD_FLAGS = {torch.float32: 0, torch.bfloat16: _lib.RLCA_BF16}


def _address(a):
    return a.buffer_info()[0]


def rlca_clip_grads(grads, max_norm, *, eps=1e-6, out=None, norm_only=False, norm=None, workspace=None, stream=None):
    """Global norm of the gradient tensors ``grads`` (each float32 or
    bfloat16, any shape) and the tensors times min(1, max_norm / (norm +
    eps)) -- unscaled when the norm is not finite: ``(clipped, norm)``, norm
    a float32 scalar tensor.  ``out`` takes the results: a list of tensors of
    the same types and element counts, or ``grads`` itself to scale in
    place.  ``norm_only`` leaves the
    tensors alone and returns ``(None, norm)``."""
    lib = _lib.load()
    grads = list(grads)
    if norm is None and not grads:
        raise ValueError("no gradients and no norm buffer: the device is unknown")
    n = len(grads)
    for k, g in enumerate(grads):
        if not isinstance(g, torch.Tensor):
            raise TypeError(f"grads[{k}] must be a torch.Tensor")
    dev = grads[0].device if grads else norm.device
    # the checks over whole lists; one that fails is looked for tensor by tensor
    flags = [_GRAD_FLAGS.get(g.dtype) for g in grads]
    if None in flags or not (all([g.device == dev for g in grads]) and all(map(torch.Tensor.is_contiguous, grads))):
        for k, g in enumerate(grads):
            _check(g, f"grads[{k}]", (_fdt(g, f"grads[{k}]"),), g.shape, dev)
    sizes = array("q", map(torch.Tensor.numel, grads))
    if norm_only:
        out = None
    elif out is None:
        out = [torch.empty_like(g, memory_format=torch.contiguous_format) for g in grads]
    else:
        out = list(out)
        if len(out) != n:
            raise ValueError(f"out has {len(out)} tensors, expected {n}")
        if not all(map(operator.is_, out, grads)):
            if not (all([isinstance(o, torch.Tensor) for o in out]) and [_GRAD_FLAGS.get(o.dtype) for o in out] == flags
                    and array("q", map(torch.Tensor.numel, out)) == sizes and all([o.device == dev for o in out])
                    and all(map(torch.Tensor.is_contiguous, out))):
                for k, (g, o) in enumerate(zip(grads, out)):
                    _check(o, f"out[{k}]", (g.dtype,), g.shape, dev)
                raise ValueError("out does not match grads")
    norm = _out(norm, "norm", torch.float32, (), dev)
    _require_cuda(dev)
    # host arrays that the call reads before it returns
    gp = array("Q", map(torch.Tensor.data_ptr, grads))
    op = None if out is None else array("Q", map(torch.Tensor.data_ptr, out))
    dtypes = array("I", flags)
    with _on(dev):
        ws, wsb = _workspace(_lib.RLCA_EST_CLIP_GRADS, n, 1, 0, 0, dev, workspace)
        check("rlca_clip_grads", lib.rlca_clip_grads(
            _address(gp), None if op is None else _address(op), _address(sizes), _address(dtypes), n, max_norm, eps,
            norm.data_ptr(), _ptr(ws), wsb, _raw_stream(dev, stream)))
        _hold(dev, stream, ws, norm, *(out or ()))
    return out, norm
