"""The policy-update operators on the GPU against the 64-bit reference.

Tolerances, set before the first run, with u = 2^-23 (float32, truncation
allowed) and r = 2^-8 (bfloat16 has 8 significant bits: half a unit of the
last place is up to 2^-8 of the value):

* a dot product of K terms in float32 is off by at most
  (4 sqrt(K) + 32) u times the sum of its terms' magnitudes: rounding errors
  of either sign, four standard deviations, and a margin of 32 roundings for
  what stands around it (splits, joins, the exponential);
* logp and lse are off by that for K = D at the largest such sum over the
  vocabulary, plus 8 u (1 + |value|) for the logarithm and the exponentials;
  the entropy by as much times 2 (1 + |lse| + |entropy| + scale's share of
  the spread), because its sensitivity to a logit is p |log p + H|;
* the gradients contract dz (magnitude M, known to the reference): relative
  2 (1 + spread) times the logits' error, one rounding of dz to bfloat16
  (r; none in float32), the dot product's own error, all times M's
  contraction, and one rounding of the result;
* in the 2-norm, where the roundings of dz are independent: r times the root
  of the sum of squares along the contraction in place of the sum of
  magnitudes;
* layer norm: a row's sums as dot products of K = D terms over the centred
  or widened row, one rounding of the result.
"""
import math

import pytest
import torch

from first_order_linear_gb300 import _lib, rlca
from oracle import policy_ref as ref

pytestmark = pytest.mark.gpu

U, R = 2.0 ** -23, 2.0 ** -8
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(autouse=True)
def _lib_ready(cuda_lib):
    yield
    torch.cuda.synchronize()
    import ctypes as C
    st = C.c_uint(0)
    assert cuda_lib.rlca_device_status(C.byref(st), 0) == 0 and st.value == 0


def dot_err(K):
    return (4.0 * math.sqrt(K) + 32.0) * U


def rounding(dtype):
    return R if dtype == torch.bfloat16 else U


def check(got, want, tol, what):
    got, want = got.double(), want.double()
    if got.numel() == 0:
        return
    assert torch.isfinite(got).all(), f"{what}: not finite"
    excess = ((got - want).abs() - tol)
    k = int(excess.argmax())
    assert excess.max().item() <= 0, (
        f"{what}: {got.reshape(-1)[k].item()} against {want.reshape(-1)[k].item()} at {k}, over by {excess.max().item()}")


def rand(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda")


def head_inputs(N, D, V, dtype, seed, mask=0.0, strided=False, shift=False, junk=False):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    w = rand(gen, V, D) * (2.0 / math.sqrt(D))
    taken = torch.randint(0, V, (N,), generator=gen, device="cuda")
    lean = 2.0 * torch.rand((N, 1), generator=gen, device="cuda")
    h = rand(gen, N, D) + lean * w[taken]
    tok = taken.to(torch.int32)
    if mask:
        off = torch.rand(N, generator=gen, device="cuda") < mask
        tok[off] = torch.where(torch.rand(N, generator=gen, device="cuda") < 0.5, -1, V).to(torch.int32)[off]
        if junk:
            h[off, 0], h[off, D - 1] = float("nan"), float("inf")
    h, w = h.to(dtype), w.to(dtype)
    if strided:  # rows of wider buffers whose pad holds NaN
        hb = torch.full((N, D + 5), float("nan"), device="cuda", dtype=dtype)
        wb = torch.full((V, D + 3), float("nan"), device="cuda", dtype=dtype)
        hb[:, 2:D + 2], wb[:, 1:D + 1] = h, w
        h, w = hb[:, 2:D + 2], wb[:, 1:D + 1]
    if shift:  # bases one element off
        def off1(t):
            b = torch.empty(t.numel() + 1, device="cuda", dtype=dtype)[1:].view(t.shape)
            return b.copy_(t)
        h, w = off1(h), off1(w)
    g, e = rand(gen, N) / max(1, N), 0.1 * rand(gen, N) / max(1, N)
    return h, w, tok, g, e


def check_head(N, D, V, dtype, seed=0, temperature=1.0, entropy=True, stream=None, **kw):
    h, w, tok, g, e = head_inputs(N, D, V, dtype, seed, **kw)
    logp0, lse0, ent0, scale = ref.token_logprob(h, w, tok, temperature)
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    logp, lse, ent = rlca.rlca_token_logprob(h, w, tok, temperature=temperature, want_entropy=entropy, stream=stream)
    # the gradient is tested on the reference's rounded statistics
    lse32, ent32 = lse0.float(), ent0.float()
    d_h, d_w = rlca.rlca_token_logprob_backward(
        h, w, tok, lse32, g, entropy=ent32 if entropy else None, d_entropy=e if entropy else None,
        temperature=temperature, stream=stream)
    if stream is not None:
        torch.cuda.current_stream().wait_stream(stream)
    zerr = dot_err(D) * scale
    part = (tok >= 0) & (tok < V)
    for got, want, name in ((logp, logp0, "logp"), (lse, lse0, "lse")):
        check(got, want, torch.where(part, 2 * zerr + 8 * U * (1 + want.abs() + lse0.abs()), 0.0), name)
    spread = 1 + lse0.abs() + ent0.abs() + 2 * scale.clamp(max=64.0)
    if entropy:
        check(ent, ent0, torch.where(part, 2 * (zerr + 8 * U) * spread, 0.0), "entropy")
    dh0, dw0, bh, bw, rh, rw = ref.token_logprob_backward(h, w, tok, lse32, g, ent32 if entropy else None,
                                                          e if entropy else None, temperature)
    rz = 2 * (float(zerr.max()) + 8 * U) * 2
    rd, out = (R if dtype == torch.bfloat16 else 0.0), rounding(dtype)
    for got, want, bound, root, K, name in ((d_h, dh0, bh, rh, V, "d_hidden"), (d_w, dw0, bw, rw, N, "d_weight")):
        check(got, want, bound * (rz + rd + dot_err(K)) + want.abs() * out, name)
        far = (got.double() - want).norm()
        assert far <= bound.norm() * (rz + dot_err(K)) + root.norm() * rd + want.norm() * out, (name, float(far))
    return logp, lse, ent, d_h, d_w


HEAD_SIZES = [
    (1, 1, 1), (1, 64, 2), (3, 8, 17), (5, 7, 11), (37, 200, 1003), (64, 64, 64), (65, 129, 257), (127, 128, 255),
    (128, 512, 1000), (129, 136, 256), (257, 1030, 300), (300, 96, 4097), (1000, 72, 511), (513, 320, 1537),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,D,V", HEAD_SIZES)
def test_head(N, D, V, dtype):
    check_head(N, D, V, DT[dtype], seed=N + D + V)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kw", [dict(), dict(mask=0.5, junk=True), dict(strided=True), dict(shift=True)])
@pytest.mark.parametrize("N,D,V", [(1, 1024, 9001), (2, 100, 300), (4, 64, 31), (5, 256, 1003), (7, 129, 77),
                                   (8, 512, 2500), (8, 4096, 1000), (9, 512, 2500)])
def test_head_few_rows(N, D, V, kw, dtype):
    check_head(N, D, V, DT[dtype], seed=N + D, **kw)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("mask,junk", [(0.4, False), (0.4, True), (0.95, True), (1.1, True)])
@pytest.mark.parametrize("N,D,V", [(9, 24, 40), (200, 128, 700), (385, 72, 300)])
def test_head_rows_that_take_no_part(N, D, V, mask, junk, dtype):
    """Masked rows give zeros and add nothing, whatever they hold; mask 1.1 leaves no row."""
    check_head(N, D, V, DT[dtype], seed=7, mask=mask, junk=junk)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kw", [dict(strided=True), dict(shift=True), dict(temperature=0.7), dict(temperature=3.0),
                                dict(entropy=False)])
@pytest.mark.parametrize("N,D,V", [(70, 64, 130), (33, 100, 515)])
def test_head_strides_alignment_temperature(N, D, V, kw, dtype):
    check_head(N, D, V, DT[dtype], seed=11, **kw)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_head_several_pieces_of_the_vocabulary(dtype):
    """dz of the whole vocabulary is 0.4 GB at two bytes an element: the gradient runs in pieces."""
    check_head(3000, 40, 70001, DT[dtype], seed=3, mask=0.2)


def test_head_pieces_beyond_a_gigabyte():
    """dz of the whole vocabulary is 1.15 GB at two bytes an element."""
    check_head(8192, 24, 70001, torch.bfloat16, seed=4, mask=0.1)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_head_many_rows(dtype):
    """More rows than the first kernel's CTAs take in one round."""
    check_head(200003, 8, 20, DT[dtype], seed=8, mask=0.3, junk=True)


def test_head_on_another_stream():
    check_head(150, 96, 600, torch.bfloat16, seed=5, stream=torch.cuda.Stream())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_head_repeats_bit_for_bit(dtype):
    a = check_head(600, 256, 3001, DT[dtype], seed=6, mask=0.3)
    b = check_head(600, 256, 3001, DT[dtype], seed=6, mask=0.3)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_head_given_workspace(dtype):
    """A workspace of exactly the size asked for, on a 16-byte boundary that is no more than that."""
    N, D, V = 200, 104, 700
    h, w, tok, g, e = head_inputs(N, D, V, DT[dtype], 12, mask=0.3)
    flags = _lib.RLCA_BF16 if dtype == "bf16" else 0

    def space(est):
        n = rlca.rlca_workspace_size(est, N, D, V, flags)
        return torch.full((n + 32,), 255, dtype=torch.uint8, device="cuda")[16:16 + n]
    want = rlca.rlca_token_logprob(h, w, tok)
    got = rlca.rlca_token_logprob(h, w, tok, workspace=space(_lib.RLCA_EST_TOKEN_LOGPROB))
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    kw = dict(entropy=want[2], d_entropy=e)
    ref_grads = rlca.rlca_token_logprob_backward(h, w, tok, want[1], g, **kw)
    got = rlca.rlca_token_logprob_backward(h, w, tok, want[1], g, workspace=space(_lib.RLCA_EST_TOKEN_LOGPROB_BACKWARD), **kw)
    assert all(torch.equal(a, b) for a, b in zip(ref_grads, got))
    with pytest.raises(ValueError):
        rlca.rlca_token_logprob(h, w, tok, workspace=space(_lib.RLCA_EST_TOKEN_LOGPROB)[:-16])


def test_head_one_output_only():
    h, w, tok, g, e = head_inputs(90, 64, 300, torch.bfloat16, 2)
    logp, lse, ent = rlca.rlca_token_logprob(h, w, tok)
    both = rlca.rlca_token_logprob_backward(h, w, tok, lse, g, entropy=ent, d_entropy=e)
    only_h = rlca.rlca_token_logprob_backward(h, w, tok, lse, g, entropy=ent, d_entropy=e, want_d_weight=False)
    only_w = rlca.rlca_token_logprob_backward(h, w, tok, lse, g, entropy=ent, d_entropy=e, want_d_hidden=False)
    assert only_h[1] is None and only_w[0] is None
    assert torch.equal(only_h[0], both[0]) and torch.equal(only_w[1], both[1])


def test_head_no_rows():
    w = torch.randn(10, 16, device="cuda")
    h, tok = torch.empty(0, 16, device="cuda"), torch.empty(0, dtype=torch.int32, device="cuda")
    logp, lse, ent = rlca.rlca_token_logprob(h, w, tok)
    assert logp.shape == (0,)
    z = torch.empty(0, device="cuda")
    dh, dw = rlca.rlca_token_logprob_backward(h, w, tok, z, z)
    assert dh.shape == (0, 16) and dw.abs().max() == 0


def test_head_offsets_past_32_bits():
    """2 rows against a weight of 2^32 and some elements: the last tokens' logits, probabilities and gradient rows."""
    N, D, V = 2, 65536, 65600
    gen = torch.Generator(device="cuda")
    gen.manual_seed(0)
    w = torch.zeros(V, D, device="cuda", dtype=torch.bfloat16)
    live = torch.tensor([0, 1, 40000, V - 2, V - 1], device="cuda")
    rows = (rand(gen, len(live), D) * (2.0 / math.sqrt(D))).to(torch.bfloat16)
    w[live] = rows
    h = rand(gen, N, D).to(torch.bfloat16)
    tok = torch.tensor([V - 1, V - 2], dtype=torch.int32, device="cuda")
    g = torch.tensor([1.0, -0.5], device="cuda")
    logp, lse, _ = rlca.rlca_token_logprob(h, w, tok)
    z = h.double() @ rows.double().t()
    rest = (V - len(live)) * torch.ones(N, dtype=torch.float64, device="cuda")
    lse0 = torch.log(torch.exp(z).sum(1) + rest)
    logp0 = torch.stack([z[0, 4], z[1, 3]]) - lse0
    scale = (h.double().abs() @ rows.double().abs().t()).amax(1)
    tol = 2 * dot_err(D) * scale + 8 * U * (1 + 2 * lse0.abs())
    check(lse, lse0, tol, "lse")
    check(logp, logp0, tol, "logp")
    _, dw = rlca.rlca_token_logprob_backward(h, w, tok, lse, g, want_d_hidden=False)
    p = torch.exp(z - lse0[:, None])
    hot = torch.zeros_like(p)
    hot[0, 4] = hot[1, 3] = 1.0
    dz = g.double()[:, None] * (hot - p)
    want = dz.t() @ h.double()
    bound = (g.double().abs()[:, None] * (hot + p)).t() @ h.double().abs()
    check(dw[live], want, bound * (4 * float(tol.max()) + R + dot_err(N)) + want.abs() * R, "d_weight")


# ---- layer norm ----------------------------------------------------------------

def check_norm(N, D, dtype, seed=0, bias=True, strided=False, shift=False, eps=1e-5, offset=0.5, stream=None):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    x = (1.5 * rand(gen, N, D) + offset * rand(gen, N, 1)).to(dtype)
    dy = rand(gen, N, D).to(dtype)
    w, b = (1 + 0.1 * rand(gen, D)).to(dtype), (0.1 * rand(gen, D)).to(dtype) if bias else None
    if strided:
        xb = torch.full((N, D + 3), float("nan"), device="cuda", dtype=dtype)
        db_ = torch.full((N, D + 8), float("nan"), device="cuda", dtype=dtype)
        xb[:, 1:D + 1], db_[:, 8:] = x, dy
        x, dy = xb[:, 1:D + 1], db_[:, 8:]
    if shift:
        x = torch.empty(x.numel() + 1, device="cuda", dtype=dtype)[1:].view(N, D).copy_(x)
        dy = torch.empty(dy.numel() + 1, device="cuda", dtype=dtype)[1:].view(N, D).copy_(dy)
    y0, mean0, rstd0 = ref.layer_norm(x, w, b, eps)
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    y, mean, rstd = rlca.rlca_layer_norm(x, w, b, eps=eps, stream=stream)
    mean32, rstd32 = mean0.float(), rstd0.float()
    dx, dw, db = rlca.rlca_layer_norm_backward(dy, x, w, mean32, rstd32, stream=stream)
    if stream is not None:
        torch.cuda.current_stream().wait_stream(stream)
    xa, wa = x.double().abs(), w.double().abs()
    out = rounding(dtype)
    merr = dot_err(D) * xa.mean(1)
    check(mean, mean0, merr + U * mean0.abs(), "mean")
    # the centred row is off by the mean's error; its mean square by twice that over the spread
    rerr = rstd0 * (dot_err(D) + 2 * merr * rstd0)
    check(rstd, rstd0, rerr + 4 * U * rstd0, "rstd")
    xh = (x.double() - mean0[:, None]).abs() * rstd0[:, None]
    yerr = ((merr * rstd0)[:, None] + xh * (rerr / rstd0)[:, None] + 8 * U * (xh + xa * rstd0[:, None])) * wa
    check(y, y0, yerr + 8 * U * (0 if b is None else b.double().abs()) + y0.abs() * out, "y")
    dx0, dw0, db0 = ref.layer_norm_backward(dy, x, w, mean32, rstd32)
    g = dy.double().abs() * wa
    xhe = 4 * U * (xh + xa * rstd0[:, None])  # the normalised row's own rounding
    derr = dot_err(D) * (g + g.mean(1, keepdim=True) + xh * (g * xh).mean(1, keepdim=True))
    derr = derr + xhe * (g * xh).mean(1, keepdim=True) + xh * (g * xhe).mean(1, keepdim=True)
    check(dx, dx0, rstd0[:, None] * derr + dx0.abs() * out, "dx")
    da = dy.double().abs()
    check(dw, dw0, dot_err(N) * (da * xh).sum(0) + (da * xhe).sum(0) + dw0.abs() * out, "dweight")
    check(db, db0, dot_err(N) * da.sum(0) + db0.abs() * out, "dbias")
    return y, mean, rstd, dx, dw, db


NORM_SIZES = [(1, 1), (1, 2), (2, 3), (8, 1024), (7, 31), (33, 32), (5, 33), (64, 257), (100, 1001), (1000, 64),
              (300, 4096), (40, 4097), (17, 8192), (9, 8200), (3, 20000), (4099, 129), (2, 65536), (700, 5001), (31, 8191), (600, 8192), (33, 16384)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,D", NORM_SIZES)
def test_norm(N, D, dtype):
    check_norm(N, D, DT[dtype], seed=N + D)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kw", [dict(strided=True), dict(shift=True), dict(bias=False), dict(eps=0.0),
                                dict(offset=100.0)])
@pytest.mark.parametrize("N,D", [(21, 64), (50, 1000), (6, 5000)])
def test_norm_strides_alignment_offsets(N, D, kw, dtype):
    check_norm(N, D, DT[dtype], seed=1, **kw)


def test_norm_on_another_stream_and_repeats():
    a = check_norm(700, 512, torch.bfloat16, seed=2, stream=torch.cuda.Stream())
    b = check_norm(700, 512, torch.bfloat16, seed=2)
    assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_norm_constant_rows():
    """A row without spread: rstd is 1 / sqrt(eps), y the bias."""
    x = torch.full((5, 48), 3.25, device="cuda")
    w, b = torch.ones(48, device="cuda"), torch.arange(48.0, device="cuda")
    y, mean, rstd = rlca.rlca_layer_norm(x, w, b, eps=1e-4)
    assert torch.equal(mean, torch.full((5,), 3.25, device="cuda"))
    assert (rstd - 100.0).abs().max() < 1e-4 and torch.equal(y, b.expand(5, 48))


def test_norm_rows_with_nan_stay_apart():
    x = torch.randn(6, 200, device="cuda")
    clean = rlca.rlca_layer_norm(x, torch.ones(200, device="cuda"))[0]
    x[2, 17], x[4, 0] = float("nan"), float("inf")
    y = rlca.rlca_layer_norm(x, torch.ones(200, device="cuda"))[0]
    keep = torch.tensor([0, 1, 3, 5], device="cuda")
    assert torch.equal(y[keep], clean[keep]) and torch.isnan(y[[2, 4]]).all()


def test_norm_empty():
    w = torch.ones(12, device="cuda")
    y, mean, rstd = rlca.rlca_layer_norm(torch.empty(0, 12, device="cuda"), w)
    assert y.shape == (0, 12)
    e = torch.empty(0, 12, device="cuda")
    dx, dw, db = rlca.rlca_layer_norm_backward(e, e, w, mean, rstd)
    assert dx.shape == (0, 12) and dw.abs().max() == 0 and db.abs().max() == 0


def test_norm_only_wanted_outputs():
    x, dy, w = torch.randn(50, 96, device="cuda"), torch.randn(50, 96, device="cuda"), torch.ones(96, device="cuda")
    _, mean, rstd = rlca.rlca_layer_norm(x, w)
    full = rlca.rlca_layer_norm_backward(dy, x, w, mean, rstd)
    for k in range(3):
        want = dict(want_dx=k == 0, want_dweight=k == 1, want_dbias=k == 2)
        got = rlca.rlca_layer_norm_backward(dy, x, w, mean, rstd, **want)
        assert torch.equal(got[k], full[k]) and all(got[j] is None for j in range(3) if j != k)


def test_norm_offsets_past_32_bits():
    N, D = 70000, 65536  # 2^32 elements and some
    gen = torch.Generator(device="cuda")
    gen.manual_seed(4)
    x = torch.zeros(N, D, device="cuda", dtype=torch.bfloat16)
    last = rand(gen, 3, D).to(torch.bfloat16)
    x[N - 3:] = last
    w = (1 + 0.1 * rand(gen, D)).to(torch.bfloat16)
    y, mean, rstd = rlca.rlca_layer_norm(x, w)
    y0, mean0, rstd0 = ref.layer_norm(last, w, None, 1e-5)
    tol = dot_err(D) * (1 + last.double().abs()) * 4 + y0.abs() * R
    check(y[N - 3:], y0, tol, "y")
    assert y[:N - 3].abs().max() == 0
    dx, _, _ = rlca.rlca_layer_norm_backward(x, x, w, mean, rstd, want_dweight=False, want_dbias=False)
    dx0, _, _ = ref.layer_norm_backward(last, last, w, mean[N - 3:], rstd[N - 3:])
    check(dx[N - 3:], dx0, dot_err(D) * 8 * (1 + last.double().abs()) * rstd0[:, None] + dx0.abs() * R, "dx")


# ---- clipping --------------------------------------------------------------------

def grads_of(sizes, seed=0, scale=1.0, mixed=True, shift=False):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    out = []
    for k, n in enumerate(sizes):
        dt = torch.bfloat16 if mixed and k % 2 else torch.float32
        t = torch.empty(n + 1, device="cuda", dtype=dt)[1:] if shift else torch.empty(n, device="cuda", dtype=dt)
        out.append(t.copy_(rand(gen, n) * scale))
    return out


def check_clip(grads, max_norm, **kw):
    want, norm0, scale = ref.clip_grads(grads, max_norm)
    before = [g.clone() for g in grads]
    got, norm = rlca.rlca_clip_grads(grads, max_norm, **kw)
    # squares: float32 over runs of at most a few thousand elements of one sign of error each, halved by the root
    assert abs(norm.item() - norm0.item()) <= 32 * U * norm0.item() + 1e-37, (norm.item(), norm0.item())
    for g, w, b in zip(got, want, before):
        check(g, w, w.abs() * (34 * U + rounding(b.dtype)) + 1e-40, "clipped")
    return got, norm, before


@pytest.mark.parametrize("scale,max_norm", [(1.0, 1.0), (1e-3, 1e6), (1e4, 0.5), (1.0, 0.0), (1.0, math.inf)])
@pytest.mark.parametrize("shift", [False, True])
def test_clip(scale, max_norm, shift):
    sizes = [1, 3, 8, 17, 1000, 4096, 32768, 32769, 100001, 1 << 20]
    check_clip(grads_of(sizes, seed=1, scale=scale, shift=shift), max_norm)


def test_clip_in_place_and_norm_only():
    grads = grads_of([5, 70000, 333], seed=2)
    alone = rlca.rlca_clip_grads(grads, 1.0, norm_only=True)
    got, norm, before = check_clip(grads, 1.0, out=grads)
    assert alone[0] is None and torch.equal(alone[1], norm) and all(a is b for a, b in zip(got, grads))
    # a norm below the limit leaves the tensors as they are, bit for bit
    again = [g.clone() for g in grads]
    rlca.rlca_clip_grads(grads, 1e9, out=grads)
    assert all(torch.equal(a, b) for a, b in zip(grads, again))


def test_clip_many_tensors():
    """More tensors than one launch's table holds, empty ones among them."""
    sizes = [(k * 37) % 61 for k in range(2500)]
    got, norm, _ = check_clip(grads_of(sizes, seed=3), 1.0)
    again, norm2 = rlca.rlca_clip_grads(grads_of(sizes, seed=3), 1.0)
    assert torch.equal(norm, norm2) and all(torch.equal(a, b) for a, b in zip(got, again))


def test_clip_shapes_and_other_stream():
    s = torch.cuda.Stream()
    grads = [torch.randn(3, 5, 7, device="cuda"), torch.randn((), device="cuda"), torch.randn(64, 64, device="cuda")]
    s.wait_stream(torch.cuda.current_stream())
    got, norm = rlca.rlca_clip_grads(grads, 0.25, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    want, norm0, _ = ref.clip_grads(grads, 0.25)
    assert abs(norm.item() - norm0.item()) < 1e-5 * norm0.item()
    for g, w in zip(got, want):
        assert g.shape == w.shape
        check(g, w, w.abs() * 40 * U, "clipped")


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_clip_not_finite(bad):
    grads = grads_of([100, 50000], seed=4, mixed=False)
    grads[1][777] = bad
    got, norm = rlca.rlca_clip_grads(grads, 1.0)
    assert not math.isfinite(norm.item())
    for g, b in zip(got, grads):
        assert torch.equal(torch.nan_to_num(g, 1.0, 2.0, 3.0), torch.nan_to_num(b, 1.0, 2.0, 3.0))


def test_clip_empty():
    norm = torch.full((), 7.0, device="cuda")
    got, n = rlca.rlca_clip_grads([], 1.0, norm=norm)
    assert got == [] and n.item() == 0.0
    got, n = rlca.rlca_clip_grads([torch.empty(0, device="cuda")], 1.0)
    assert n.item() == 0.0


def test_clip_offsets_past_32_bits():
    n = (1 << 32) + 100003
    g = torch.zeros(n, device="cuda", dtype=torch.bfloat16)
    g[0], g[-1], g[1 << 32] = 3.0, 4.0, 12.0
    got, norm = rlca.rlca_clip_grads([g], 1.3)
    assert abs(norm.item() - 13.0) < 1e-4
    for at, want in ((0, 0.3), (n - 1, 0.4), (1 << 32, 1.2)):
        assert abs(got[0][at].item() - want) <= want * (R + 1e-5)


# ---- as a user runs them ------------------------------------------------------------

def test_status_word_and_graph_capture():
    """The calls neither allocate nor synchronise below the binding: they replay from a CUDA graph."""
    h, w, tok, g, e = head_inputs(100, 64, 500, torch.bfloat16, 9)
    x = torch.randn(100, 64, device="cuda", dtype=torch.bfloat16)
    nw = torch.ones(64, device="cuda", dtype=torch.bfloat16)

    def step():
        y, mean, rstd = rlca.rlca_layer_norm(x, nw)
        logp, lse, ent = rlca.rlca_token_logprob(y, w, tok)
        dy, dw = rlca.rlca_token_logprob_backward(y, w, tok, lse, g, entropy=ent, d_entropy=e)
        dx, dnw, _ = rlca.rlca_layer_norm_backward(dy, x, nw, mean, rstd, want_dbias=False)
        clipped, norm = rlca.rlca_clip_grads([dx, dnw, dw], 0.01)
        return [logp, lse, ent, norm] + clipped

    plain = step()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    graph.replay()
    torch.cuda.synchronize()
    if _lib.load().rlca_index_checks() == 0:
        assert all(torch.equal(a, b) for a, b in zip(plain, out))
