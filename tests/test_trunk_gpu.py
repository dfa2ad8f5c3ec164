"""The operators of a recurrent policy's trunk against the 64-bit reference.

Rounding errors are counted in units u = 2^-24, the largest relative error of
one float32 operation.

Gated scan.  A gate's exponential, reciprocal and product leave sigma(g) and
1 - sigma(g) each 10 u off at most (exp 2 last places = 4 u, of which the sum
with 1 keeps less than all; the reciprocal 2 u, the sum and the product 1 u
each).  bfloat16 calls take a shorter exponential, 2 + 1.2 |g| last places off
in the worst case.  A step adds the errors of its gates, of two products, of a
sum, and of the same composed in another order (a product of gates instead of
one): less than 2 (10 + 3) u of its magnitude.  The reference's bound adds up the
magnitudes; SCAN counts the units.

RMS norm.  Sums of D squares in partial sums of at most D / 32 + 32 terms; each
result a few operations more.
"""
import pytest
import torch

from first_order_linear_gb300 import _lib, rlca
from oracle import trunk_ref as ref

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
SCAN = {torch.float32: 26.0, torch.bfloat16: 64.0}   # (|g| up to 12: 17 last places = 34 u in place of 4)
DTYPES = [torch.float32, torch.bfloat16]


@pytest.fixture(autouse=True)
def _lib_and_status(cuda_lib):
    yield
    import ctypes as C
    st = C.c_uint(0)
    assert cuda_lib.rlca_device_status(C.byref(st), 1) == _lib.RLCA_OK and st.value == 0


def half_step(dtype):
    return torch.finfo(dtype).eps / 2 if dtype != torch.float32 else U


def _close(got, want, bound, what):
    far = (got.double() - want).abs() - bound
    assert not torch.isnan(got).any(), f"{what}: NaN"
    assert far.max().item() <= 0, f"{what}: {far.max().item():.3e} beyond the bound (of {bound.max().item():.3e})"


def _norm_close(got, want, tol, what):
    """In the 2-norm, over enough values for their errors to be an average: a rounding to bfloat16 spreads over half a
    step, 2^-8 of the value at most, so it is 2^-8 / sqrt(3) = 2.26e-3 off on average at most (and a single value 3.9e-3)."""
    if want.numel() < 4096:
        return
    far = ((got.double() - want).norm() / want.norm().clamp(min=1e-300)).item()
    assert far <= tol, f"{what}: {far:.3e} off in the 2-norm, {tol:.1e} allowed"


def steps_problem(E, T, D, dtype, seed=0, ends=0.05, lengths=None, time_major=False, fused=False, shift=False, state=True,
                  bias=4.0):
    """Inputs of a gated scan; what lies behind a row's length is NaN and flagged."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    shape = (T, E) if time_major else (E, T)
    # the halves of a projection's rows, or matrices of their own; one element off a vector's boundary
    width = 2 * D + 3 if fused else D
    off = 1 if shift else 0

    def place(v):
        if not fused:
            buf = torch.full((v.numel() + off,), float("nan"), dtype=dtype, device="cuda")
            out = buf[off:].view(*shape, D)
        else:
            out = torch.full((*shape, width), float("nan"), dtype=dtype, device="cuda")[..., off:off + D]
        out.copy_(v)
        return out

    def flags(p):
        return (torch.rand(shape, generator=gen, device="cuda") < p).to(torch.uint8)

    x, dh = n(*shape, D), n(*shape, D)
    gate = n(*shape, D) + bias * torch.rand(D, generator=gen, device="cuda")
    d = dict(terminated=flags(ends) if ends else None, truncated=flags(ends / 2) if ends else None,
             state=n(E, D) if state else None, lengths=None, time_major=time_major)
    if lengths is not None:
        ln = torch.tensor([lengths[e % len(lengths)] for e in range(E)], device="cuda", dtype=torch.int32)
        d["lengths"] = ln
        behind = torch.arange(T, device="cuda")[None, :] >= ln[:, None]
        behind = behind.t() if time_major else behind
        for v in (x, gate, dh):
            v[behind] = float("nan")
        for k in ("terminated", "truncated"):
            if d[k] is not None:
                d[k][behind] = 1
    if fused and not shift:
        both = torch.full((*shape, width), float("nan"), dtype=dtype, device="cuda")
        both[..., :D], both[..., D:2 * D] = x, gate
        d.update(x=both[..., :D], gate=both[..., D:2 * D])
    else:
        d.update(x=place(x), gate=place(gate))
    d["dh"] = place(dh)
    d["d_last"] = n(E, D)
    return d


def check_scan(E, T, D, dtype, backward=True, tol=1e-6, **kw):
    d = steps_problem(E, T, D, dtype, **kw)
    dh, d_last = d.pop("dh"), d.pop("d_last")
    tm = d["time_major"]
    want_h, want_last, bh, bl = ref.gated_scan(**d)
    nan = float("nan")
    h = torch.full(d["x"].shape, nan, dtype=dtype, device="cuda")
    last = torch.full((E, D), nan, device="cuda")
    rlca.rlca_gated_scan(**d, h=h, last=last)
    k = SCAN[dtype] * U
    _close(h, want_h, k * bh + half_step(dtype) * (want_h.abs() + k * bh), "h")
    _close(last, want_last, k * bl + U * want_last.abs(), "last")
    if T > 0 and want_h.norm() > 0:
        _norm_close(h, want_h, tol if dtype == torch.float32 else 2.4e-3, "h")
    if not backward:
        return
    want = ref.gated_scan_backward(dh, d["x"], d["gate"], h, d["terminated"], d["truncated"], d["state"], d["lengths"],
                                   d_last, tm)
    # gradients side by side in one matrix's rows, with columns of no one's between and behind them
    grads = torch.full((*d["x"].shape[:2], 2 * D + 9), nan, dtype=dtype, device="cuda")
    dx, dgate = grads[..., :D], grads[..., D + 8:2 * D + 8]
    d_state = torch.full((E, D), nan, device="cuda")
    rlca.rlca_gated_scan_backward(dh, d["x"], d["gate"], h, d["terminated"], d["truncated"], d["state"], d["lengths"],
                                  d_last=d_last, time_major=tm, dx=dx, dgate=dgate, d_state=d_state)
    for name, got, w, b in (("dx", dx, want[0], want[3]), ("dgate", dgate, want[1], want[4])):
        _close(got, w, k * b + half_step(dtype) * (w.abs() + k * b), name)
        if T > 0 and w.norm() > 0:
            _norm_close(got, w, tol if dtype == torch.float32 else 2.4e-3, name)
    _close(d_state, want[2], k * want[5] + U * want[2].abs(), "d_state")
    assert torch.isnan(grads[..., D:D + 8]).all() and torch.isnan(grads[..., 2 * D + 8:]).all()


# one step, one and several tiles of steps, one past and one short of them; channels that fill vectors and warps and
# that do not; rows that share the SMs and one row alone
SCAN_SIZES = [(1, 1, 1), (3, 1, 130), (1, 2, 64), (2, 7, 33), (5, 16, 128), (2, 63, 100), (1, 64, 256), (3, 65, 65),
              (2, 127, 72), (1, 129, 8), (4, 255, 40), (1, 300, 514), (2, 513, 96), (70, 33, 192), (1, 2049, 64),
              (1, 5000, 130), (9, 1000, 24), (1, 2300, 40), (2, 2999, 64)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("E,T,D", SCAN_SIZES)
def test_gated_scan_sizes(E, T, D, dtype):
    check_scan(E, T, D, dtype, seed=E + T + D)
    check_scan(E, T, D, dtype, seed=E + T + D + 1, time_major=True, ends=0.0, fused=True)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("time_major", [False, True])
@pytest.mark.parametrize("fused,shift", [(False, False), (False, True), (True, False), (True, True)])
def test_gated_scan_layouts(dtype, time_major, fused, shift):
    for E, T, D in ((3, 200, 96), (2, 150, 61), (1, 700, 64)):
        check_scan(E, T, D, dtype, seed=D, time_major=time_major, fused=fused, shift=shift)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("time_major", [False, True])
def test_gated_scan_lengths(dtype, time_major):
    for E, T, D in ((6, 300, 72), (5, 1, 64), (7, 64, 129), (3, 2000, 64), (6, 2500, 40), (40, 12, 64)):
        check_scan(E, T, D, dtype, seed=T, time_major=time_major, lengths=[T, 0, 1, T // 2 + 1, max(T - 1, 0), 64])
        check_scan(E, T, D, dtype, seed=T, time_major=time_major, lengths=[0], state=False)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("time_major", [False, True])
def test_gated_scan_many_short_rows(dtype, time_major):
    """Far more rows than the SMs hold, of a few dozen steps at most: walked step by step, in vectors and not."""
    for E, T, D in ((3000, 12, 64), (9000, 33, 40), (2500, 11, 61)):
        check_scan(E, T, D, dtype, seed=E, time_major=time_major, lengths=[T, 0, 1, T - 1, 5, 8])
        check_scan(E, T, D, dtype, seed=E + 1, time_major=time_major, ends=0.0, fused=True)


def test_gated_scan_lengths_out_of_range_and_bool_flags():
    d = steps_problem(4, 90, 64, torch.float32, seed=4)
    for k in ("dh", "d_last"):
        d.pop(k)
    wild = torch.tensor([-5, 1000, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32, device="cuda")
    tame = torch.tensor([0, 90, 90, 0], dtype=torch.int32, device="cuda")
    a = rlca.rlca_gated_scan(**dict(d, lengths=wild))
    b = rlca.rlca_gated_scan(**dict(d, lengths=tame, terminated=d["terminated"].bool(), truncated=d["truncated"].bool()))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("ends", [0.0, 0.002, 0.5, 1.0])
def test_gated_scan_boundaries(dtype, ends):
    check_scan(4, 700, 64, dtype, seed=3, ends=ends)
    check_scan(4, 700, 64, dtype, seed=4, ends=ends, time_major=True, state=False)


@pytest.mark.parametrize("dtype", DTYPES)
def test_gated_scan_long_memory(dtype):
    """Gates up to sigma(12): states that hardly decay over thousands of steps.  Such a state is rounded at every step, by
    half a unit for the step's gate (next to 1, whose spacing below is 1 u) and one for its sum; T independent errors of up
    to 1.5 u, 0.9 u on average, add up to 0.9 sqrt(T) u, and what does not cancel like that is a bias."""
    check_scan(1, 6000, 128, dtype, seed=1, ends=0.0, bias=10.0, tol=2 * U * 6000 ** 0.5)
    check_scan(3, 3000, 64, dtype, seed=2, ends=0.0005, bias=10.0, time_major=True, tol=2 * U * 3000 ** 0.5)


@pytest.mark.parametrize("E,T,D", [(3, 1, 64), (3, 5, 61), (2, 200, 64), (1, 900, 64), (1, 9001, 64), (2, 7000, 61)])
def test_gated_scan_states_in_place(E, T, D):
    """last in the state's buffer and d_state in d_last's give what buffers of their own give, however a row is shared out."""
    d = steps_problem(E, T, D, torch.bfloat16, seed=T, ends=0.0005)
    dh, d_last = d.pop("dh"), d.pop("d_last")
    h, last = rlca.rlca_gated_scan(**d)
    args = (dh, d["x"], d["gate"], h, d["terminated"], d["truncated"], d["state"])
    grads = rlca.rlca_gated_scan_backward(*args, d_last=d_last)
    for _ in range(5):
        own = d["state"].clone()
        h1, last1 = rlca.rlca_gated_scan(**dict(d, state=own), last=own)
        assert last1 is own and torch.equal(last1, last) and torch.equal(h1, h)
        own = d_last.clone()
        g1 = rlca.rlca_gated_scan_backward(*args, d_last=own, d_state=own)
        assert g1[2] is own and all(torch.equal(a, b) for a, b in zip(g1, grads))


def test_offsets_past_32_bits():
    """Matrices of more than 2^31 elements: their ends against the same rows by themselves."""
    D, T = 2048, (1 << 20) + 333
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    both = torch.empty(1, T, 2 * D, dtype=torch.bfloat16, device="cuda")
    both.normal_(generator=gen)
    x, gate = both[..., :D], both[..., D:]
    ends = torch.zeros(1, T, dtype=torch.uint8, device="cuda")
    cut = T - 500
    ends[0, cut - 1] = 1
    h, last = rlca.rlca_gated_scan(x, gate, ends)
    assert h.numel() > 1 << 31
    h_end, last_end = rlca.rlca_gated_scan(x[:, cut:], gate[:, cut:])
    assert (h[:, cut:].float() - h_end.float()).norm() <= 1e-3 * h_end.float().norm()
    assert (last - last_end).norm() <= 1e-5 * last_end.norm()
    grads = torch.empty_like(both)
    dl = torch.randn(1, D, device="cuda")
    rlca.rlca_gated_scan_backward(h, x, gate, h, ends, d_last=dl, dx=grads[..., :D], dgate=grads[..., D:])
    dx, dgate, _ = rlca.rlca_gated_scan_backward(h[:, cut:], x[:, cut:], gate[:, cut:], h[:, cut:], d_last=dl)
    assert (grads[:, cut:, :D].float() - dx.float()).norm() <= 1e-3 * dx.float().norm()
    assert (grads[:, cut:, D:].float() - dgate.float()).norm() <= 1e-3 * dgate.float().norm()
    del grads, dx, dgate, h, both
    N = (1 << 20) + 333
    rows = torch.empty(N, D, dtype=torch.bfloat16, device="cuda")
    rows.normal_(generator=gen)
    w = torch.ones(D, dtype=torch.bfloat16, device="cuda")
    y, total, rstd, y8, t8 = rlca.rlca_rms_norm(rows, w, rows.clone(), want_y8=True, want_total8=True)
    y1, total1, rstd1, y81, t81 = rlca.rlca_rms_norm(rows[-300:], w, rows[-300:].clone(), want_y8=True, want_total8=True)
    for a, b in ((y, y1), (total, total1), (rstd, rstd1), (y8[0].view(torch.uint8), y81[0].view(torch.uint8)), (y8[1], y81[1]),
                 (t8[0].view(torch.uint8), t81[0].view(torch.uint8)), (t8[1], t81[1])):
        assert torch.equal(a[-300:], b)
    for kept, kept1 in ((total, total1), (t8, t81)):
        dx, _ = rlca.rlca_rms_norm_backward(y, kept, w, rstd, d_total=rows)
        dx1, _ = rlca.rlca_rms_norm_backward(y1, kept1, w, rstd1, d_total=rows[-300:])
        assert torch.equal(dx[-300:], dx1)


def test_gated_scan_cut_in_calls():
    """A rollout in three calls, the state handed on in its own buffer."""
    d = steps_problem(3, 400, 96, torch.float32, seed=9)
    want_h, want_last, bh, bl = ref.gated_scan(**{k: v for k, v in d.items() if k not in ("dh", "d_last")})
    state, parts = d["state"].clone(), []
    for lo, hi in ((0, 130), (130, 131), (131, 400)):
        cut = {k: d[k][:, lo:hi].contiguous() for k in ("x", "gate", "terminated", "truncated")}
        h, last = rlca.rlca_gated_scan(state=state, last=state, **cut)
        assert last is state
        parts.append(h)
    _close(torch.cat(parts, 1), want_h, 30 * U * bh + U * want_h.abs(), "h")
    _close(state, want_last, 30 * U * bl + U * want_last.abs(), "last")


@pytest.mark.parametrize("time_major", [False, True])
def test_gated_scan_nothing_leaks(time_major):
    """NaN and infinities in front of an episode's end, in other rows and in other channels reach nothing else."""
    for T, at in ((700, 333), (40, 7), (6000, 4097)):
        d = steps_problem(3, T, 64, torch.float32, seed=2, ends=0.0, time_major=time_major)
        clean = {k: v for k, v in d.items() if k not in ("dh", "d_last")}
        clean["terminated"] = torch.zeros(d["x"].shape[:2], dtype=torch.uint8, device="cuda")
        sel = (lambda e, t: (t, e)) if time_major else (lambda e, t: (e, t))
        clean["terminated"][sel(1, at)] = 1
        h0, l0 = rlca.rlca_gated_scan(**clean)
        g0 = rlca.rlca_gated_scan_backward(d["dh"], clean["x"], clean["gate"], h0, clean["terminated"],
                                           state=clean["state"], d_last=d["d_last"], time_major=time_major)
        bad = dict(clean, x=clean["x"].clone(), gate=clean["gate"].clone(), state=clean["state"].clone())
        bad["x"][sel(1, at - 3)] = float("nan")
        bad["gate"][sel(1, at - 5)] = float("nan")
        bad["state"][1] = float("inf")
        h1, l1 = rlca.rlca_gated_scan(**bad)
        g1 = rlca.rlca_gated_scan_backward(d["dh"], bad["x"], bad["gate"], h1, bad["terminated"], state=bad["state"],
                                           d_last=d["d_last"], time_major=time_major)
        same = torch.ones(d["x"].shape[:2], dtype=torch.bool, device="cuda")
        for t in range(0, at + 1):
            same[sel(1, t)] = False
        assert torch.equal(h0[same], h1[same]) and torch.equal(l0, l1)
        assert torch.isnan(h1[sel(1, at - 1)]).all()
        assert torch.equal(g0[0][same], g1[0][same]) and torch.equal(g0[1][same], g1[1][same])
        # gradients from behind the end reach nothing in front of it
        dh = d["dh"].clone()
        dh[sel(1, at + 2)] = float("nan")
        g2 = rlca.rlca_gated_scan_backward(dh, clean["x"], clean["gate"], h0, clean["terminated"], state=clean["state"],
                                           d_last=d["d_last"], time_major=time_major)
        front = torch.ones_like(same)
        for t in range(at + 1, at + 3):
            front[sel(1, t)] = False
        assert torch.equal(g0[0][front], g2[0][front]) and torch.equal(g0[1][front], g2[1][front])
        assert torch.equal(g0[2], g2[2])


def test_gated_scan_extreme_gates():
    x = torch.randn(2, 200, 64, device="cuda")
    state = torch.randn(2, 64, device="cuda")
    for g, want in ((float("inf"), state[:, None].expand_as(x)), (-float("inf"), x), (200.0, state[:, None].expand_as(x)),
                    (-200.0, x)):
        h, _ = rlca.rlca_gated_scan(x, torch.full_like(x, g), state=state)
        assert torch.equal(h, want), g
        # (bfloat16: a shut gate counts as one of up to 2 u)
        xb = x.bfloat16()
        h, _ = rlca.rlca_gated_scan(xb, torch.full_like(xb, g), state=state)
        want = want.double() if g > 0 else xb.double()
        _close(h, want, half_step(torch.bfloat16) * want.abs() + 4 * U * state.abs().amax(), f"gates of {g}")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("E,T,D", [(2, 700, 64), (1, 900, 96), (2, 2999, 64), (4, 7, 64)])
def test_gated_scan_closed_gates_beside_open_ones(E, T, D, dtype):
    """Channels whose gates are shut so far that products of them vanish, next to channels that remember, with ends of
    episodes between: what marks an end in one channel's product says nothing in another's."""
    d = steps_problem(E, T, D, dtype, seed=T, ends=0.02)
    dh, d_last = d.pop("dh"), d.pop("d_last")
    shut = torch.tensor([-20.0, -100.0, -17.0, -60.0], device="cuda").repeat(T)[:T].to(dtype)
    d["gate"][..., 0::2] = shut[:, None]
    want_h, want_last, bh, bl = ref.gated_scan(**d)
    h, last = rlca.rlca_gated_scan(**d)
    k = SCAN[dtype] * U
    # (a gate below 2^-24 counts as one of up to 2 u: that much of the state may pass)
    leak = 2 * U * want_h.abs().amax()
    _close(h, want_h, k * bh + leak + half_step(dtype) * (want_h.abs() + k * bh), "h")
    _close(last, want_last, k * bl + leak + U * want_last.abs(), "last")
    want = ref.gated_scan_backward(dh, d["x"], d["gate"], h, d["terminated"], d["truncated"], d["state"], None, d_last)
    dx, dgate, d_state = rlca.rlca_gated_scan_backward(dh, d["x"], d["gate"], h, d["terminated"], d["truncated"], d["state"],
                                                       d_last=d_last)
    big = want[3].amax() + want[4].amax() + want[5].amax()
    for name, got, w, b in (("dx", dx, want[0], want[3]), ("dgate", dgate, want[1], want[4]), ("d_state", d_state, want[2], want[5])):
        _close(got, w, k * b + 4 * U * big + half_step(got.dtype) * (w.abs() + k * b), name)


def test_gated_scan_empty():
    s, dl = torch.randn(3, 8, device="cuda"), torch.randn(3, 8, device="cuda")
    x = torch.zeros(3, 0, 8, device="cuda")
    h, last = rlca.rlca_gated_scan(x, x, state=s)
    assert h.shape == (3, 0, 8) and torch.equal(last, s)
    assert torch.equal(rlca.rlca_gated_scan(x, x)[1], torch.zeros_like(s))
    dx, dg, ds = rlca.rlca_gated_scan_backward(x, x, x, h, state=s, d_last=dl)
    assert dx.shape == (3, 0, 8) and torch.equal(ds, dl)
    x = torch.zeros(0, 5, 8, device="cuda")
    assert rlca.rlca_gated_scan(x, x)[1].shape == (0, 8)
    x = torch.zeros(2, 5, 0, device="cuda")
    assert rlca.rlca_gated_scan(x, x)[0].shape == (2, 5, 0)


def test_gated_scan_backward_of_the_last_state_alone():
    """d_state in d_last's own buffer; d_last absent counts as 0."""
    d = steps_problem(2, 300, 64, torch.float32, seed=8, ends=0.0)
    h, _ = rlca.rlca_gated_scan(d["x"], d["gate"], state=d["state"])
    args = (d["dh"], d["x"], d["gate"], h)
    a = rlca.rlca_gated_scan_backward(*args, state=d["state"], d_last=d["d_last"])
    buf = d["d_last"].clone()
    b = rlca.rlca_gated_scan_backward(*args, state=d["state"], d_last=buf, d_state=buf)
    assert b[2] is buf and all(torch.equal(p, q) for p, q in zip(a, b))
    c = rlca.rlca_gated_scan_backward(*args, state=d["state"])
    z = rlca.rlca_gated_scan_backward(*args, state=d["state"], d_last=torch.zeros_like(buf), want_d_state=False)
    assert torch.equal(c[0], z[0]) and torch.equal(c[1], z[1]) and z[2] is None


# ---- RMS norm -----------------------------------------------------------------

def _matrix(N, D, dtype, gen, strided=False, shift=False, wide=True):
    v = torch.randn(N, D, generator=gen, device="cuda")
    if wide:
        v *= 1 + 20 * (torch.rand(D, generator=gen, device="cuda") < 0.02)
    if strided:
        buf = torch.full((N, D + 24), float("nan"), dtype=dtype, device="cuda")
        out = buf[:, 8:8 + D]
    elif shift:
        out = torch.full((N * D + 1,), float("nan"), dtype=dtype, device="cuda")[1:].view(N, D)
    else:
        out = torch.empty(N, D, dtype=dtype, device="cuda")
    out.copy_(v)
    return out


def _check_eight(pair, value, bound, what):
    """A pair against the values it stands for, each `bound` off before its rounding."""
    q, scale = pair
    s = ref.scales(value)
    wide = s.repeat_interleave(ref.GROUP, 1)[:, :value.shape[1]]
    far = torch.stack([g.amax(1) for g in torch.split(bound, ref.GROUP, 1)], 1) / ref.E4M3_MAX
    # (the scale's own product and the reciprocal behind the quotient: 4 u)
    _close(scale, s, far + 4 * U * s, f"{what}: scales")
    _close(ref.read_back(q, scale), value, (2.0 ** -4 + 8 * U) * value.abs() + 2 * bound + 1.01 * 2.0 ** -10 * wide, what)
    # half a step at most of what e4m3 has at the value over its scale, not just some value near it
    ratio = value / wide
    step = torch.exp2(torch.floor(torch.log2(ratio.abs().clamp(min=2.0 ** -6))) - 3)
    _close(q, ratio, 0.5 * step * (1 + 1e-6) + 2 * bound / wide + 8 * U * ratio.abs(), f"{what}: values")


def check_rms(N, D, dtype, seed=0, residual=True, eps=1e-6, **kw):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    x = _matrix(N, D, dtype, gen, **kw)
    r = _matrix(N, D, dtype, gen, **kw) if residual else None
    w = (1 + 0.2 * torch.randn(D, generator=gen, device="cuda")).to(dtype)
    nan = float("nan")
    buf = lambda *s: torch.full(s, nan, dtype=dtype, device="cuda")  # noqa: E731
    y, total, y8, t8 = buf(N, D), buf(N, D) if residual else None, None, None
    y, total, rstd, y8, t8 = rlca.rlca_rms_norm(x, w, r, eps=eps, y=y, total=total, want_y8=True, want_total8=True)
    want_total = x if r is None else (x.float() + r.float()).to(dtype)
    assert torch.equal(total, want_total)
    want_y, want_rstd = ref.rms_norm(want_total, w, eps)
    k = (D / 32 + 40) * U
    _close(rstd, want_rstd, k * want_rstd, "rstd")
    by = k * want_y.abs()
    _close(y, want_y, by + half_step(dtype) * (want_y.abs() + by), "y")
    _check_eight(y8, want_y, by, "y8")
    _check_eight(t8, want_total.double(), torch.zeros_like(want_y), "total8")
    # an output does not depend on which others are wanted, nor total on where it goes
    only8 = rlca.rlca_rms_norm(x, w, r, eps=eps, want_y=False, want_y8=True)
    assert only8[0] is None and only8[4] is None
    assert torch.equal(only8[3][0].view(torch.uint8), y8[0].view(torch.uint8)) and torch.equal(only8[3][1], y8[1])
    plain = rlca.rlca_rms_norm(x, w, r, eps=eps)
    assert torch.equal(plain[0], y) and plain[3] is None and torch.equal(plain[2], rstd)
    if residual:
        own = r.contiguous().clone()
        got = rlca.rlca_rms_norm(x, w, own, eps=eps, total=own)
        assert got[1] is own and torch.equal(own, total) and torch.equal(got[0], y)

    for kept in (total, t8):
        dy = _matrix(N, D, dtype, gen, wide=False, **kw)
        dt = _matrix(N, D, dtype, gen, wide=False, **kw) if residual else None
        value = ref.read_back(*kept) if isinstance(kept, tuple) else kept
        dx, dw, along, mag = ref.rms_norm_backward(dy, value, w, rstd, dt)
        got_dx, got_dw = rlca.rlca_rms_norm_backward(dy, kept, w, rstd, d_total=dt, dx=buf(N, D), dweight=buf(D))
        s = (value.double() * rstd.double()[:, None]).abs()
        g = (dy.double() * w.double()).abs()
        b = rstd.double()[:, None] * (4 * U * g + s * (D / 32 + 44) * U * along) + 2 * U * dx.abs()
        if dt is not None:
            b = b + U * dt.double().abs()
        _close(got_dx, dx, b + half_step(dtype) * (dx.abs() + b), "dx")
        bw = (N / 64 + 80) * U * mag
        _close(got_dw, dw, bw + half_step(dtype) * (dw.abs() + bw), "dweight")
        one, none = rlca.rlca_rms_norm_backward(dy, kept, w, rstd, d_total=dt, want_dweight=False)
        assert none is None and torch.equal(one, got_dx)
        none, one = rlca.rlca_rms_norm_backward(dy, kept, w, rstd, d_total=dt, want_dx=False)
        assert none is None and torch.equal(one, got_dw)


# rows of one element, of part of a group, of one and of several groups, at both alignments and in every variant by width
RMS_SIZES = [(1, 1), (2, 7), (5, 32), (33, 100), (17, 128), (64, 129), (9, 136), (130, 256), (40, 1001), (300, 1024),
             (7, 1544), (61, 2048), (1000, 520), (37, 4096), (5, 5000), (19, 8192), (3, 8200), (2, 20000), (700, 64),
             (3000, 40)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("N,D", RMS_SIZES)
def test_rms_norm_sizes(N, D, dtype):
    check_rms(N, D, dtype, seed=N + D)
    check_rms(N, D, dtype, seed=N + D + 1, residual=False)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("kw", [dict(strided=True), dict(shift=True)], ids=["strided", "shifted"])
def test_rms_norm_layouts(dtype, kw):
    for N, D in ((33, 256), (20, 1000), (9, 4096), (50, 130)):
        check_rms(N, D, dtype, seed=D, **kw)
        check_rms(N, D, dtype, seed=D + 1, residual=False, **kw)


def test_rms_norm_many_rows():
    check_rms(20011, 512, torch.bfloat16, seed=1)
    check_rms(9001, 1001, torch.float32, seed=2)


def test_rms_norm_no_rows():
    x, w = torch.zeros(0, 256, device="cuda"), torch.ones(256, device="cuda")
    y, total, rstd, y8, t8 = rlca.rlca_rms_norm(x, w, x.clone(), want_y8=True, want_total8=True)
    assert y.shape == (0, 256) and y8[1].shape == (0, 2)
    dx, dw = rlca.rlca_rms_norm_backward(x, t8, w, rstd)
    assert dx.shape == (0, 256) and torch.equal(dw, torch.zeros(256, device="cuda"))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D", [256, 300, 8200])
def test_rows_in_8_bits_of_unusual_values(dtype, D):
    x = torch.randn(6, D, device="cuda")
    x[0] = 0
    x[1, :128] = 0
    x[2, 5] = float("nan")
    x[3, 200] = float("inf")
    x[4] *= 1e-30
    x[5] *= 1e15
    x = x.to(dtype)
    w = torch.ones(D, dtype=dtype, device="cuda")
    _, _, rstd, _, (q, scale) = rlca.rlca_rms_norm(x, w, want_total8=True)
    back = ref.read_back(q, scale)
    assert torch.equal(scale[0], torch.full_like(scale[0], 2.0 ** -126)) and (back[0] == 0).all()
    assert scale[1, 0] == 2.0 ** -126 and (back[1, :128] == 0).all()
    assert torch.isnan(back[2, 5]) and not torch.isnan(back[2, :5]).any() and not torch.isnan(back[2, 6:]).any()
    assert torch.isnan(back[3, 128:min(D, 256)]).all() and not torch.isnan(back[3, :128]).any()
    for k in (4, 5):
        err = ((back[k] - x[k].double()).norm() / x[k].double().norm()).item()
        # half a step is 2^-4 of a value at most, and on average over a binade less than two thirds of that; what lies below
        # e4m3's normal range, 2^-9 of a group's maximum of some 4, adds less than 2^-10 / 448 of it
        assert err < 2.0 ** -4, (k, err)
    assert rstd[3] == 0 and torch.isnan(rstd[2])


def test_streams_and_graphs():
    """Calls on another stream than the current one, and captured and replayed on new values."""
    d = steps_problem(2, 500, 64, torch.bfloat16, seed=1)
    x, w = torch.randn(65, 512, device="cuda").bfloat16(), torch.ones(512, device="cuda").bfloat16()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    scan = {k: d[k] for k in ("x", "gate", "terminated", "truncated", "state")}
    h, last = rlca.rlca_gated_scan(**scan, stream=side)
    y, total, rstd, y8, t8 = rlca.rlca_rms_norm(x, w, x.clone(), want_y8=True, want_total8=True, stream=side)
    dx, dw = rlca.rlca_rms_norm_backward(y, t8, w, rstd, stream=side)
    grads = rlca.rlca_gated_scan_backward(d["dh"], d["x"], d["gate"], h, d["terminated"], d["truncated"], d["state"],
                                          d_last=d["d_last"], stream=side)
    torch.cuda.current_stream().wait_stream(side)
    with torch.cuda.stream(side):
        pass
    h0, last0 = rlca.rlca_gated_scan(**scan)
    assert torch.equal(h, h0) and torch.equal(last, last0)
    dx0, dw0 = rlca.rlca_rms_norm_backward(y, t8, w, rstd)
    assert torch.equal(dx, dx0) and torch.equal(dw, dw0)
    grads0 = rlca.rlca_gated_scan_backward(d["dh"], d["x"], d["gate"], h, d["terminated"], d["truncated"], d["state"],
                                           d_last=d["d_last"])
    assert all(torch.equal(a, b) for a, b in zip(grads, grads0))

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gh, gl = rlca.rlca_gated_scan(**scan)
        gg = rlca.rlca_gated_scan_backward(d["dh"], d["x"], d["gate"], gh, d["terminated"], d["truncated"], d["state"],
                                           d_last=d["d_last"])
        gy = rlca.rlca_rms_norm(x, w, y, want_y8=True, want_total8=True)
        gdx = rlca.rlca_rms_norm_backward(y, gy[4], w, gy[2])
    for seed in (3, 4):
        new = steps_problem(2, 500, 64, torch.bfloat16, seed=seed)
        for k in ("x", "gate", "terminated", "truncated", "state", "dh", "d_last"):
            d[k].copy_(new[k])
        x.copy_(torch.randn(65, 512, device="cuda"))
        graph.replay()
        h1, l1 = rlca.rlca_gated_scan(**scan)
        g1 = rlca.rlca_gated_scan_backward(d["dh"], d["x"], d["gate"], h1, d["terminated"], d["truncated"], d["state"],
                                           d_last=d["d_last"])
        y1 = rlca.rlca_rms_norm(x, w, y, want_y8=True, want_total8=True)
        d1 = rlca.rlca_rms_norm_backward(y, y1[4], w, y1[2])
        assert torch.equal(gh, h1) and torch.equal(gl, l1) and all(torch.equal(a, b) for a, b in zip(gg, g1))
        assert torch.equal(gy[0], y1[0]) and torch.equal(gy[3][1], y1[3][1])
        assert torch.equal(gdx[0], d1[0]) and torch.equal(gdx[1], d1[1])


def test_gradients_against_differences():
    """The kernels' gradients against central differences of the 64-bit forward pass (truncation 1e-10, see
    test_trunk_cpu.py), at float32's own errors: sums of 600 products of terms of order 1, 100 u each at most."""
    d = steps_problem(2, 50, 6, torch.float32, seed=6)
    dh, dl = d.pop("dh"), d.pop("d_last")
    h, _ = rlca.rlca_gated_scan(**d)
    got = rlca.rlca_gated_scan_backward(dh, d["x"], d["gate"], h, d["terminated"], d["truncated"], d["state"], d_last=dl)

    def value(**k):
        hh, last, _, _ = ref.gated_scan(**dict(d, **k))
        return ((hh * dh.double()).sum() + (last * dl.double()).sum()).item()

    for name, grad in zip(("x", "gate", "state"), got):
        v = d[name].double()
        step = torch.randn_like(v)
        diff = (value(**{name: v + 1e-5 * step}) - value(**{name: v - 1e-5 * step})) / 2e-5
        scale = (grad.double() * step).abs().sum().item()
        assert abs(diff - (grad.double() * step).sum().item()) < 100 * U * scale + 1e-6, name
