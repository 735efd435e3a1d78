"""The selective state space scan against its definition in 64 bits (bounds in state_space_testutil)."""
import ctypes
import math

import pytest
import torch

import state_space_testutil as R
from ops_testutil import normal

GRADS = ("dX", "ddt", "dz", "dB", "dC", "dA", "dD", "ddt_bias")


def _case(T, C, G, S, nseq, kind, seed):
    """Steps of 1/1000 to 1/10 (some rows far from that), decays of up to S times that."""
    gen = torch.Generator().manual_seed(seed)
    want = torch.exp(torch.rand(C, generator=gen) * math.log(100.0) + math.log(0.001))
    dt = torch.randn(T, C, generator=gen)
    dt[::7] *= 6
    c = dict(x=normal(gen, T, C, kind=kind), dt=dt.to(R.TYPES[kind]),
             A=-torch.arange(1, S + 1).float() * torch.exp(0.2 * torch.randn(C, S, generator=gen)),
             B=normal(gen, T, G, S, kind=kind), C=normal(gen, T, G, S, kind=kind), D=torch.randn(C, generator=gen),
             z=normal(gen, T, C, kind=kind), bias=want + torch.log(-torch.expm1(-want)))
    return c, normal(gen, T, C, kind=kind), 0.5 * torch.randn(nseq, C, S, generator=gen), torch.randn(nseq, C, S, generator=gen)


def _rows(c):
    return c["x"], c["dt"], c["A"], c["B"], c["C"]


def _cuda(c):
    return {k: v.cuda() for k, v in c.items()}


def _options(c, gated=True, plain=False):
    """D, gate, bias; `plain`: none of them, and no softplus."""
    if plain:
        return dict(softplus=False)
    return dict(D=c["D"], z=c["z"] if gated else None, dt_bias=c["bias"])


# ------------------------------------------------------------------------------------------------ without a GPU

@pytest.mark.parametrize("gated", [True, False])
def test_the_gradient_formulas_against_differences(gated):
    c, dy, st, dl = _case(6, 2, 1, 4, 2, "f32", 1)
    c = {k: v.double() for k, v in c.items()}
    off, names = [0, 4, 6], ("x", "dt", "A", "B", "C", "D", "z", "bias")
    z = lambda c: c["z"] if gated else None  # noqa: E731

    def loss(c, st):
        (Y, last), _ = R.scan(c["x"], c["dt"], c["A"], c["B"], c["C"], c["D"], z(c), c["bias"], True, off, st)
        return float((Y * dy.double()).sum() + (last * dl.double()).sum())

    g, _ = R.scan_backward(c["x"], c["dt"], c["A"], c["B"], c["C"], dy, c["D"], z(c), c["bias"], True, off, st, dl.double())
    of = dict(zip(names, ("dX", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias")))
    st = st.double()
    for name in names + ("st",):
        if name == "z" and not gated:
            continue
        grad = g[of[name]] if name != "st" else g["dstate_in"]
        for at in range(grad.numel()):
            ends = []
            for s in (1e-5, -1e-5):
                d, h = {k: v.clone() for k, v in c.items()}, st.clone()
                (h if name == "st" else d[name]).view(-1)[at] += s
                ends.append(loss(d, h))
            assert abs((ends[0] - ends[1]) / 2e-5 - float(grad.reshape(-1)[at])) < 1e-7, (name, at)


def test_refuses_on_the_host():
    from bwd_la_fwd_gb300 import la
    lib = la.load_library()
    P = lambda k: k << 32  # noqa: E731

    def call(x=P(1), dt=P(2), A=P(3), B=P(4), C=P(5), D=None, z=None, bias=None, first=None, y=P(6), last=None, marks=None,
             off=None, nseq=2, N=4, ch=64, G=1, S=16, dtype=1, strides=None, ws=P(7), size=1 << 30):
        st = None if strides is None else (ctypes.c_longlong * 14)(*strides)
        return lib.la_selective_scan(x, dt, A, B, C, D, z, bias, 1, first, y, last, marks, off, nseq, N, ch, G, S, dtype, st, ws,
                                     size, None)

    assert call(dtype=5) == 1 and call(nseq=-1) == 1 and call(N=-1) == 1 and call(ch=0) == 1 and call(G=0) == 1 and call(G=3) == 1
    assert call(ch=2 ** 24) == 1
    assert call(S=12) == 2 and call(S=64) == 2 and call(ch=20, G=5) == 2
    for k in ("x", "dt", "A", "B", "C", "y"):
        assert call(**{k: None}) == 1 and call(**{k: P(9) + 8}) == 1, k
    assert call(D=P(9) + 4) == 1 and call(bias=P(9) + 4) == 1 and call(first=P(9) + 4) == 1 and call(marks=P(9) + 4) == 1
    assert call(ch=33) == 1
    assert call(y=P(1)) == 1 and call(y=P(4)) == 1 and call(last=P(6)) == 1 and call(first=P(9), last=P(9)) == 1
    assert call(marks=P(6)) == 1 and call(ws=None) == 3 and call(size=128) == 3 and call(ws=P(7) + 16) == 3 and call(y=P(7)) == 1
    assert call(strides=[256, 64] * 4 + [64, 16, 8] * 2) != 0                 # B's rows overlap where they are stepped
    assert call(off=P(9) + 2) == 1 and call(off=P(6)) == 1
    assert call(nseq=2 ** 16, N=2 ** 16) == 1 and call(nseq=0) == 0

    def back(dx=P(8), ddt=P(9), dA=P(10), dB=P(11), dC=P(12), dD=None, dz=None, db=None, marks=P(13), z=None, dy=P(6), ws=P(7),
             size=1 << 30):
        return lib.la_selective_scan_backward(P(1), P(2), P(3), P(4), P(5), None, z, None, 1, dy, marks, None, dx, ddt, dA, dB, dC, dD,
                                              dz, db, None, None, 2, 4, 64, 1, 16, 1, None, ws, size, None)

    for k in ("dx", "ddt", "dA", "dB", "dC", "marks", "dy"):
        assert back(**{k: None}) == 1, k
    assert back(z=P(14)) == 1 and back(dz=P(14)) == 1                          # z and its gradient come together
    assert back(dx=P(9)) == 1 and back(dB=P(12)) == 1 and back(dA=P(3)) == 1 and back(dx=P(6)) == 1 and back(dC=P(13)) == 1
    assert back(ws=None) == 3 and back(size=256) == 3

    def step(s=P(7), y=P(6), n=2, x=P(1), S=16):
        return lib.la_selective_scan_step(x, P(2), P(3), P(4), P(5), None, None, None, 1, s, y, n, 64, 1, S, 1, None, None)

    assert step(s=None) == 1 and step(s=P(7) + 4) == 1 and step(y=P(7)) == 1 and step(y=P(1)) == 1 and step(x=None) == 1
    assert step(S=7) == 2 and step(n=0) == 0
    assert lib.la_selective_scan_workspace_bytes(100, 1, 64, 1, 5, 1, 0) == 0 and lib.la_selective_scan_marks_bytes(100, 1, 64, 5) == 0


def test_binding_refuses():
    from bwd_la_fwd_gb300 import la
    c, dy, st, _ = _case(8, 64, 1, 16, 2, "bf16", 1)
    b = {k: v.view(2, 4, *v.shape[1:]) if k in ("x", "dt", "z", "B", "C") else v for k, v in c.items()}
    off = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="without seq_offsets"):
        la.la_selective_scan(*_rows(c))
    with pytest.raises(ValueError, match="packed"):
        la.la_selective_scan(*_rows(b), seq_offsets=off)
    with pytest.raises(ValueError, match="CUDA"):
        la.la_selective_scan(*_rows(b))
    with pytest.raises(ValueError, match="A:"):
        la.la_selective_scan(b["x"], b["dt"], b["A"][:, :8], b["B"], b["C"])
    with pytest.raises(ValueError, match="B, C"):
        la.la_selective_scan(b["x"], b["dt"], b["A"], b["B"].float(), b["C"])
    with pytest.raises(ValueError):
        la.la_selective_scan(b["x"], b["dt"], b["A"], b["B"], b["C"][:1])
    with pytest.raises(ValueError, match="D:"):
        la.la_selective_scan(*_rows(b), D=torch.empty(3))
    with pytest.raises(ValueError, match="state_in"):
        la.la_selective_scan(*_rows(b), state_in=st[:1])
    with pytest.raises(ValueError, match="marks"):
        la.la_selective_scan(*_rows(b), marks=torch.empty(5))
    with pytest.raises(ValueError, match="marks"):
        la.la_selective_scan_backward(*_rows(b), b["x"], torch.empty(5))
    with pytest.raises(ValueError, match="state"):
        la.la_selective_scan_step(st[:, :3], c["x"][:2], c["dt"][:2], c["A"], c["B"][:2], c["C"][:2])


# --------------------------------------------------------------------------------------------------- on the GPU

def _forward(c, off, st, kind, pad, options, marks=None):
    from bwd_la_fwd_gb300 import la
    g = _cuda(c)
    T, C = c["x"].shape
    G, S = c["B"].shape[1:]
    n = len(off) - 1
    offs = torch.tensor(off, dtype=torch.int32, device="cuda")
    ws = la.new_selective_scan_workspace(T, n, C, G, S, la.LA_BF16 if kind == "bf16" else la.LA_F32)
    Y = torch.full((T, C), 3.0, dtype=c["x"].dtype, device="cuda")
    last = torch.full((n, C, S), 9.0, device="cuda")
    la.la_selective_scan(*_rows(g), **{k: v.cuda() if torch.is_tensor(v) else v for k, v in options.items()}, seq_offsets=offs,
                         state_in=None if st is None else st.cuda(), state_out=last, Y=Y, marks=marks, workspace=ws)
    assert la.la_get_status(ws) == 0
    return Y, last


def _check_forward(c, off, st, kind, options, extra=0):
    Y, last = _forward(c, off, st, kind, 0, options)
    sp = options.get("softplus", True)
    (y, h), (ey, eh) = R.scan(*_rows(c), options.get("D"), options.get("z"), options.get("dt_bias"), sp, off, st, extra)
    s = slice(off[0], off[-1])
    R.assert_within("Y", Y[s], y[s], R.rounded(y, ey, kind)[s])
    assert (Y[:off[0]] == 3).all() and (Y[off[-1]:] == 3).all()
    R.assert_within("state", last, h, eh)


LENGTHS = [[1], [2, 0, 1, 17, 0], [31, 16, 33], [129], [0, 5]]


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("S", [8, 16, 32])
@pytest.mark.parametrize("lens", LENGTHS)
def test_packed_sequences(lens, S, kind):
    """All options on and off; rows before the first and behind the last sequence stay as they are."""
    for C, G, pad, resumed, gated, plain in ((8, 1, 0, True, True, False), (144, 2, 3, False, False, False), (72, 3, 5, True, True, True)):
        off = [pad]
        for n in lens:
            off.append(off[-1] + n)
        c, _, st, _ = _case(off[-1] + pad, C, G, S, len(lens), kind, S + C + off[-1])
        if plain:
            c["dt"] = c["dt"].abs() * 0.1
        _check_forward(c, off, st if resumed else None, kind, _options(c, gated, plain))


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("lens", [[3000], [1500, 0, 1, 1100, 4], [3] * 12 + [1500]])
def test_time_in_parts(lens, kind):
    """Few channels and long sequences, or one that is far longer than the others: parts folded together (a part's sum of d is off by a half step
    for each of its rows)."""
    off = [2]
    for n in lens:
        off.append(off[-1] + n)
    c, _, st, _ = _case(off[-1] + 2, 16, 1, 16, len(lens), kind, 5)
    _check_forward(c, off, st, kind, _options(c), extra=0.4 * 3000)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("S", [8, 16, 32])
@pytest.mark.parametrize("lens", [[1], [2, 0, 1, 17, 0], [40, 16, 33], [1100], [2] * 12 + [900]])
def test_gradients(lens, S, kind):
    from bwd_la_fwd_gb300 import la
    if max(lens) > 500 and S != 16:
        pytest.skip("long sequences with one size of state")
    for C, G, pad, resumed, gated in ((8, 1, 0, True, True), (144, 2, 3, False, False), (72, 3, 1, True, True)):
        off = [pad]
        for n in lens:
            off.append(off[-1] + n)
        T, n = off[-1] + pad, len(lens)
        c, dy, st, dl = _case(T, C, G, S, n, kind, S + C + T)
        opt = _options(c, gated)
        dl = dl if resumed else None
        marks = la.new_selective_scan_marks(T, n, C, S)
        _forward(c, off, st, kind, pad, opt, marks=marks)
        ref, tol = R.scan_backward(*_rows(c), dy, opt["D"], opt["z"], opt["dt_bias"], True, off, st, dl,
                                   extra=0.4 * 1100 if max(lens) > 500 else 0)  # long enough for parts
        g = _cuda(c)
        offs = torch.tensor(off, dtype=torch.int32, device="cuda")
        ws = la.new_selective_scan_workspace(T, n, C, G, S, la.LA_BF16 if kind == "bf16" else la.LA_F32, backward=True)
        call = lambda: la.la_selective_scan_backward(  # noqa: E731
            *_rows(g), dy.cuda(), marks, **{k: v.cuda() if torch.is_tensor(v) else v for k, v in opt.items()}, seq_offsets=offs,
            dstate_out=None if dl is None else dl.cuda(), workspace=ws)
        got = call()
        assert la.la_get_status(ws) == 0
        for name in GRADS + ("dstate_in",):
            if name == "dz" and not gated:
                assert got.dz is None
                continue
            t, typed = getattr(got, name), name in ("dX", "ddt", "dz", "dB", "dC")
            R.assert_within(name, t, ref[name], R.rounded(ref[name], tol[name], kind) if typed else tol[name])
        again = call()
        for name in GRADS:
            assert name == "dz" and not gated or torch.equal(getattr(got, name), getattr(again, name)), name


@pytest.mark.gpu
def test_gradients_against_differences():
    """fp32 gradients along random directions against central differences of the 64-bit forward."""
    from bwd_la_fwd_gb300 import la
    T, C, G, S, off = 70, 24, 1, 16, [0, 30, 70]
    c, dy, st, dl = _case(T, C, G, S, 2, "f32", 11)
    marks = la.new_selective_scan_marks(T, 2, C, S)
    _forward(c, off, st, "f32", 0, _options(c), marks=marks)
    got = la.la_selective_scan_backward(*_rows(_cuda(c)), dy.cuda(), marks, **{k: v.cuda() for k, v in _options(c).items()},
                                        seq_offsets=torch.tensor(off, dtype=torch.int32, device="cuda"), dstate_out=dl.cuda())
    _, tol = R.scan_backward(*_rows(c), dy, c["D"], c["z"], c["bias"], True, off, st, dl)
    c["st"] = st

    def loss(c):
        (Y, last), _ = R.scan(*_rows(c), c["D"], c["z"], c["bias"], True, off, c["st"])
        return float((Y * dy.double()).sum() + (last * dl.double()).sum())

    gen = torch.Generator().manual_seed(2)
    for name, grad in zip(("x", "dt", "z", "B", "C", "A", "D", "bias", "st"), GRADS + ("dstate_in",)):
        d = torch.randn(c[name].shape, generator=gen, dtype=torch.float64)
        ends = []
        for s in (1e-6, -1e-6):
            args = {k: v.double() for k, v in c.items()}
            args[name] = args[name] + s * d
            ends.append(loss(args))
        want, t = (ends[0] - ends[1]) / 2e-6, getattr(got, grad).double().cpu()
        size = float((d.abs() * (tol[grad] + 2 * R.U * t.abs())).sum())
        assert abs(float((t * d).sum()) - want) <= size + 1e-5 * (1 + abs(want)), name


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("S", [8, 16, 32])
def test_tokens_continue_a_prompt(S, kind):
    """A prompt and then single tokens against the definition over the whole sequence."""
    from bwd_la_fwd_gb300 import la
    n, P, T, C, G = 3, 21, 27, 72, 3
    c, _, _, _ = _case(n * T, C, G, S, n, kind, S)
    off = [i * T for i in range(n + 1)]
    (y, h), (ey, eh) = R.scan(*_rows(c), c["D"], c["z"], c["bias"], True, off, None)
    v = {k: t.cuda().view(n, T, *t.shape[1:]) if k in ("x", "dt", "z", "B", "C") else t.cuda() for k, t in c.items()}
    at = lambda s: {k: t[:, s] if k in ("x", "dt", "z", "B", "C") else t for k, t in v.items()}  # noqa: E731
    state = torch.empty(n, C, S, device="cuda")
    p = at(slice(0, P))
    rows = [la.la_selective_scan(*_rows(p), **_options(p), state_out=state)]
    for t in range(P, T):
        one = at(t)
        rows.append(la.la_selective_scan_step(state, *_rows(one), **_options(one))[:, None])
    got = torch.cat(rows, 1).reshape(n * T, C)
    R.assert_within("Y", got, y, R.rounded(y, ey, kind))
    R.assert_within("state", state, h, eh)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_batches_strides_and_odd_channels(kind):
    """Slices of fused projections, channels that are no whole vector, in a batch: as the packed call on copies; gradients too."""
    from bwd_la_fwd_gb300 import la
    B, N, C, S, wide = 2, 50, 75, 16, 400
    c, dy, st, _ = _case(B * N, C, 1, S, B, kind, 3)
    off = torch.tensor([0, N, 2 * N], dtype=torch.int32, device="cuda")
    g = _cuda(c)
    buf = torch.full((B, N, wide), 7.0, dtype=c["x"].dtype, device="cuda")
    views = {}
    for i, k in enumerate(("x", "dt", "z", "dy")):
        views[k] = buf[:, :, 80 * i:80 * i + C]
        views[k].copy_((dy.cuda() if k == "dy" else g[k]).view(B, N, C))
    views["B"], views["C"] = (buf[:, :, 320 + 16 * i:336 + 16 * i].unflatten(2, (1, S)) for i in range(2))
    views["B"].copy_(g["B"].view(B, N, 1, S)), views["C"].copy_(g["C"].view(B, N, 1, S))
    out = torch.full((B, N, wide), 7.0, dtype=c["x"].dtype, device="cuda")
    padded = {k: torch.zeros(B * N, 80, dtype=c["x"].dtype, device="cuda") for k in ("x", "dt", "z", "dy")}
    for k, t in padded.items():
        t[:, :C] = dy.cuda() if k == "dy" else g[k]
    opt = dict(D=g["D"], dt_bias=g["bias"], state_in=st.cuda())
    marks = [la.new_selective_scan_marks(B * N, B, C, S) for _ in range(2)]
    last = [torch.empty(B, C, S, device="cuda") for _ in range(2)]
    Y = la.la_selective_scan(views["x"], views["dt"], g["A"], views["B"], views["C"], z=views["z"], Y=out[:, :, 16:16 + C],
                             state_out=last[0], marks=marks[0], **opt)
    p = {k: t[:, :C] for k, t in padded.items()}
    Z = la.la_selective_scan(p["x"], p["dt"], g["A"], g["B"], g["C"], z=p["z"], seq_offsets=off, state_out=last[1], marks=marks[1],
                             Y=torch.zeros(B * N, 80, dtype=buf.dtype, device="cuda")[:, :C], **opt)
    assert torch.equal(Y.reshape(B * N, C), Z) and torch.equal(*last)
    assert (out[:, :, :16] == 7).all() and (out[:, :, 16 + C:] == 7).all()
    (y, _), (ey, _) = R.scan(*_rows(c), c["D"], c["z"], c["bias"], True, [0, N, 2 * N], st)
    R.assert_within("Y", Z, y, R.rounded(y, ey, kind))
    with pytest.raises(la.LAError):  # rows of 75 channels as contiguous gradients are no whole vectors apart
        la.la_selective_scan_backward(views["x"], views["dt"], g["A"], views["B"], views["C"], views["dy"], marks[0], z=views["z"],
                                      D=g["D"], dt_bias=g["bias"])


@pytest.mark.gpu
def test_sequences_do_not_meet():
    """Infinities and NaN of a sequence, and of rows outside all, have no part in another."""
    from bwd_la_fwd_gb300 import la
    c, dy, _, _ = _case(60, 64, 1, 16, 3, "f32", 12)
    off = [2, 20, 45, 50]
    bad = {k: v.clone() for k, v in c.items()}
    for k in ("x", "dt", "z", "B", "C"):
        bad[k][:2], bad[k][50:] = math.nan, math.nan
    bad["x"][40], bad["B"][21], bad["dt"][44, 0] = math.inf, math.nan, math.nan
    marks = [la.new_selective_scan_marks(60, 3, 64, 16) for _ in range(2)]
    a, _ = _forward(c, off, None, "f32", 0, _options(c), marks=marks[0])
    b, _ = _forward(bad, off, None, "f32", 0, _options(bad), marks=marks[1])
    assert torch.equal(a[:20], b[:20]) and torch.equal(a[45:], b[45:]) and torch.equal(a[20], b[20])
    assert not torch.isfinite(b[21:45]).any()
    offs = torch.tensor(off, dtype=torch.int32, device="cuda")
    got = [la.la_selective_scan_backward(*_rows(_cuda(t)), dy.cuda(), m, **{k: v.cuda() for k, v in _options(t).items()}, seq_offsets=offs)
           for t, m in zip((c, bad), marks)]
    for name in ("dX", "ddt", "dz", "dB", "dC"):
        p, q = (getattr(t, name) for t in got)
        assert torch.equal(p[:20], q[:20]) and torch.equal(p[45:], q[45:]), name


@pytest.mark.gpu
def test_offsets_out_of_order_compute_nothing():
    from bwd_la_fwd_gb300 import la
    c, dy, _, _ = _case(50, 64, 1, 16, 3, "bf16", 13)
    g = _cuda(c)
    for off in ([0, 30, 20, 50], [0, 10, 20, 51], [-1, 10, 20, 50]):
        offs = torch.tensor(off, dtype=torch.int32, device="cuda")
        ws = la.new_selective_scan_workspace(50, 3, 64, 1, 16, la.LA_BF16, backward=True)
        Y = torch.full((50, 64), 3.0, dtype=g["x"].dtype, device="cuda")
        last = torch.full((3, 64, 16), 3.0, device="cuda")
        la.la_selective_scan(*_rows(g), seq_offsets=offs, state_out=last, Y=Y, workspace=ws)
        assert la.la_get_status(ws) == 6 and (Y == 3).all() and (last == 3).all()
        got = la.la_selective_scan_backward(*_rows(g), dy.cuda(), torch.zeros(10 ** 5, device="cuda"), seq_offsets=offs, workspace=ws)
        assert la.la_get_status(ws) == 6
        assert not any(getattr(got, k).any() for k in ("dX", "ddt", "dA", "dB", "dC", "dD", "ddt_bias"))


@pytest.mark.gpu
def test_no_rows_leave_the_state():
    from bwd_la_fwd_gb300 import la
    A = -torch.ones(64, 16, device="cuda")
    e, b = torch.empty(2, 0, 64, device="cuda"), torch.empty(2, 0, 1, 16, device="cuda")
    st, last = torch.randn(2, 64, 16, device="cuda"), torch.empty(2, 64, 16, device="cuda")
    marks = la.new_selective_scan_marks(0, 2, 64, 16)
    assert la.la_selective_scan(e, e, A, b, b, state_in=st, state_out=last, marks=marks).shape == e.shape
    assert torch.equal(st, last)
    got = la.la_selective_scan_backward(e, e, A, b, b, e, marks, dstate_out=st)
    assert torch.equal(got.dstate_in, st) and not got.dA.any()


@pytest.mark.gpu
def test_on_another_stream_and_captured():
    from bwd_la_fwd_gb300 import la
    c, dy, st, _ = _case(3000, 64, 1, 16, 2, "bf16", 14)
    g, dy, st = _cuda(c), dy.cuda(), st.cuda()
    offs = torch.tensor([0, 1700, 3000], dtype=torch.int32, device="cuda")
    opt = dict(**_options(g), seq_offsets=offs)
    marks = la.new_selective_scan_marks(3000, 2, 64, 16)
    want = la.la_selective_scan(*_rows(g), state_in=st, marks=marks, **opt)
    grads = la.la_selective_scan_backward(*_rows(g), dy, marks, **opt)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = la.la_selective_scan(*_rows(g), state_in=st, stream=s, **opt)
    s.synchronize()
    assert torch.equal(got, want)
    ws = la.new_selective_scan_workspace(3000, 2, 64, 1, 16, la.LA_BF16)
    back = la.new_selective_scan_workspace(3000, 2, 64, 1, 16, la.LA_BF16, backward=True)
    Y = torch.zeros_like(want)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        la.la_selective_scan(*_rows(g), state_in=st, marks=marks, Y=Y, workspace=ws, **opt)
        held = la.la_selective_scan_backward(*_rows(g), dy, marks, workspace=back, **opt)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(Y, want)
    for name in GRADS:
        assert torch.equal(getattr(held, name), getattr(grads, name)), name
