"""Products of many gates: NaN among them before a cut, and beyond fp32's range."""
import math

import pytest
import torch

import ops_testutil as R
from test_gated_scan import _inputs


@pytest.mark.gpu
@pytest.mark.parametrize("gate", ["log", "sigmoid"])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("N,cut", [(200, 7), (700, 400), (9000, 4000)])
def test_a_nan_gate_before_a_cut_has_no_part_behind_it(N, cut, kind, gate):
    """Rows of padding may hold anything, gates that are NaN too: the restart behind them (and backwards, the one before
    them) keeps it out, in the same run of rows, the same part of time or another."""
    from bwd_la_fwd_gb300 import la
    x, w, h0, dh, dl = _inputs(1, N, 24, kind, gate, seed=N)
    w[:, cut] = -math.inf
    bad = w.clone()
    bad[:, cut - 3:cut] = math.nan
    x, w, h0, dh, dl, bad = (t.cuda() for t in (x, w, h0, dh, dl, bad))
    (H, last), (H2, last2) = (la.la_gated_scan(x, t, gate, h0=h0) for t in (bad, w))
    assert torch.equal(H[:, cut:], H2[:, cut:]) and torch.equal(last, last2)
    assert torch.isnan(H[:, cut - 3:cut]).all() and torch.equal(H[:, :cut - 3], H2[:, :cut - 3])
    bad = w.clone()
    bad[:, cut + 1:cut + 3] = math.nan
    a, b = (la.la_gated_scan_backward(x, t, H2, dh, gate, h0=h0, dh_last=dl) for t in (bad, w))
    assert torch.equal(a[0][:, :cut], b[0][:, :cut]) and torch.equal(a[1][:, :cut + 1], b[1][:, :cut + 1])
    assert torch.equal(a[2], b[2]) and torch.isnan(a[1][:, cut + 1:cut + 3]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("N,rate,tail", [(64, 6.0, 4), (9000, 0.125, 200)])
@pytest.mark.parametrize("with_cut", [False, True])
def test_growth_beyond_fp32_of_nothing_is_nothing(N, rate, tail, kind, with_cut):
    """Gates above 1 over rows without an input: the product of a run's gates is infinite, what enters it is 0."""
    from bwd_la_fwd_gb300 import la
    C = 8
    gen = torch.Generator().manual_seed(N)
    some = R.normal(gen, 1, tail, C, kind=kind)
    w = torch.full((1, N, C), rate).to(R.TYPES[kind])
    x, dh = torch.zeros_like(w), torch.zeros_like(w)
    x[:, N - tail:], dh[:, :tail] = some, some
    if with_cut:
        w[:, N // 3] = -math.inf
    ref, tol = R.scan(x, w, "log", None)
    H, last = la.la_gated_scan(x.cuda(), w.cuda(), "log")
    R.assert_within("H", H, ref, tol + R.half_step(kind) * (ref.abs() + tol))
    R.assert_within("h_last", last, ref[:, -1], tol[:, -1])
    H = ref.to(R.TYPES[kind])
    refs, tols = R.scan_backward(x, w, H, dh, "log", None, None)
    got = la.la_gated_scan_backward(*(t.cuda() for t in (x, w, H, dh)), "log")
    for name, g, r, t in zip(("dX", "dW"), got, refs, tols):
        R.assert_within(name, g, r, t + R.half_step(kind) * (r.abs() + t))
    R.assert_within("dh0", got[2], refs[2], tols[2])
