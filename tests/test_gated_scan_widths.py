"""The gated recurrence in the wide channel blocks that batches of training take (64 or 32 channels to a CTA; few sequences
of few channels, as in the other tests, take 16)."""
import math

import pytest
import torch

import ops_testutil as R
from test_gated_scan import _inputs

# 240 blocks of 64 channels, then 232 of 32 (116 of 64); the last block has 8 of its channels; several rounds of rows
SHAPES = [(12, 270, 1224), (4, 530, 1832)]


def _run(B, N, C, kind, gate, seed, plant=False, narrow=0):
    """Inputs and outputs of one case; `narrow` channels less than C, inside rows of C."""
    from bwd_la_fwd_gb300 import la
    x, w, h0, dh, dl = _inputs(B, N, C, kind, gate, seed=seed, cuts=0.005)
    if plant:
        cut = N // 2
        w[:, cut] = -math.inf
        x[0, 20], x[1, cut - 1], dh[2, N - 3] = math.inf, math.nan, -math.inf
    c = C - narrow
    x, w, dh = (t[..., :c] for t in (x, w, dh))
    h0, dl = h0[:, :c].contiguous(), dl[:, :c].contiguous()
    ref, tol = R.scan(x, w, gate, h0)
    given = torch.zeros(B, N, C, dtype=R.TYPES[kind])
    given[..., :c] = ref.nan_to_num(posinf=1.0, neginf=1.0).to(R.TYPES[kind])
    given = given[..., :c]
    dev = [torch.zeros(B, N, C, dtype=t.dtype, device="cuda")[..., :c].copy_(t) for t in (x, w, given, dh)]
    out = [torch.full((B, N, C), 5.0, dtype=R.TYPES[kind], device="cuda") for _ in range(3)]
    H, last = la.la_gated_scan(dev[0], dev[1], gate, h0=h0.cuda(), H=out[0][..., :c])
    dx, dw, dh0 = la.la_gated_scan_backward(*dev, gate, h0=h0.cuda(), dh_last=dl.cuda(), dX=out[1][..., :c], dW=out[2][..., :c])
    assert all(bool((o[..., c:] == 5.0).all()) for o in out)
    return (x, w, given, dh, h0, dl), (ref, tol), (H, last, dx, dw, dh0)


@pytest.mark.gpu
@pytest.mark.parametrize("gate", ["log", "sigmoid"])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("narrow", [0, 5])
@pytest.mark.parametrize("B,N,C", SHAPES)
def test_wide_blocks_match_the_definition(B, N, C, narrow, kind, gate):
    (x, w, given, dh, h0, dl), (ref, tol), (H, last, dx, dw, dh0) = _run(B, N, C, kind, gate, seed=N, narrow=narrow)
    R.assert_within("H", H, ref, tol + R.half_step(kind) * (ref.abs() + tol))
    R.assert_within("h_last", last, ref[:, -1], tol[:, -1])
    refs, tols = R.scan_backward(x, w, given, dh, gate, h0, dl)
    for name, g, r, t in zip(("dX", "dW"), (dx, dw), refs, tols):
        R.assert_within(name, g, r, t + R.half_step(kind) * (r.abs() + t))
    R.assert_within("dh0", dh0, refs[2], tols[2])


@pytest.mark.gpu
@pytest.mark.parametrize("gate", ["log", "sigmoid"])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("B,N,C", SHAPES)
def test_cuts_in_wide_blocks(B, N, C, kind, gate):
    """Infinities and NaN before a restart and an infinite gradient behind it leave the other side's bits."""
    _, _, bad = _run(B, N, C, kind, gate, seed=N + 1, plant=True)
    from bwd_la_fwd_gb300 import la
    x, w, h0, dh, dl = _inputs(B, N, C, kind, gate, seed=N + 1, cuts=0.005)
    cut = N // 2
    w[:, cut] = -math.inf
    H, last = la.la_gated_scan(x.cuda(), w.cuda(), gate, h0=h0.cuda())
    assert torch.equal(bad[0][:, cut:], H[:, cut:]) and torch.equal(bad[1], last)
    assert torch.equal(bad[0][0, :20], H[0, :20]) and torch.equal(bad[0][2:], H[2:])
    assert not torch.isfinite(bad[0][0, 20]).any() and torch.isnan(bad[0][1, cut - 1]).all()
    assert torch.isinf(bad[2][2, N - 3]).all()
    assert bool(torch.isfinite(bad[2][2, :cut]).all()) and bool(torch.isfinite(bad[4]).all())
