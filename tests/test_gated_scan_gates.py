"""Gates at the ends of their range: the types' lowest values as masks, infinities, NaN."""
import math

import pytest
import torch

import ops_testutil as R
from test_gated_scan import _inputs

LOWEST = [float(torch.finfo(torch.bfloat16).min), float(torch.finfo(torch.float32).min)]


def _gate_values(kind):
    """Every kind of gate: dense where e^w is a normal number, past both its ends, the types' lowest and highest values."""
    w = torch.cat([torch.linspace(-104.0, 0.0, 4001), -torch.logspace(-8, 38.5, 600), torch.tensor(LOWEST),
                   torch.tensor([-math.inf, math.nan, -0.0])])
    return w.to(R.TYPES[kind])


def _check_gate(name, got, want, half_steps, kind):
    """`want` in 64 bits; below 2^-126 the hardware's 2^x is 0."""
    R.assert_within(name, got, want, half_steps * R.U * want.abs() + 2.0 ** -126 + R.half_step(kind) * want.abs() * (1 + 1e-6))


@pytest.mark.gpu
@pytest.mark.parametrize("gate", ["log", "sigmoid"])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_the_gate_itself(kind, gate):
    """One row from 1 without an input is a, and from 0 with an input of 1 is b: forward, step and backward against 64
    bits.  e^w: the hardware's 2^x within 2 ulp (4 half steps) and a rounding; the sigmoid: of e^-|w|'s 5, 1 + e's, the
    reciprocal's 1 ulp and the product's, at most 9.  Then the output's rounding."""
    from bwd_la_fwd_gb300 import la
    w = _gate_values(kind)
    if gate == "sigmoid":
        w = torch.cat([w, -w])
    w = w[: len(w) // 8 * 8]
    W = w.cuda()[None, None]
    x0, x1 = torch.zeros_like(W), torch.ones_like(W)
    h0, h1 = torch.zeros(1, len(w), device="cuda"), torch.ones(1, len(w), device="cuda")
    a, b = R.gates(w.double(), gate)
    steps = 5 if gate == "log" else 9
    H, last = la.la_gated_scan(x0, W, gate, h0=h1)
    _check_gate("a", H[0, 0], a, steps, kind)
    _check_gate("a in fp32", last[0], a, steps, "f32")
    state = h1.clone()
    h = la.la_gated_scan_step(state, x0[:, 0], W[:, 0], gate)
    assert torch.equal(torch.nan_to_num(h, 2.0), torch.nan_to_num(H[:, 0], 2.0))
    _check_gate("state", state[0], a, steps, "f32")
    H, last = la.la_gated_scan(x1, W, gate, h0=h0)
    _check_gate("b", H[0, 0], torch.where(torch.isnan(a), a, b), steps, kind)
    # dh0 = a, dX = b, dW = a h0 (log) or a b h0 (sigmoid)
    dx, dw, dh0 = la.la_gated_scan_backward(x0, W, x1, x1, gate, h0=h1)
    _check_gate("dh0", dh0[0], a, steps, "f32")
    _check_gate("dX", dx[0, 0], torch.ones_like(a) if gate == "log" else b, steps, kind)
    _check_gate("dW", dw[0, 0], a if gate == "log" else a * b, 2 * steps + 2, kind)


@pytest.mark.gpu
def test_growing_log_gates():
    """e^w up to fp32's end, and infinite past it."""
    from bwd_la_fwd_gb300 import la
    w = torch.cat([torch.linspace(0.0, 88.72, 2000), torch.linspace(88.73, 200.0, 100), torch.tensor([1e30, 3e38, math.inf, -1.0])])
    W = w.cuda()[None, None]
    want = torch.exp(w.double())
    want[want > float(torch.finfo(torch.float32).max)] = math.inf
    H, _ = la.la_gated_scan(torch.zeros_like(W), W, "log", h0=torch.ones(1, len(w), device="cuda"))
    _check_gate("a", H[0, 0], want, 5, "f32")


@pytest.mark.gpu
@pytest.mark.parametrize("lowest", LOWEST)
@pytest.mark.parametrize("gate", ["log", "sigmoid"])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_the_lowest_value_cuts_like_minus_infinity(kind, gate, lowest):
    """Restarts marked by the types' lowest finite values have the bits of restarts marked by -inf."""
    from bwd_la_fwd_gb300 import la
    x, w, h0, dh, dl = _inputs(2, 700, 40, kind, gate, seed=8)
    where = torch.rand(w.shape, generator=torch.Generator().manual_seed(1)) < 0.01
    w[:, 100] = 0.0
    where[:, 100] = True
    x, h0, dh, dl = (t.cuda() for t in (x, h0, dh, dl))
    outs = []
    for mask in (-math.inf, lowest):
        W = torch.where(where, torch.tensor(mask, dtype=torch.float32), w.float()).to(R.TYPES[kind]).cuda()
        H, last = la.la_gated_scan(x, W, gate, h0=h0)
        state = h0.clone()
        h = la.la_gated_scan_step(state, x[:, 0], W[:, 100], gate)
        outs.append((H, last, *la.la_gated_scan_backward(x, W, H, dh, gate, h0=h0, dh_last=dl), h, state))
    assert all(bool(torch.isfinite(t).all()) for t in outs[0])
    assert all(torch.equal(a, b) for a, b in zip(*outs))
