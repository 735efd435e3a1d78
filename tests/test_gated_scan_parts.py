"""The gated recurrence where few channel blocks have their time cut into parts, the CTAs of a cluster that write to one
another's shared memory."""
import glob
import math
import os
import re

import pytest
import torch

import ops_testutil as R
from test_gated_scan import _inputs

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bwd_la_fwd_gb300", "csrc")


# ------------------------------------------------------------------------------------------------ without a GPU

def test_kernels_meet_before_they_touch_another_cta_s_shared_memory():
    """A CTA's shared memory may be accessed by others of its cluster once it has begun, which only a cluster barrier
    tells: in every kernel's source one that is waited for stands before the first remote access."""
    seen = 0
    for path in glob.glob(os.path.join(CSRC, "*.cu")):
        with open(path) as f:
            text = re.sub(r"//[^\n]*", "", f.read())
        for kernel in text.split("__global__")[1:]:
            remote = kernel.find("map_shared_rank(")
            if remote < 0:
                continue
            seen += 1
            before = kernel[:remote]
            assert "cluster.sync()" in before or "barrier.cluster.wait" in before, os.path.basename(path)
    assert seen >= 4


# --------------------------------------------------------------------------------------------------- on the GPU

# forward in 2, 4 and 16 parts of bf16, 4, 8 and 16 of fp32; the first case has two rounds of rows in a part
SHAPES = [(1, 2048, 8), (3, 5003, 24), (1, 16500, 16)]


@pytest.mark.gpu
@pytest.mark.parametrize("gate", ["log", "sigmoid"])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("B,N,C", SHAPES)
def test_parts_match_the_recurrence(B, N, C, kind, gate):
    """Forward and backward against the definition, and the same bits call after call."""
    from bwd_la_fwd_gb300 import la
    x, w, h0, dh, dl = _inputs(B, N, C, kind, gate, seed=N, cuts=0.002)
    ref, tol = R.scan(x, w, gate, h0)
    H = ref.to(R.TYPES[kind])
    args = [t.cuda() for t in (x, w, h0, H, dh, dl)]
    first = None
    for _ in range(20):
        got = la.la_gated_scan(*args[:2], gate, h0=args[2])
        got += la.la_gated_scan_backward(args[0], args[1], args[3], args[4], gate, h0=args[2], dh_last=args[5])
        first = first or got
        assert all(torch.equal(a, b) for a, b in zip(first, got))
    R.assert_within("H", first[0], ref, tol + R.half_step(kind) * (ref.abs() + tol))
    R.assert_within("h_last", first[1], ref[:, -1], tol[:, -1])
    refs, tols = R.scan_backward(x, w, H, dh, gate, h0, dl)
    for name, g, r, t in zip(("dX", "dW"), first[2:4], refs, tols):
        R.assert_within(name, g, r, t + R.half_step(kind) * (r.abs() + t))
    R.assert_within("dh0", first[4], refs[2], tols[2])


@pytest.mark.gpu
@pytest.mark.parametrize("gate", ["log", "sigmoid"])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_a_cut_keeps_other_parts_infinities_out(kind, gate):
    """Infinities and NaN some parts before the cut, and infinite gradients some parts behind it."""
    from bwd_la_fwd_gb300 import la
    B, N, C, cut = 2, 6000, 16, 4500
    x, w, h0, dh, dl = _inputs(B, N, C, kind, gate, seed=3)
    w[:, cut] = -math.inf
    bad, worse = x.clone(), dh.clone()
    bad[0, 20], bad[1, 2999] = math.inf, math.nan
    worse[0, 5990], worse[1, 4501] = math.inf, math.nan
    x, w, h0, dh, dl, bad, worse = (t.cuda() for t in (x, w, h0, dh, dl, bad, worse))
    (H, last), (H2, last2) = (la.la_gated_scan(t, w, gate, h0=h0) for t in (bad, x))
    assert torch.equal(H[:, cut:], H2[:, cut:]) and torch.equal(last, last2)
    assert torch.equal(H[0, :20], H2[0, :20]) and torch.equal(H[1, :2999], H2[1, :2999])
    assert not torch.isfinite(H[0, 20]).any() and torch.isnan(H[1, 2999]).all()
    a, b = (la.la_gated_scan_backward(x, w, H2, t, gate, h0=h0, dh_last=dl) for t in (worse, dh))
    assert torch.equal(a[0][:, :cut], b[0][:, :cut]) and torch.equal(a[1][:, :cut + 1], b[1][:, :cut + 1])
    assert torch.equal(a[2], b[2])
