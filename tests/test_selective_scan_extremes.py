"""Rates A at the end of fp32's range, whose exponents pass it."""
import pytest
import torch

import state_space_testutil as R
from test_selective_scan import GRADS, _case, _options, _rows

pytestmark = pytest.mark.gpu


def _cuda(c):
    return {k: v.cuda()[None] if k in ("x", "dt", "z", "B", "C") else v.cuda() for k, v in c.items()}


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("S", [8, 16, 32])
def test_states_that_a_row_forgets(S, kind):
    """Some states keep nothing from one row to the next (A = -3e38); the last tile is not full, and its missing rows leave the
    others as they are.  Forward, token and gradients."""
    from bwd_la_fwd_gb300 import la
    T, C = 50, 24
    c, dy, st, dl = _case(T, C, 1, S, 1, kind, S)
    c["A"][::2, ::3] = -3e38
    g, opt = _cuda(c), {}
    opt = _options(g)
    marks, last = la.new_selective_scan_marks(T, 1, C, S), torch.empty(1, C, S, device="cuda")
    Y = la.la_selective_scan(*_rows(g), **opt, state_in=st.cuda(), state_out=last, marks=marks)
    (y, h), (ey, eh) = R.scan(*_rows(c), c["D"], c["z"], c["bias"], True, [0, T], st)
    R.assert_within("Y", Y[0], y, R.rounded(y, ey, kind))
    R.assert_within("state", last, h, eh)
    state = st.cuda()
    rows = []
    for t in range(T):
        one = {k: v[:, t] if k in ("x", "dt", "z", "B", "C") else v for k, v in g.items()}
        rows.append(la.la_selective_scan_step(state, *_rows(one), **_options(one)))
    R.assert_within("tokens", torch.cat(rows), y, R.rounded(y, ey, kind))
    R.assert_within("their state", state, h, eh)
    got = la.la_selective_scan_backward(*_rows(g), dy.cuda()[None], marks, **opt, dstate_out=dl.cuda())
    ref, tol = R.scan_backward(*_rows(c), dy, c["D"], c["z"], c["bias"], True, [0, T], st, dl)
    for name in GRADS + ("dstate_in",):
        t, typed = getattr(got, name), name in ("dX", "ddt", "dz", "dB", "dC")
        R.assert_within(name, t.reshape(ref[name].shape), ref[name], R.rounded(ref[name], tol[name], kind) if typed else tol[name])


@pytest.mark.parametrize("T", [1, 33])
def test_steps_of_zero_change_nothing(T):
    """Whatever A is."""
    from bwd_la_fwd_gb300 import la
    C, S = 64, 16
    z, bc, st = torch.zeros(2, T, C, device="cuda"), torch.ones(2, T, 1, S, device="cuda"), torch.randn(2, C, S, device="cuda")
    A = torch.tensor([-3.4e38, 3.4e38, -1.0, 0.0], device="cuda").repeat(C, S // 4)
    last = torch.empty_like(st)
    la.la_selective_scan(z, z, A, bc, bc, softplus=False, state_in=st, state_out=last)
    assert torch.equal(st, last)
    la.la_selective_scan_step(last, z[:, 0], z[:, 0], A, bc[:, 0], bc[:, 0], softplus=False)
    assert torch.equal(st, last)
