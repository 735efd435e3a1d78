"""The selective scan over one row of channels that are no whole 16-byte vectors: such rows need not lie a multiple of 16 bytes
apart, as there is no second one, and a tile's rows behind it are not there."""
import pytest
import torch

import state_space_testutil as R
from test_selective_scan import GRADS, _case, _cuda, _options, _rows

pytestmark = pytest.mark.gpu


def _check(c, dy, st, off, kind, view, offs):
    """Forward with its states and the gradients; `view`: how the call has the rows."""
    from bwd_la_fwd_gb300 import la
    T, C = c["x"].shape
    S, n = c["A"].shape[1], len(off) - 1
    g = {k: view(v) if k in ("x", "dt", "z", "B", "C") else v for k, v in _cuda(c).items()}
    last, marks = torch.full((n, C, S), 9.0, device="cuda"), la.new_selective_scan_marks(T, n, C, S)
    Y = la.la_selective_scan(*_rows(g), **_options(g), seq_offsets=offs, state_in=st.cuda(), state_out=last, marks=marks,
                             Y=view(torch.zeros(T, C, dtype=c["x"].dtype, device="cuda")))
    (y, h), (ey, eh) = R.scan(*_rows(c), c["D"], c["z"], c["bias"], True, off, st)
    R.assert_within("Y", Y.reshape(T, C), y, R.rounded(y, ey, kind))
    R.assert_within("state", last, h, eh)
    if T > 1:
        return  # (contiguous gradients of several rows have to be whole vectors apart)
    ref, tol = R.scan_backward(*_rows(c), dy, c["D"], c["z"], c["bias"], True, off, st, None)
    got = la.la_selective_scan_backward(*_rows(g), view(dy.cuda()), marks, **_options(g), seq_offsets=offs)
    for name in GRADS + ("dstate_in",):
        t, typed = getattr(got, name), name in ("dX", "ddt", "dz", "dB", "dC")
        R.assert_within(name, t.reshape(ref[name].shape), ref[name], R.rounded(ref[name], tol[name], kind) if typed else tol[name])


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("S", [8, 16, 32])
@pytest.mark.parametrize("C", [1, 75, 83])
def test_one_row(C, S, kind):
    c, dy, st, _ = _case(1, C, 1, S, 1, kind, C + S)
    _check(c, dy, st, [0, 1], kind, lambda t: t[None], None)
    _check(c, dy, st, [0, 1], kind, lambda t: t, torch.tensor([0, 1], dtype=torch.int32, device="cuda"))


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_one_row_and_sequences_without_rows(kind):
    c, dy, st, _ = _case(1, 75, 1, 16, 4, kind, 7)
    off = [0, 0, 1, 1, 1]
    _check(c, dy, st, off, kind, lambda t: t, torch.tensor(off, dtype=torch.int32, device="cuda"))


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_a_batch_of_one_row_each(kind):
    """The sequences lie 80 channels apart."""
    B, C = 3, 75
    c, dy, st, _ = _case(B, C, 1, 16, B, kind, 8)

    def view(t):
        if t.dim() == 3:  # B, C
            return t[:, None]
        wide = torch.full((B, 1, 80), 7.0, dtype=t.dtype, device="cuda")
        wide[:, 0, :C] = t
        return wide[:, :, :C]

    _check(c, dy, st, list(range(B + 1)), kind, view, None)


def test_no_rows_of_odd_channels():
    from bwd_la_fwd_gb300 import la
    A = -torch.ones(75, 16, device="cuda")
    e, b = torch.empty(2, 0, 75, device="cuda"), torch.empty(2, 0, 1, 16, device="cuda")
    st, last = torch.randn(2, 75, 16, device="cuda"), torch.empty(2, 75, 16, device="cuda")
    marks = la.new_selective_scan_marks(0, 2, 75, 16)
    la.la_selective_scan(e, e, A, b, b, z=e, state_in=st, state_out=last, marks=marks)
    got = la.la_selective_scan_backward(e, e, A, b, b, e, marks, z=e, dstate_out=st)
    assert torch.equal(st, last) and torch.equal(got.dstate_in, st) and not got.dA.any()
