"""States that grow (A > 0) over sequences that are cut into parts: a part may multiply what it starts from by more than fp32 holds
and leave a number all the same, and zeros stay zeros.  As row by row."""
import pytest
import torch

import state_space_testutil as R
from test_selective_scan import GRADS, _rows

pytestmark = pytest.mark.gpu
C, PART = 16, 128


def _case(T, S, kind, step):
    """Steps of `step` (exact, as their sums are) times A of 1/2 to 1; nothing enters yet."""
    gen = torch.Generator().manual_seed(T + S)
    dtype = R.TYPES[kind]
    z = lambda *s: torch.zeros(*s, dtype=dtype)  # noqa: E731
    return dict(x=z(T, C), dt=torch.full((T, C), step, dtype=dtype), A=0.5 + 0.5 * torch.rand(C, S, generator=gen),
                B=torch.randn(T, 1, S, generator=gen).to(dtype), C=torch.randn(T, 1, S, generator=gen).to(dtype)), z(T, C), gen


def _check(c, dy, st, dl, kind):
    """Folding a part in is four exponentials of a quarter of its exponent e < 140 and their products: 3 e + 4 x 5 + 4 = 444 half
    steps of what it started from, beside the bounds of row after row."""
    from bwd_la_fwd_gb300 import la
    T, S = c["x"].shape[0], c["A"].shape[1]
    g = {k: v.cuda() if k == "A" else v.cuda()[None] for k, v in c.items()}
    off, extra = [0, T], 444
    marks, last = la.new_selective_scan_marks(T, 1, C, S), torch.empty(1, C, S, device="cuda")
    Y = la.la_selective_scan(*_rows(g), softplus=False, state_in=st.cuda(), state_out=last, marks=marks)
    (y, h), (ey, eh) = R.scan(*_rows(c), None, None, None, False, off, st, extra)
    R.assert_within("Y", Y[0], y, R.rounded(y, ey, kind))
    R.assert_within("state", last, h, eh)
    got = la.la_selective_scan_backward(*_rows(g), dy.cuda()[None], marks, softplus=False, dstate_out=dl.cuda())
    ref, tol = R.scan_backward(*_rows(c), dy, None, None, None, False, off, st, dl, extra)
    for name in GRADS + ("dstate_in",):
        if name != "dz":
            t, typed = getattr(got, name), name in ("dX", "ddt", "dB", "dC")
            R.assert_within(name, t.reshape(ref[name].shape), ref[name], R.rounded(ref[name], tol[name], kind) if typed else tol[name])


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("S", [8, 16, 32])
def test_nothing_before_the_last_rows(S, kind):
    """Tokens in the last 40 of 1000 rows, gradients in the first 40."""
    c, dy, gen = _case(1000, S, kind, 1.0)
    c["x"][-40:] = torch.randn(40, C, generator=gen).to(dy.dtype)
    dy[:40] = torch.randn(40, C, generator=gen).to(dy.dtype)
    zero = torch.zeros(1, C, S)
    _check(c, dy, zero, zero, kind)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("S", [8, 16, 32])
def test_a_part_grows_beyond_the_range(S, kind):
    """The second of three parts multiplies by 2^92 to 2^185: states and gradients from some 2^-100 on."""
    c, dy, gen = _case(3 * PART, S, kind, 0.0)
    c["dt"][PART:2 * PART] = 1.0
    small = lambda: torch.randn(1, C, S, generator=gen) * 2.0 ** -100  # noqa: E731
    _check(c, dy, small(), small(), kind)
