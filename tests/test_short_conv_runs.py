"""The short convolution where a thread walks more rows than are loaded together, and sequences pass from one run to the next."""
import pytest
import torch

import state_space_testutil as R
from test_short_conv import _case, _packed

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("K", [2, 3, 4])
@pytest.mark.parametrize("lens", [[1500], [700, 0, 1, 3, 795]])
def test_long_runs(lens, K, kind, act):
    """Runs of 23 rows forward, 30 backward."""
    from bwd_la_fwd_gb300 import la
    C = 4104
    off, T = _packed(lens, 2)
    x, do, w, b, st = _case(T, C, K, len(lens), kind, T + K)
    (o, last), tol = R.conv(x, w, b, act, off, st)
    args = dict(bias=b.cuda(), activation=act, seq_offsets=torch.tensor(off, dtype=torch.int32, device="cuda"), state_in=st.cuda())
    O, after = torch.full((T, C), 3.0, dtype=x.dtype, device="cuda"), torch.empty(len(lens), K - 1, C, dtype=x.dtype, device="cuda")
    la.la_short_conv(x.cuda(), w.cuda(), state_out=after, O=O, **args)
    s = slice(off[0], off[-1])
    R.assert_within("O", O[s], o[s], R.rounded(o, tol, kind)[s])
    assert (O[:off[0]] == 3).all() and (O[off[-1]:] == 3).all() and torch.equal(after.cpu().double(), last)
    grads, tols = R.conv_backward(x, w, do, b, act, off, st)
    dX, dW, db = la.la_short_conv_backward(x.cuda(), w.cuda(), do.cuda(), **args)
    R.assert_within("dX", dX[s], grads[0][s], R.rounded(grads[0], tols[0], kind)[s])
    R.assert_within("dW", dW, grads[1], tols[1])
    R.assert_within("dbias", db, grads[2], tols[2])
