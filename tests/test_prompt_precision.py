"""la_prompt on tensor cores: what its bf16 operands may add to the output's own rounding."""
import math

import pytest
import torch

import ops_testutil as R
from test_prompt import _offsets, _state, _tokens


def _over_rounding(O, ref):
    """The error's norm over that of the exact output's own rounding to bf16."""
    ref = ref.double().cpu()
    return float((O.double().cpu() - ref).norm() / (ref.to(torch.bfloat16).double() - ref).norm())


@pytest.mark.gpu
@pytest.mark.parametrize("D", [32, 64, 128])
def test_weights_of_a_sequence_s_first_rows_keep_sixteen_bits(D):
    """Each weight rounded to bf16 would err as the output's own rounding does: the sum of i weights' errors, relative to
    O, is sqrt(i) / i over 1 / sqrt(i), so the first chunk would be off by sqrt(2) of the rounding.  In two parts it adds
    nothing; S, rounded, enters O by a share of 1 / sqrt(D) (of unit V and Q, K of variance 1 / D): sqrt(1 + 1 / D), 1.02
    at most.  1.2 tells the two apart."""
    from bwd_la_fwd_gb300 import la
    lens = [128, 512, 500]
    off = _offsets(lens)
    q, k, v = _tokens(off[-1], 4, 2, D, "bf16", seed=D)
    O = la.la_prompt(q, k, v, torch.tensor(off, dtype=torch.int32, device="cuda"))
    (ref, _), _ = R.prompt(q, k, v, off, R.empty_state(len(lens), 2, D), "bf16", True)
    for lo, hi in zip(off, off[1:]):
        assert _over_rounding(O[lo:lo + 128], ref[lo:lo + 128]) <= 1.2
        assert _over_rounding(O[lo:hi], ref[lo:hi]) <= 1.2


@pytest.mark.gpu
@pytest.mark.parametrize("D", [32, 64, 128])
def test_z_keeps_sixteen_bits(D):
    """301 equal rows k = c, of which the first has v = 1 and the others 0, then rows the same with v = 0: z = 301 c takes
    nine bits, everything else is exact, q . k = 8, and O = 1 / m for the m-th row.  z in one bf16 would put 8 / 9 of
    1 / 301 into every row, twice the output's own rounding; in two parts nothing is added to that but fp32's."""
    from bwd_la_fwd_gb300 import la
    first, more, r = 301, 200, 3
    q = torch.full((first + more, r, D), 0.5, dtype=torch.bfloat16, device="cuda")
    k = torch.full((first + more, 1, D), 16.0 / D, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    v[0] = 1.0
    state = _state(1, 1, D, "bf16")
    for lo, hi, resume in ((0, first, False), (first, first + more, True)):
        off = torch.tensor([0, hi - lo], dtype=torch.int32, device="cuda")
        O = la.la_prompt(q[lo:hi], k[lo:hi], v[lo:hi], off, state, resume=resume)
        ref = (1.0 / torch.arange(lo + 1, hi + 1, dtype=torch.float64))[:, None, None].expand(hi - lo, r, D)
        for h in range(r):
            assert _over_rounding(O[:, h], ref[:, h]) <= 1.05
    assert math.isclose(float(state.z[0, 0, 0]), 501 * 16.0 / D)
