"""What the selective scan's fp32 arithmetic leaves after many rows."""
import pytest
import torch

from ops_testutil import U

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("k", [3, 6, 8, 11])
def test_decays_are_not_off_to_one_side(k):
    """States that only fade, by 2^-(2^-k) to 2^-(4 2^-k) a row: the mean error of 81,920 of them after 64 rows is 64 times a
    decay's mean error, which may be 2^-26, a quarter of half a step; the errors' spread adds 8 x 5e-8 / sqrt(81,920) = 1.4e-9
    to that mean, seven times which are 1e-8.  (Time is not cut into parts here: rows are few.)"""
    from bwd_la_fwd_gb300 import la
    n, T, C, S = 80, 64, 64, 16
    gen = torch.Generator().manual_seed(k)
    d = 1 + torch.rand(n, T, C, generator=gen)
    A = -(1 + torch.rand(C, S, generator=gen)) * 2.0 ** -k * 0.6931472
    zero, bc = torch.zeros(n, T, C, device="cuda"), torch.zeros(n, T, 1, S, device="cuda")
    last = torch.empty(n, C, S, device="cuda")
    la.la_selective_scan(zero, d.cuda(), A.cuda(), bc, bc, softplus=False, state_in=torch.ones(n, C, S, device="cuda"), state_out=last)
    want = torch.exp(d.double().sum(1)[..., None] * A.double())
    mean = float((last.double().cpu() / want - 1).mean())
    assert abs(mean) <= T * 2.0 ** -26 + 1e-8


def test_the_gradient_of_a_over_many_rows():
    """Terms of dA that are all d: no decay (A = 0), a state and its gradient of one, tokens of zero; so all is exact but the sum
    of 8192 of them.  The sums are of 8 rows, of 16 tiles of these and of their 64 groups, and other sequences add zeros: 88
    roundings.  A tile's 6 + 0.45 steps of a sum from 4096 on loses the fraction each time where the sums of tiles are added
    one behind another: 167 half steps off."""
    from bwd_la_fwd_gb300 import la
    n, T, C, S = 76, 8192, 64, 16  # as many sequences as leave time in one part
    d = (6 + 0.45 * 2.0 ** -11) / 8
    zero, bc = torch.zeros(n, T, C, device="cuda"), torch.zeros(n, T, 1, S, device="cuda")
    dt, A = torch.full((n, T, C), d, device="cuda"), torch.zeros(C, S, device="cuda")
    marks = la.new_selective_scan_marks(n * T, n, C, S)
    la.la_selective_scan(zero, dt, A, bc, bc, softplus=False, state_in=torch.ones(n, C, S, device="cuda"), marks=marks)
    last = torch.zeros(n, C, S, device="cuda")
    last[0] = 1
    got = la.la_selective_scan_backward(zero, dt, A, bc, bc, zero, marks, softplus=False, dstate_out=last)
    want = T * float(dt[0, 0, 0])
    assert float((got.dA.double() - want).abs().max()) <= 88 * U * want
