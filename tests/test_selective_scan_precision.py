"""What the selective scan's fp32 arithmetic leaves after many rows."""
import pytest
import torch

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
