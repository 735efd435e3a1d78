"""Rotary positions where each thread turns many heads one after another (long sequences of many heads)."""
import pytest
import torch

import ops_testutil as R
from test_rotary import _case, _check

# 2 x 2500 rows make over 608 blocks of all 40 heads, four thread rows to a block: ten heads to a thread
B, HQ, HK, N, D = 2, 32, 8, 2500, 128


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("inter,dim", [(False, 128), (True, 96), (False, 96)])
def test_many_heads_to_a_thread(inter, dim, kind):
    from bwd_la_fwd_gb300 import la
    q, k, _ = _case(B, HQ, HK, N, D, kind, seed=dim, fused=True)
    pos = torch.randint(0, 100000, (B, N), generator=torch.Generator().manual_seed(2), dtype=torch.int32)
    f = la.la_rotary_frequencies(dim)
    qr, kr = la.la_rotary(q, k, f, positions=pos.cuda(), interleaved=inter)
    for name, got, x in (("Q", qr, q), ("K", kr, k)):
        _check(name, got, x, pos, R.frequencies(dim), dim, inter, 1.0, False, kind)
    la.la_rotary(q, k, f, positions=pos.cuda(), interleaved=inter, Q_out=q, K_out=k)  # in place
    assert torch.equal(q, qr) and torch.equal(k, kr)
