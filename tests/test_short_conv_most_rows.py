"""The short convolution of nearly as many rows as an int numbers (100 GB on the device)."""
import pytest
import torch

from ops_testutil import U

pytestmark = pytest.mark.gpu


def test_most_rows():
    """The rows at the end, in runs of millions of rows, equal those of a call on them alone, forward and gradient."""
    from bwd_la_fwd_gb300 import la
    if torch.cuda.get_device_properties(0).total_memory < 150 * 2 ** 30:
        pytest.skip("needs 150 GB")
    T, C, K, last = 2 ** 31 - 1100, 8, 4, 1000
    gen = torch.Generator(device="cuda").manual_seed(0)
    x = torch.zeros(1, T, C, device="cuda", dtype=torch.bfloat16)
    for s in (slice(0, last), slice(T // 2, T // 2 + last), slice(T - 2 * last, T)):
        x[:, s] = torch.randn(x[:, s].shape, generator=gen, device="cuda").bfloat16()
    w = torch.randn(C, K, generator=gen, device="cuda")
    o = torch.full_like(x, 3.0)
    after = torch.empty(1, K - 1, C, device="cuda", dtype=x.dtype)
    la.la_short_conv(x, w, O=o, state_out=after)
    state = lambda a: x[:, a - K + 1:a].contiguous()  # noqa: E731
    assert torch.equal(after, state(T))
    for a in (T // 2, T - last):
        assert torch.equal(o[:, a:a + last], la.la_short_conv(x[:, a:a + last], w, state_in=state(a))), a
    assert torch.equal(o[:, :last], la.la_short_conv(x[:, :last], w))
    dx, dw, db = la.la_short_conv_backward(x, w, x, dX=o)
    few, _, _ = la.la_short_conv_backward(x[:, -last:], w, x[:, -last:])
    assert torch.equal(dx[:, -last:], few)
    few, _, _ = la.la_short_conv_backward(x[:, :last], w, x[:, :last])
    assert torch.equal(dx[:, :last - K + 1], few[:, :last - K + 1])
    # all rows but those of three stretches are zeros, so the sums are those of the stretches: 3000 rows' terms, each added with
    # a rounding of the sum's sizes, on both sides
    rows = [x[:, a:b] for a, b in ((0, last + 8), (T // 2 - 8, T // 2 + last + 8), (T - 2 * last - 8, T))]
    parts = [la.la_short_conv_backward(t, w, t)[1:] for t in rows]
    size = sum(float(t.double().abs().sum((0, 1)).max() + t.double().square().sum((0, 1)).max()) for t in rows)
    for k, got in enumerate((dw, db)):
        assert float((got - sum(p[k] for p in parts)).abs().max()) <= 2 * 4 * last * U * size
    del x, o, dx, rows, parts
    torch.cuda.empty_cache()
