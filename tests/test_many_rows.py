"""Rows whose elements are numbered beyond 2^31 (some 40 GB on the device): the last sequences of a large packed call equal
those of a call on them alone."""
import pytest
import torch

pytestmark = pytest.mark.gpu

C, LEN = 1024, 1000
T = 2 ** 31 // C + 4 * LEN  # the last four sequences begin behind element 2^31
LAST = 3                    # sequences compared


@pytest.fixture(scope="module")
def rows():
    if torch.cuda.get_device_properties(0).total_memory < 100 * 2 ** 30:
        pytest.skip("needs 100 GB")
    gen = torch.Generator(device="cuda").manual_seed(0)
    x = torch.randn(T, C, generator=gen, device="cuda", dtype=torch.bfloat16)
    first = T - LAST * LEN
    off = torch.cat([torch.arange(0, first, LEN, device="cuda"), torch.arange(first, T + 1, LEN, device="cuda")]).int()
    yield x, off, torch.arange(0, LAST * LEN + 1, LEN, device="cuda").int(), gen
    torch.cuda.empty_cache()


def test_norm(rows):
    from bwd_la_fwd_gb300 import la
    x, w = rows[0], torch.rand(C, device="cuda")
    y, _ = la.la_rms_norm(x, w)
    assert torch.equal(y[-LEN:], la.la_rms_norm(x[-LEN:], w)[0])
    y8, scales, _ = la.la_rms_norm_8bit(x, w)
    a, s, _ = la.la_rms_norm_8bit(x[-LEN:], w)
    assert torch.equal(y8[-LEN:].view(torch.uint8), a.view(torch.uint8)) and torch.equal(scales[-LEN:], s)
    dx, _ = la.la_rms_norm_backward(x, w, y)
    assert torch.equal(dx[-LEN:], la.la_rms_norm_backward(x[-LEN:], w, y[-LEN:])[0])


def test_convolution(rows):
    from bwd_la_fwd_gb300 import la
    x, off, few, gen = rows
    w = torch.randn(C, 4, generator=gen, device="cuda")
    n, tail = off.numel() - 1, x[-LAST * LEN:]
    last = [torch.empty(k, 3, C, dtype=x.dtype, device="cuda") for k in (n, LAST)]
    o = la.la_short_conv(x, w, activation="silu", seq_offsets=off, state_out=last[0])
    p = la.la_short_conv(tail, w, activation="silu", seq_offsets=few, state_out=last[1])
    assert torch.equal(o[-LAST * LEN:], p) and torch.equal(last[0][-LAST:], last[1])
    dx = la.la_short_conv_backward(x, w, o, activation="silu", seq_offsets=off)[0]
    assert torch.equal(dx[-LAST * LEN:], la.la_short_conv_backward(tail, w, p, activation="silu", seq_offsets=few)[0])


def test_scan(rows):
    """The few sequences alone are cut into parts, so fp32 sums differ in their order: bf16 outputs by a few of their steps
    of 2^-8 of the largest value, where rows from another place would be off by all of it."""
    from bwd_la_fwd_gb300 import la
    x, off, few, gen = rows
    S, n = 8, off.numel() - 1
    dt = torch.randn(T, C, generator=gen, device="cuda", dtype=torch.bfloat16) - 3
    bc = torch.randn(T, 2, S, generator=gen, device="cuda", dtype=torch.bfloat16)
    A = -torch.arange(1, S + 1, device="cuda").float().repeat(C, 1)
    tail = slice(T - LAST * LEN, T)

    def call(rows, off, n):
        args = x[rows], dt[rows], A, bc[rows, :1], bc[rows, 1:]
        last = torch.empty(n, C, S, device="cuda")
        marks = la.new_selective_scan_marks(args[0].shape[0], n, C, S)
        y = la.la_selective_scan(*args, seq_offsets=off, state_out=last, marks=marks)
        g = la.la_selective_scan_backward(*args, x[rows], marks, seq_offsets=off)
        k = LAST * LEN
        return [t.clone() for t in (y[-k:], last[-LAST:], g.dX[-k:], g.ddt[-k:], g.dB[-k:], g.dC[-k:])]

    for a, b in zip(call(slice(0, T), off, n), call(tail, few, LAST)):
        assert float((a.float() - b.float()).abs().max()) <= 2.0 ** -6 * float(b.float().abs().max())
