"""The selective scan over nearly as many rows as an int numbers (140 to 180 GB on the device): one sequence in parts of millions,
and a token of as many sequences."""
import pytest
import torch

from ops_testutil import U

pytestmark = pytest.mark.gpu


def test_most_rows():
    """Tokens in the last rows only, in a sequence that forgets: what a call on these rows alone gives.  A state remembers some 2.5
    rows (decays of e^-0.5 and less), each of them within 20 half steps; outputs are rounded to bf16, where a difference in
    fp32 may be a step."""
    from bwd_la_fwd_gb300 import la
    if torch.cuda.get_device_properties(0).total_memory < 200 * 2 ** 30:
        pytest.skip("needs 200 GB")
    T, C, S, last = 2 ** 31 - 1100, 8, 8, 1000
    gen = torch.Generator(device="cuda").manual_seed(0)
    new = lambda v, *s: torch.full((1, T, *s), v, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    x, dt, b, y = new(0.0, C), new(0.5, C), new(0.0, 1, S), new(3.0, C)
    for t in (x, b):
        t[:, -last:] = torch.randn(t[:, -last:].shape, generator=gen, device="cuda").bfloat16()
    A = -torch.arange(1, S + 1, device="cuda").float().repeat(C, 1)
    h, few = (torch.empty(1, C, S, device="cuda") for _ in range(2))
    la.la_selective_scan(x, dt, A, b, b, softplus=False, state_out=h, Y=y)
    z = la.la_selective_scan(*(t[:, -last:] for t in (x, dt)), A, b[:, -last:], b[:, -last:], softplus=False, state_out=few)
    assert float((h - few).abs().max()) <= 2 * 2.5 * 20 * U * 16  # inputs are under 4, their products under 16
    assert ((y[:, -last:].float() - z.float()).abs() <= 2.0 ** -7 * z.float().abs() + 2 * 2.5 * 20 * U * 16 * 4 * S).all()
    assert not y[:, :-last:100003].any() and not y[:, :1000].any()
    del x, dt, b, y
    torch.cuda.empty_cache()


def test_a_token_of_most_sequences():
    """The last and some other sequences: the bits of a call on them alone."""
    from bwd_la_fwd_gb300 import la
    if torch.cuda.get_device_properties(0).total_memory < 200 * 2 ** 30:
        pytest.skip("needs 200 GB")
    n, S, some = 2 ** 31 - 1100, 8, 1001
    gen = torch.Generator(device="cuda").manual_seed(1)
    bc = torch.zeros(n, 1, S, device="cuda", dtype=torch.bfloat16)  # B, C and (its first channel) x and dt
    y = torch.full((n, S), 3.0, device="cuda", dtype=torch.bfloat16)
    state = torch.zeros(n, 1, S, device="cuda")
    places = [slice(0, some), slice(n // 2, n // 2 + some), slice(n - some, n)]
    for s in places:
        bc[s] = torch.randn(bc[s].shape, generator=gen, device="cuda").bfloat16()
        state[s] = torch.randn(state[s].shape, generator=gen, device="cuda")
    A = -torch.arange(1, S + 1, device="cuda").float()[None]
    before = [state[s].clone() for s in places]
    x = bc[:, 0, :1]
    la.la_selective_scan_step(state, x, x, A, bc, bc, y=y[:, :1])
    for s, h in zip(places, before):
        z = torch.empty(some, S, device="cuda", dtype=torch.bfloat16)[:, :1]
        la.la_selective_scan_step(h, x[s], x[s], A, bc[s], bc[s], y=z)
        assert torch.equal(y[s, :1], z) and torch.equal(state[s], h)
    assert (y[:, 1:][::100003] == 3).all() and not y[some:n // 2, 0][::10007].any()
    del bc, x, y, state
    torch.cuda.empty_cache()
