"""What la_prompt does to the state that it continues from: it keeps all of its bits (64 of them for fp32 tokens)."""
import math

import pytest
import torch

import ops_testutil as R
from test_prompt import _offsets, _state, _tokens


def _fill(state, seed):
    """Values of all 53 bits, of a long cache's sizes, with an infinity and one past fp32's range."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    for t in (state.S, state.z, state.a):
        t.copy_(torch.randn(t.shape, generator=gen, device="cuda", dtype=torch.float64) * 1e6)
    state.n.fill_(1000)
    return [t.clone() for t in (state.S, state.z, state.a, state.n)]


@pytest.mark.gpu
@pytest.mark.parametrize("D", [16, 64, 256])
@pytest.mark.parametrize("rows", [0, 40])
def test_a_sequence_without_rows_keeps_its_state(D, rows):
    from bwd_la_fwd_gb300 import la
    off = _offsets([0, rows, 0])
    q, k, v = _tokens(off[-1], 4, 2, D, "f32", seed=D)
    state = _state(3, 2, D, "f32")
    _fill(state, D)
    state.S[0, 0, 3, 5], state.S[2, 1, 0, 0], state.z[0, 1, 2], state.a[2, 0, 1] = math.inf, -1e300, -math.inf, math.nan
    before = [t.clone() for t in (state.S, state.z, state.a, state.n)]
    la.la_prompt(q, k, v, torch.tensor(off, dtype=torch.int32, device="cuda"), state, resume=True)
    for i in (0, 2) if rows else (0, 1, 2):
        for t, was in zip((state.S, state.z, state.a, state.n), before):
            assert torch.equal(torch.nan_to_num(t[i].double(), 7.0, 8.0, 9.0), torch.nan_to_num(was[i].double(), 7.0, 8.0, 9.0))
            assert torch.equal(torch.isfinite(t[i]), torch.isfinite(was[i]))


@pytest.mark.gpu
@pytest.mark.parametrize("D", [16, 64, 128, 256])
@pytest.mark.parametrize("rows", [0, 200])
def test_a_bf16_sequence_without_rows_keeps_its_state(D, rows):
    """Between sequences with rows and without any; unresumed, it is emptied."""
    from bwd_la_fwd_gb300 import la
    off = _offsets([0, rows, 0])
    q, k, v = _tokens(off[-1], 4, 2, D, "bf16", seed=D)
    state = _state(3, 2, D, "bf16")
    _fill(state, D)
    state.S[0, 0, 3, 5], state.z[0, 1, 2], state.a[2, 0, 1] = math.inf, -math.inf, math.nan
    before = [t.clone() for t in (state.S, state.z, state.a, state.n)]
    o = torch.tensor(off, dtype=torch.int32, device="cuda")
    la.la_prompt(q, k, v, o, state, resume=True)
    for i in (0, 2) if rows else (0, 1, 2):
        for t, was in zip((state.S, state.z, state.a, state.n), before):
            assert torch.equal(torch.nan_to_num(t[i].double(), 7.0, 8.0, 9.0), torch.nan_to_num(was[i].double(), 7.0, 8.0, 9.0))
    la.la_prompt(q, k, v, o, state)
    for i in (0, 2) if rows else (0, 1, 2):
        assert not any(bool(t[i].any()) for t in (state.S, state.z, state.a, state.n))


@pytest.mark.gpu
@pytest.mark.parametrize("lens", [[40], [33, 700, 1], [3000]], ids=str)
@pytest.mark.parametrize("D,Hkv", [(16, 1), (64, 2), (128, 1)])
def test_rows_are_added_to_all_bits_of_the_state(D, Hkv, lens):
    """state + sums: the sums of this call's rows as pairs of floats (2^-44 of their terms' magnitudes, as
    ops_testutil counts them), and the addition rounded once in 64 bits."""
    from bwd_la_fwd_gb300 import la
    off = _offsets(lens)
    q, k, v = _tokens(off[-1], Hkv, Hkv, D, "f32", seed=off[-1])
    state = _state(len(lens), Hkv, D, "f32")
    was = _fill(state, D)
    state.S[0, 0, 1, 2] = was[0][0, 0, 1, 2] = math.inf
    la.la_prompt(q, k, v, torch.tensor(off, dtype=torch.int32, device="cuda"), state, resume=True)
    for i, n in enumerate(lens):
        kd, vd = (t[off[i]:off[i + 1]].double().transpose(0, 1) for t in (k, v))
        for name, got, first, add, size in (("S", state.S, was[0], kd.transpose(1, 2) @ vd, kd.abs().transpose(1, 2) @ vd.abs()),
                                            ("z", state.z, was[1], kd.sum(1), kd.abs().sum(1)),
                                            ("a", state.a, was[2], vd.sum(1), vd.abs().sum(1))):
            want = first[i] + add
            R.assert_within(name, got[i], want, 2.0 ** -44 * (n + 1) * size + 2.0 ** -52 * (first[i].abs() + size).nan_to_num(posinf=0.0))
    assert torch.equal(state.n, was[3] + torch.tensor(lens, dtype=torch.int32, device="cuda")[:, None])


@pytest.mark.gpu
def test_an_infinite_key_leaves_infinite_sums():
    """As plain sums would: inf where one sign of it was added, nothing else of the state touched by it."""
    from bwd_la_fwd_gb300 import la
    T, D = 90, 64
    q, k, v = _tokens(T, 1, 1, D, "f32", seed=4)
    k[50, 0, 3] = math.inf
    state = _state(1, 1, D, "f32")
    la.la_prompt(q, k, v, torch.tensor([0, T], dtype=torch.int32, device="cuda"), state)
    want = k[:, 0].double().T @ v[:, 0].double()
    assert torch.equal(state.S[0, 0, 3], want[3]) and torch.isinf(want[3]).all()
    assert float(state.z[0, 0, 3]) == math.inf
    assert bool(torch.isfinite(state.S[0, 0, :3]).all()) and bool(torch.isfinite(state.S[0, 0, 4:]).all())
    assert bool(torch.isfinite(state.a).all())
