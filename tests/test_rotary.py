"""Rotary positions: la_rotary and la_rotary_backward against the rotation in 64 bits (bounds in ops_testutil)."""
import ctypes

import pytest
import torch

import ops_testutil as R


def _case(B, Hq, Hk, N, D, kind, seed=0, fused=False):
    gen = torch.Generator().manual_seed(seed)
    if fused:
        x = R.normal(gen, B, N, Hq + 2 * Hk, D, kind=kind).cuda()
        return x[:, :, :Hq].transpose(1, 2), x[:, :, Hq:Hq + Hk].transpose(1, 2), x
    return R.normal(gen, B, Hq, N, D, kind=kind).cuda(), R.normal(gen, B, Hk, N, D, kind=kind).cuda(), None


def _check(name, got, x, pos, freq, dim, inter, mag, inverse, kind):
    y, tol = R.rotary(x, pos, freq, dim, inter, mag, inverse)
    rounded = torch.zeros_like(y)
    rounded[..., :dim] = R.half_step(kind) * (y[..., :dim].abs() + tol[..., :dim])  # copied channels are exact
    R.assert_within(name, got, y, tol + rounded)


# ------------------------------------------------------------------------------------------------ without a GPU

def test_frequencies_are_the_formula_s():
    from bwd_la_fwd_gb300 import la
    two_pi = 2 * torch.pi
    for kw in ({}, dict(scaling="linear", factor=4.0), dict(scaling="by_turns", factor=8.0, original_length=8192.0)):
        for dim in (2, 6, 64, 256):
            got = torch.tensor([v / 2.0 ** 64 * two_pi for v in la.la_rotary_frequencies(dim, 10000.0, **kw).values],
                               dtype=torch.float64)
            want = R.frequencies(dim, 10000.0, **kw)
            # a few roundings in 64 bits, and the fixed point's own: half of 2^-64 turns is pi 2^-64 radians
            assert bool(((got - want).abs() <= 8 * 2.0 ** -53 * want + torch.pi * 2.0 ** -64).all())
    plain, turns = (la.la_rotary_frequencies(128, 10000.0, **kw).values for kw in
                    ({}, dict(scaling="by_turns", factor=8.0, original_length=8192.0)))
    assert turns[0] == plain[0]                                # many turns: unchanged
    assert abs(turns[63] * 8 - plain[63]) <= plain[63] * 2.0 ** -50 + 8  # few turns: divided (and rounded to units)


@pytest.mark.parametrize("kw", [dict(rotary_dim=3), dict(rotary_dim=0), dict(rotary_dim=64, base=0.5),
                                dict(rotary_dim=64, base=float("nan")), dict(rotary_dim=64, scaling="linear", factor=0.5),
                                dict(rotary_dim=64, scaling="by_turns", factor=2.0),
                                dict(rotary_dim=64, scaling="by_turns", factor=2.0, original_length=100.0, low_turns=4.0,
                                     high_turns=4.0), dict(rotary_dim=258)])
def test_frequencies_refused(kw):
    from bwd_la_fwd_gb300 import la
    with pytest.raises(la.LAError):
        la.la_rotary_frequencies(**kw)


def _abi(lib, q=0x10000, k=0x20000, qr=0x30000, kr=0x40000, pos=None, pstride=0, mag=1.0, B=1, Hq=2, Hk=1, N=4, D=64,
         dim=64, dtype=1, strides=None):
    f = (ctypes.c_ulonglong * 128)()
    st = None if strides is None else (ctypes.c_longlong * len(strides))(*strides)
    return lib.la_rotary(q, k, qr, kr, f, pos, pstride, 0, 0, mag, B, Hq, Hk, N, D, dim, dtype, st, None)


def test_rotary_refuses_on_the_host():
    from bwd_la_fwd_gb300 import la
    lib = la.load_library()
    INVALID, UNSUPPORTED = 1, 2
    assert _abi(lib, dtype=5) == INVALID
    assert _abi(lib, q=None) == INVALID and _abi(lib, kr=None) == INVALID
    assert _abi(lib, q=0x10008) == INVALID
    assert _abi(lib, dim=63) == INVALID and _abi(lib, dim=66) == INVALID and _abi(lib, dim=0) == INVALID
    assert _abi(lib, D=264, dim=64) == UNSUPPORTED and _abi(lib, D=36, dim=32) == UNSUPPORTED
    assert _abi(lib, mag=float("nan")) == INVALID
    assert _abi(lib, pos=0x50000, pstride=3) == INVALID
    assert _abi(lib, qr=0x10000 + 64) == INVALID          # meets its input without being it
    assert _abi(lib, kr=0x30000) == INVALID               # outputs meet
    assert _abi(lib, qr=0x20000) == INVALID               # Q's output on K
    assert _abi(lib, pos=0x30000) == INVALID              # positions inside an output
    assert _abi(lib, strides=[512, 256, 60] + [256, 256, 64] + [512, 256, 64] + [256, 256, 64]) == INVALID  # 16 bytes
    assert _abi(lib, strides=[512, 32, 64] + [256, 256, 64] + [512, 256, 64] + [256, 256, 64]) == INVALID   # rows overlap
    assert _abi(lib, N=0) == 0 and _abi(lib, B=0) == 0    # nothing to do


def test_binding_refuses():
    from bwd_la_fwd_gb300 import la
    f = la.la_rotary_frequencies(64)
    q = torch.empty(1, 2, 8, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        la.la_rotary(q, None, f)
    with pytest.raises(ValueError):
        la.la_rotary(q, torch.empty(1, 2, 9, 64, dtype=torch.bfloat16), f)
    with pytest.raises(ValueError, match="positions"):
        la.la_rotary(q, None, f, positions=torch.zeros(8, dtype=torch.int64))
    with pytest.raises(ValueError, match="contiguous"):
        la.la_rotary(torch.empty(1, 2, 64, 8, dtype=torch.bfloat16).transpose(2, 3), None, f)
    with pytest.raises(TypeError):
        la.la_rotary(q.half(), None, f)


# --------------------------------------------------------------------------------------------------- on the GPU

CASES = [  # B, Hq, Hk, N, D, rotated, interleaved, kind, fused
    (1, 1, 1, 1, 16, 16, False, "bf16", False),
    (2, 4, 2, 37, 128, 128, False, "bf16", True),
    (2, 4, 2, 37, 128, 128, True, "bf16", True),
    (3, 3, 1, 65, 64, 32, False, "bf16", False),
    (1, 8, 8, 130, 64, 20, False, "bf16", True),    # halves of 10: pairs of two channels
    (1, 9, 2, 33, 256, 6, False, "bf16", False),    # halves of 3: single channels
    (2, 2, 1, 19, 32, 10, True, "bf16", False),     # a vector half turned, half copied
    (2, 5, 3, 40, 128, 64, True, "f32", True),
    (1, 2, 2, 50, 24, 24, False, "f32", False),
    (1, 2, 2, 50, 36, 14, False, "f32", False),
    (1, 17, 0, 300, 128, 128, False, "bf16", False),  # no K; more heads than a thread takes
]


@pytest.mark.gpu
@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("B,Hq,Hk,N,D,dim,inter,kind,fused", CASES)
def test_rotary_matches_the_formula(B, Hq, Hk, N, D, dim, inter, kind, fused, inverse):
    from bwd_la_fwd_gb300 import la
    q, k, _ = _case(B, Hq, max(Hk, 1), N, D, kind, seed=N + D, fused=fused)
    k = k if Hk else None
    gen = torch.Generator().manual_seed(1)
    pos = torch.randint(-50, 1000000, (B, N), generator=gen, dtype=torch.int32)
    kw = dict(scaling="by_turns", factor=8.0, original_length=8192.0)
    f, mag = la.la_rotary_frequencies(dim, 10000.0, **kw), 1.25
    call = la.la_rotary_backward if inverse else la.la_rotary
    qr, kr = call(q, k, f, positions=pos.cuda(), interleaved=inter, magnitude=mag)
    for name, got, x in (("Q", qr, q), ("K", kr, k)):
        if x is not None:
            _check(name, got, x, pos, R.frequencies(dim, 10000.0, **kw), dim, inter, mag, inverse, kind)


@pytest.mark.gpu
def test_shared_and_implied_positions():
    from bwd_la_fwd_gb300 import la
    q, k, _ = _case(3, 2, 1, 20, 64, "f32")
    f = la.la_rotary_frequencies(64)
    pos = torch.arange(7, 27, dtype=torch.int32)
    want = la.la_rotary(q, k, f, positions=pos.expand(3, 20).contiguous().cuda())
    for got in (la.la_rotary(q, k, f, positions=pos.cuda()), la.la_rotary(q, k, f, first_position=7),
                la.la_rotary(q, k, f, positions=pos.cuda().expand(3, 20))):
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    _check("Q", want[0], q, pos.expand(3, 20), R.frequencies(64), 64, False, 1.0, False, "f32")


@pytest.mark.gpu
@pytest.mark.parametrize("inter", [False, True])
def test_in_place_on_a_fused_projection(inter):
    """Q and K turned in place inside one projection's output: V and the channels past the rotated ones stay."""
    from bwd_la_fwd_gb300 import la
    q, k, x = _case(2, 4, 2, 33, 64, "bf16", fused=True)
    before = x.clone()
    f = la.la_rotary_frequencies(24)
    want = la.la_rotary(q, k, f, first_position=3, interleaved=inter)
    la.la_rotary(q, k, f, first_position=3, interleaved=inter, Q_out=q, K_out=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert torch.equal(x[:, :, 6:], before[:, :, 6:]) and torch.equal(x[..., 24:], before[..., 24:])


@pytest.mark.gpu
def test_backward_is_the_transposed_map():
    """<dy, R x> = <R^T dy, x>, and R is linear, so R^T dy is the gradient; fp32, so both sides to their roundings."""
    from bwd_la_fwd_gb300 import la
    q, _, _ = _case(1, 2, 1, 30, 64, "f32", seed=3)
    dy, _, _ = _case(1, 2, 1, 30, 64, "f32", seed=4)
    f = la.la_rotary_frequencies(48)
    kw = dict(first_position=1000, magnitude=0.75, interleaved=True)
    y, dx = la.la_rotary(q, None, f, **kw)[0], la.la_rotary_backward(dy, None, f, **kw)[0]
    left, right = (dy.double() * y.double()).sum(), (dx.double() * q.double()).sum()
    size = (dy.double().abs() * q.double().abs()).sum() * 2
    assert abs(float(left - right)) <= 2 * 14 * R.U * float(size)


@pytest.mark.gpu
def test_rotary_in_a_graph_and_on_another_stream():
    """A decode step's positions live on the device: a captured call follows them."""
    from bwd_la_fwd_gb300 import la
    q, k, _ = _case(4, 8, 2, 1, 128, "bf16")
    f = la.la_rotary_frequencies(128)
    pos = torch.zeros(4, 1, dtype=torch.int32, device="cuda")
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        la.la_rotary(q, k, f, positions=pos, Q_out=qo, K_out=ko, stream=side)
    for p in (5, 123456):
        pos.fill_(p)
        graph.replay()
        want = la.la_rotary(q, k, f, first_position=p)
        assert torch.equal(qo, want[0]) and torch.equal(ko, want[1])
    got = la.la_rotary(q, k, f, first_position=9, stream=side)  # outputs allocated for that stream
    side.synchronize()
    want = la.la_rotary(q, k, f, first_position=9)
    assert torch.equal(got[0], want[0])


@pytest.mark.gpu
def test_copied_channels_keep_their_bits():
    from bwd_la_fwd_gb300 import la
    q = torch.full((1, 1, 2, 32), float("nan"), dtype=torch.bfloat16, device="cuda")
    q.view(torch.int16)[..., 16:] = torch.arange(0x7F00, 0x7F10, dtype=torch.int16, device="cuda")
    for inter in (False, True):
        y, _ = la.la_rotary(q, None, la.la_rotary_frequencies(16), interleaved=inter)
        assert torch.equal(y.view(torch.int16)[..., 16:], q.view(torch.int16)[..., 16:])


@pytest.mark.gpu
@pytest.mark.parametrize("B,N", [(0, 3), (2, 0)])
def test_rotary_of_nothing(B, N):
    from bwd_la_fwd_gb300 import la
    f = la.la_rotary_frequencies(64)
    Q, K = la.la_rotary(torch.empty(B, 4, N, 64, device="cuda"), torch.empty(B, 2, N, 64, device="cuda"), f)
    assert Q.shape == (B, 4, N, 64) and K.shape == (B, 2, N, 64)
