"""The short causal convolution against its definition in 64 bits (bounds in state_space_testutil)."""
import ctypes
import math

import pytest
import torch

import state_space_testutil as R
from ops_testutil import normal


def _case(T, C, K, nseq, kind, seed):
    gen = torch.Generator().manual_seed(seed)
    x, do = normal(gen, T, C, kind=kind), normal(gen, T, C, kind=kind)
    w, b = torch.randn(C, K, generator=gen), torch.randn(C, generator=gen)
    return x, do, w, b, normal(gen, nseq, K - 1, C, kind=kind)


# ------------------------------------------------------------------------------------------------ without a GPU

@pytest.mark.parametrize("act", ["none", "silu"])
def test_the_gradient_formulas_against_differences(act):
    x, do, w, b, st = (t.double() for t in _case(7, 2, 3, 2, "f32", 1))
    off = [0, 1, 6]
    do[6] = 0

    def loss(x, w, b):
        return float((R.conv(x, w, b, act, off, st)[0][0] * do).sum())

    grads, _ = R.conv_backward(x, w, do, b, act, off, st)
    for k, g in enumerate(grads):
        for at in range(g.numel()):
            ends = []
            for s in (1e-5, -1e-5):
                args = [t.clone() for t in (x, w, b)]
                args[k].view(-1)[at] += s
                ends.append(loss(*args))
            assert abs((ends[0] - ends[1]) / 2e-5 - float(g.reshape(-1)[at])) < 1e-8


def test_refuses_on_the_host():
    from bwd_la_fwd_gb300 import la
    lib = la.load_library()

    def call(x=1 << 20, w=2 << 20, b=None, first=None, o=3 << 20, last=None, off=None, nseq=2, N=4, C=64, K=4, act=0, dtype=1,
             strides=None, ws=None, size=0):
        st = None if strides is None else (ctypes.c_longlong * 4)(*strides)
        return lib.la_short_conv(x, w, b, first, o, last, off, nseq, N, C, K, act, dtype, st, ws, size, None)

    assert call(dtype=2) == 1 and call(act=2) == 1 and call(nseq=-1) == 1 and call(N=-1) == 1 and call(C=0) == 1 and call(K=0) == 1
    assert call(K=1) == 2 and call(K=5) == 2 and call(C=2 ** 24) == 1
    assert call(x=None) == 1 and call(w=None) == 1 and call(o=None) == 1 and call(o=(3 << 20) + 8) == 1 and call(b=5) == 1
    assert call(C=33) == 1 and call(strides=[256, 32, 256, 64]) == 1
    assert call(o=1 << 20) == 1 and call(o=2 << 20) == 1                       # no form in place
    assert call(first=4 << 20, last=4 << 20) == 1 and call(last=3 << 20) == 1 and call(last=(4 << 20) + 2) == 1
    assert call(off=5 << 20) == 3 and call(off=5 << 20, ws=6 << 20, size=128) == 3 and call(off=(5 << 20) + 2, ws=6 << 20, size=256) == 1
    assert call(off=3 << 20, ws=6 << 20, size=256) == 1 and call(off=5 << 20, ws=5 << 20, size=256) == 1
    assert call(nseq=2, N=2 ** 30) == 1 and call(nseq=0) == 0 and call(N=0) == 0

    def back(dx=4 << 20, dw=5 << 20, db=None, ws=16 << 20, size=None, do=3 << 20, off=None, K=4):
        size = lib.la_short_conv_workspace_bytes(64, K) if size is None else size
        return lib.la_short_conv_backward(1 << 20, 2 << 20, None, None, do, dx, dw, db, off, 2, 4, 64, K, 0, 1, None, ws, size, None)

    assert lib.la_short_conv_workspace_bytes(0, 4) == 0 and lib.la_short_conv_workspace_bytes(64, 5) == 0
    assert back(ws=None) == 3 and back(size=256) == 3 and back(dw=None) == 1 and back(dx=3 << 20) == 1 and back(dw=2 << 20) == 1
    assert back(db=5 << 20) == 1 and back(do=None) == 1 and back(dx=16 << 20) == 1 and back(K=5, size=1 << 30) == 2

    def step(x=1 << 20, s=3 << 20, o=4 << 20, n=2, C=64, K=4):
        return lib.la_short_conv_step(x, 2 << 20, None, s, o, n, C, K, 0, 1, None, None)

    assert step(s=None) == 1 and step(s=(3 << 20) + 8) == 1 and step(o=1 << 20) == 1 and step(o=3 << 20) == 1 and step(C=5) == 1
    assert step(K=6) == 2 and step(n=0) == 0


def test_binding_refuses():
    from bwd_la_fwd_gb300 import la
    x, w = torch.empty(2, 4, 64, dtype=torch.bfloat16), torch.empty(64, 4)
    off = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="activation"):
        la.la_short_conv(x, w, activation="relu")
    with pytest.raises(ValueError, match="W"):
        la.la_short_conv(x, w.double())
    with pytest.raises(ValueError, match="bias"):
        la.la_short_conv(x, w, bias=torch.empty(4))
    with pytest.raises(ValueError, match="packed"):
        la.la_short_conv(x, w, seq_offsets=off)
    with pytest.raises(ValueError, match="without seq_offsets"):
        la.la_short_conv(x[0], w)
    with pytest.raises(ValueError, match="seq_offsets"):
        la.la_short_conv(x[0], w, seq_offsets=off.long())
    with pytest.raises(ValueError, match="state_in"):
        la.la_short_conv(x, w, state_in=torch.empty(2, 4, 64, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="CUDA"):
        la.la_short_conv(x, w)
    with pytest.raises(ValueError):
        la.la_short_conv_backward(x, w, x.float())
    with pytest.raises(ValueError, match="state"):
        la.la_short_conv_step(torch.empty(2, 3, 64), x[:, 0], w)


# --------------------------------------------------------------------------------------------------- on the GPU

# lengths of zero, one, fewer than the taps, around a run; several sequences in a run, the last ones without rows
LENGTHS = [[1], [2, 0, 1, 3, 0], [33], [7, 64, 1, 0, 31, 32], [300], [0, 0, 5, 0]]


def _packed(lens, pad):
    off = [pad]
    for n in lens:
        off.append(off[-1] + n)
    return off, off[-1] + pad


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("K", [2, 3, 4])
@pytest.mark.parametrize("lens", LENGTHS)
def test_packed_sequences(lens, K, kind, act):
    """Rows before the first and behind the last sequence stay as they are."""
    from bwd_la_fwd_gb300 import la
    for C, pad, resumed in ((8, 0, True), (1096, 3, False), (72, 5, True)):
        off, T = _packed(lens, pad)
        x, do, w, b, st = _case(T, C, K, len(lens), kind, T + C + K)
        st = st if resumed else None
        (o, last), tol = R.conv(x, w, b, act, off, st)
        offs = torch.tensor(off, dtype=torch.int32, device="cuda")
        O = torch.full((T, C), 3.0, dtype=x.dtype, device="cuda")
        after = torch.full((len(lens), K - 1, C), 9.0, dtype=x.dtype, device="cuda")
        ws = la.new_short_conv_workspace(C, K)
        first = st.cuda() if resumed else None
        la.la_short_conv(x.cuda(), w.cuda(), bias=b.cuda(), activation=act, seq_offsets=offs, state_in=first, state_out=after, O=O,
                         workspace=ws)
        s = slice(off[0], off[-1])
        R.assert_within("O", O[s], o[s], R.rounded(o, tol, kind)[s])
        assert (O[:off[0]] == 3).all() and (O[off[-1]:] == 3).all()
        assert torch.equal(after.cpu().double(), last)
        grads, tols = R.conv_backward(x, w, do, b, act, off, st)
        dX = torch.full((T, C), 3.0, dtype=x.dtype, device="cuda")
        got = la.la_short_conv_backward(x.cuda(), w.cuda(), do.cuda(), bias=b.cuda(), activation=act, seq_offsets=offs,
                                        state_in=first, dX=dX, workspace=ws)
        R.assert_within("dX", dX[s], grads[0][s], R.rounded(grads[0], tols[0], kind)[s])
        assert (dX[:off[0]] == 3).all() and (dX[off[-1]:] == 3).all()
        R.assert_within("dW", got[1], grads[1], tols[1])
        R.assert_within("dbias", got[2], grads[2], tols[2])
        assert la.la_get_status(ws) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("B,N,C", [(1, 1, 8), (3, 2, 40), (2, 65, 264), (4, 500, 64)])
def test_batches_are_sequences_of_one_length(B, N, C, kind):
    from bwd_la_fwd_gb300 import la
    K = 4
    x, do, w, b, st = _case(B * N, C, K, B, kind, B + N)
    off = [i * N for i in range(B + 1)]
    offs = torch.tensor(off, dtype=torch.int32, device="cuda")
    args = dict(bias=b.cuda(), activation="silu", state_in=st.cuda())
    after = [torch.empty(B, K - 1, C, dtype=x.dtype, device="cuda") for _ in range(2)]
    O = la.la_short_conv(x.cuda().view(B, N, C), w.cuda(), state_out=after[0], **args)
    P = la.la_short_conv(x.cuda(), w.cuda(), seq_offsets=offs, state_out=after[1], **args)
    assert torch.equal(O.view(B * N, C), P) and torch.equal(*after)
    (o, _), tol = R.conv(x, w, b, "silu", off, st)
    R.assert_within("O", P, o, R.rounded(o, tol, kind))
    g = la.la_short_conv_backward(x.cuda().view(B, N, C), w.cuda(), do.cuda().view(B, N, C), **args)
    h = la.la_short_conv_backward(x.cuda(), w.cuda(), do.cuda(), seq_offsets=offs, **args)
    assert all(torch.equal(p.reshape(q.shape), q) for p, q in zip(g, h))
    again = la.la_short_conv_backward(x.cuda(), w.cuda(), do.cuda(), seq_offsets=offs, **args)
    assert all(torch.equal(p, q) for p, q in zip(h, again))


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_strided_views_with_odd_channels(kind):
    """Slices of a fused projection, channels that are no whole vector; nothing around the output is written."""
    from bwd_la_fwd_gb300 import la
    B, N, C, wide, K = 2, 37, 83, 256, 4
    gen = torch.Generator().manual_seed(2)
    buf, out = normal(gen, B, N, wide, kind=kind).cuda(), torch.full((B, N, wide), 5.0, dtype=R.TYPES[kind], device="cuda")
    x, o = buf[:, :, 16:16 + C], out[:, :, 96:96 + C]
    w, st = torch.randn(C, K, generator=gen), normal(gen, B, K - 1, C, kind=kind)
    after = torch.empty(B, K - 1, C, dtype=buf.dtype, device="cuda")
    la.la_short_conv(x, w.cuda(), state_in=st.cuda(), state_out=after, O=o)
    flat = x.reshape(B * N, C).cpu()
    (ref, last), tol = R.conv(flat, w, None, "none", [0, N, 2 * N], st)
    R.assert_within("O", o.reshape(B * N, C), ref, R.rounded(ref, tol, kind))
    assert torch.equal(after.cpu().double(), last) and (out[:, :, :96] == 5).all() and (out[:, :, 96 + C:] == 5).all()
    do = normal(gen, B, N, C + 5, kind=kind).cuda()[:, :, :C].contiguous() if C % 8 else None
    dob = torch.zeros(B, N, wide, dtype=buf.dtype, device="cuda")
    dob[:, :, :C] = do
    dx = torch.full((B, N, wide), 5.0, dtype=buf.dtype, device="cuda")
    got = la.la_short_conv_backward(x, w.cuda(), dob[:, :, :C], state_in=st.cuda(), dX=dx[:, :, 8:8 + C])
    grads, tols = R.conv_backward(flat, w, do.reshape(B * N, C).cpu(), None, "none", [0, N, 2 * N], st)
    R.assert_within("dX", got[0].reshape(B * N, C), grads[0], R.rounded(grads[0], tols[0], kind))
    R.assert_within("dW", got[1], grads[1], tols[1])
    assert (dx[:, :, :8] == 5).all() and (dx[:, :, 8 + C:] == 5).all()


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("K", [2, 3, 4])
def test_tokens_continue_a_prompt(K, kind):
    """A prompt, its second part from the state, then single tokens: the rows of the whole sequence, bit for bit."""
    from bwd_la_fwd_gb300 import la
    T, C, n = 60, 136, 3
    x, _, w, b, _ = _case(n * T, C, K, n, kind, K)
    x = x.view(n, T, C).cuda()
    w, b = w.cuda(), b.cuda()
    whole = la.la_short_conv(x, w, bias=b, activation="silu")
    st = [torch.empty(n, K - 1, C, dtype=x.dtype, device="cuda") for _ in range(2)]
    a = la.la_short_conv(x[:, :2], w, bias=b, activation="silu", state_out=st[0])
    c = la.la_short_conv(x[:, 2:50], w, bias=b, activation="silu", state_in=st[0], state_out=st[1])
    rows = [a, c]
    for t in range(50, T):
        rows.append(la.la_short_conv_step(st[1], x[:, t], w, bias=b, activation="silu")[:, None])
    assert torch.equal(torch.cat(rows, 1), whole) and torch.equal(st[1], x[:, T - K + 1:])


@pytest.mark.gpu
def test_sequences_do_not_meet():
    """Infinities and NaN of a sequence, and of rows outside all, have no part in another."""
    from bwd_la_fwd_gb300 import la
    x, do, w, b, _ = _case(50, 64, 4, 3, "f32", 8)
    off = torch.tensor([2, 20, 40, 45], dtype=torch.int32, device="cuda")
    bad = x.clone()
    bad[:2], bad[39], bad[45:] = math.nan, math.inf, math.nan
    args = dict(activation="silu", seq_offsets=off)
    a, c = (la.la_short_conv(t.cuda(), w.cuda(), **args) for t in (x, bad))
    assert torch.equal(a[:39], c[:39]) and torch.equal(a[40:], c[40:])
    worse = do.clone()
    worse[:2], worse[40], worse[45:] = math.nan, math.inf, math.nan
    g, h = (la.la_short_conv_backward(x.cuda(), w.cuda(), t.cuda(), **args)[0] for t in (do, worse))
    assert torch.equal(g[:40], h[:40]) and torch.equal(g[41:], h[41:])


@pytest.mark.gpu
def test_offsets_out_of_order_compute_nothing():
    from bwd_la_fwd_gb300 import la
    x, do, w, b, _ = _case(50, 64, 4, 3, "bf16", 9)
    for off in ([0, 30, 20, 50], [0, 10, 20, 51], [-1, 10, 20, 50]):
        offs = torch.tensor(off, dtype=torch.int32, device="cuda")
        ws = la.new_short_conv_workspace(64, 4)
        O = torch.full((50, 64), 3.0, dtype=x.dtype, device="cuda")
        after = torch.full((3, 3, 64), 3.0, dtype=x.dtype, device="cuda")
        la.la_short_conv(x.cuda(), w.cuda(), seq_offsets=offs, state_out=after, O=O, workspace=ws)
        assert la.la_get_status(ws) == 6 and (O == 3).all() and (after == 3).all()
        dX = torch.full((50, 64), 3.0, dtype=x.dtype, device="cuda")
        got = la.la_short_conv_backward(x.cuda(), w.cuda(), do.cuda(), seq_offsets=offs, dX=dX, workspace=ws)
        assert la.la_get_status(ws) == 6 and (dX == 3).all() and not got[1].any() and not got[2].any()


@pytest.mark.gpu
def test_no_rows_leave_the_state():
    from bwd_la_fwd_gb300 import la
    w = torch.ones(64, 4, device="cuda")
    st = torch.randn(2, 3, 64, device="cuda")
    after = torch.empty_like(st)
    assert la.la_short_conv(torch.empty(2, 0, 64, device="cuda"), w, state_in=st, state_out=after).shape == (2, 0, 64)
    assert torch.equal(after, st)
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    la.la_short_conv(torch.empty(0, 64, device="cuda"), w, seq_offsets=off, state_out=after)
    assert not after.any()
    e = torch.empty(0, 64, device="cuda")
    got = la.la_short_conv_backward(e, w, e, seq_offsets=off, dW=torch.ones_like(w))
    assert not got[1].any() and not got[2].any()


@pytest.mark.gpu
def test_on_another_stream_and_captured():
    from bwd_la_fwd_gb300 import la
    x, do, w, b, _ = (t.cuda() for t in _case(600, 72, 4, 3, "bf16", 10))
    offs = torch.tensor([0, 100, 101, 600], dtype=torch.int32, device="cuda")
    want = la.la_short_conv(x, w, seq_offsets=offs)
    grads = la.la_short_conv_backward(x, w, do, seq_offsets=offs)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = la.la_short_conv(x, w, seq_offsets=offs, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    ws = la.new_short_conv_workspace(72, 4)
    O, out = torch.zeros_like(x), [torch.empty_like(t) for t in grads]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        la.la_short_conv(x, w, seq_offsets=offs, O=O, workspace=ws)
        la.la_short_conv_backward(x, w, do, seq_offsets=offs, dX=out[0], dW=out[1], dbias=out[2], workspace=ws)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(O, want) and all(torch.equal(p, q) for p, q in zip(out, grads))
