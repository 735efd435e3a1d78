"""Packed prompts with grouped heads (la_prompt) and single tokens of grouped heads (la_decode_step_grouped) against
explicit weights in 64 bits (bounds in ops_testutil)."""
import ctypes
import math

import pytest
import torch

import ops_testutil as R

TENSOR_CORE = {("bf16", 32), ("bf16", 64), ("bf16", 128)}


def _tokens(T, Hq, Hkv, D, kind, seed):
    """Q, K ~ N(0, 1 / D), V ~ N(0, 1) as slices of one projection's output."""
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(T, Hq + 2 * Hkv, D, generator=gen)
    x[:, :Hq + Hkv] /= math.sqrt(D)
    x = x.to(R.TYPES[kind]).cuda()
    return x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]


def _offsets(lens, start=0):
    off = [start]
    for n in lens:
        off.append(off[-1] + n)
    return off


def _state(nseq, Hkv, D, kind):
    from bwd_la_fwd_gb300 import la
    return la.DecodeState(nseq, Hkv, D, R.TYPES[kind])


def _check(O, state, ref, tol, off, name=""):
    (Or, sr), (ot, *st) = ref, tol
    lo, hi = off[0], off[-1]
    R.assert_within(name + "O", O[lo:hi], Or[lo:hi], ot[lo:hi])
    if hi > lo:  # worst cases aside: roundings are not all of one sign, so the whole is within 3 bf16 half steps
        off_by = float((O[lo:hi].double().cpu() - Or[lo:hi]).norm() / Or[lo:hi].norm())
        assert off_by <= (3 * 2.0 ** -8 if O.dtype == torch.bfloat16 else 1e-5), (name, off_by)
    if state is not None:
        for what, got, want, t in zip("Sza", (state.S, state.z, state.a), sr, st):
            R.assert_within(name + what, got, want, t)
        assert torch.equal(state.n.cpu().long(), sr[3])


# ------------------------------------------------------------------------------------------------ without a GPU

def test_prompt_refuses_on_the_host():
    from bwd_la_fwd_gb300 import la
    lib = la.load_library()

    def call(q=0x100000, k=0x200000, v=0x300000, off=0x400000, o=0x500000, S=0x600000, z=0x700000, a=0x800000, n=0x900000,
             resume=0, T=8, nseq=2, Hq=4, Hkv=2, D=64, dtype=1, strides=None, ws=0xA00000, wsb=1 << 28):
        st = None if strides is None else (ctypes.c_longlong * 8)(*strides)
        return lib.la_prompt(q, k, v, off, o, S, z, a, n, resume, T, nseq, Hq, Hkv, D, dtype, st, ws, wsb, None)

    INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
    assert call(dtype=2) == INVALID and call(Hq=3) == INVALID and call(Hkv=0) == INVALID and call(T=-1) == INVALID
    assert call(D=48) == UNSUPPORTED
    assert call(ws=None) == WORKSPACE and call(ws=0xA00010) == WORKSPACE and call(wsb=16) == WORKSPACE
    assert call(off=None) == INVALID and call(q=None) == INVALID and call(o=0x500008) == INVALID
    assert call(z=None) == INVALID                                            # a state in part
    assert call(S=None, z=None, a=None, n=None, resume=1) == INVALID          # nothing to continue from
    assert call(S=0x600008) == INVALID and call(z=0x600000) == INVALID        # misaligned; the state's parts meet
    assert call(o=0x100000) == INVALID and call(o=0x200000) == INVALID        # the output on an input
    assert call(S=0x500000) == INVALID and call(off=0x500000) == INVALID and call(off=0x600000) == INVALID
    assert call(ws=0x100000) == INVALID and call(ws=0x600000) == INVALID
    assert call(strides=[64, 60] + [64, 128] * 2 + [64, 256]) == INVALID      # rows of whole 16-byte vectors
    assert call(strides=[64, 192] + [64, 128] * 2 + [64, 256]) == INVALID     # rows overlap
    assert call(nseq=0) == 0
    assert lib.la_prompt_workspace_bytes(8, 2, 4, 2, 64, 1) > 0
    for bad in ((8, 2, 4, 3, 64, 1), (8, 2, 4, 2, 48, 1), (-1, 2, 4, 2, 64, 1), (8, 2, 4, 2, 64, 2)):
        assert lib.la_prompt_workspace_bytes(*bad) == 0


def test_prompt_refuses_more_rows_than_an_int_numbers():
    from bwd_la_fwd_gb300 import la
    lib = la.load_library()
    for T, fine in ((2 ** 31 - 1 - 256, True), (2 ** 31 - 256, False), (2 ** 31 - 1, False)):
        assert (lib.la_prompt_workspace_bytes(T, 1, 1, 1, 32, 1) > 0) == fine
    assert lib.la_prompt(0x100000, 0x200000, 0x300000, 0x400000, 0x500000, None, None, None, None, 0, 2 ** 31 - 100, 1, 1, 1,
                         32, 1, None, 0xA00000, 1 << 50, None) == 1


def test_grouped_decode_refuses_on_the_host():
    from bwd_la_fwd_gb300 import la
    lib = la.load_library()

    def call(q=0x100000, k=0x200000, v=0x300000, o=0x400000, g=None, S=0x600000, z=0x700000, a=0x800000, n=0x900000, B=2,
             Hq=4, Hkv=2, D=64, dtype=1, strides=None):
        st = None if strides is None else (ctypes.c_longlong * 8)(*strides)
        return lib.la_decode_step_grouped(q, k, v, o, g, S, z, a, n, B, Hq, Hkv, D, dtype, st, None)

    assert call(dtype=2) == 1 and call(Hq=5) == 1 and call(Hkv=0) == 1 and call(B=-1) == 1
    assert call(D=48) == 2 and call(Hq=130, Hkv=2) == 2
    assert call(q=None) == 1 and call(o=0x400004) == 1 and call(S=None) == 1 and call(g=0x400002) == 1
    assert call(o=0x100000) == 1 and call(S=0x100000) == 1 and call(z=0x600000) == 1 and call(g=0x400000) == 1
    assert call(strides=[256, 32] + [128, 64] * 2 + [256, 64]) == 1
    assert call(B=0) == 0


def test_binding_refuses():
    from bwd_la_fwd_gb300 import la
    q, k = torch.empty(8, 4, 64, dtype=torch.bfloat16), torch.empty(8, 2, 64, dtype=torch.bfloat16)
    off = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        la.la_prompt(q, k, k, off)
    with pytest.raises(ValueError, match="multiple"):
        la.la_prompt(q, torch.empty(8, 3, 64, dtype=torch.bfloat16), torch.empty(8, 3, 64, dtype=torch.bfloat16), off)
    with pytest.raises(ValueError, match="seq_offsets"):
        la.la_prompt(q, k, k, off.long())
    with pytest.raises(ValueError, match="resume"):
        la.la_prompt(q, k, k, off, resume=True)
    with pytest.raises(ValueError, match="state"):
        la.la_prompt(q, k, k, off, la.DecodeState(2, 4, 64, torch.bfloat16, device="cpu"))
    with pytest.raises(ValueError):
        la.DecodeState(2, 2, 64, torch.bfloat16, tensors=(torch.zeros(2, 2, 64, 64),) * 4)
    st = la.DecodeState(8, 2, 64, torch.bfloat16, device="cpu")
    with pytest.raises(ValueError, match="CUDA"):
        la.la_decode_step_grouped(st, q, k, k)
    with pytest.raises(ValueError):
        la.la_decode_step_grouped(st, torch.empty(8, 5, 64, dtype=torch.bfloat16), k, k)
    with pytest.raises(ValueError, match="dtype"):
        la.la_decode_step_grouped(st, q.float(), k, k)


# --------------------------------------------------------------------------------------------------- on the GPU

LENS = [[1], [0], [5, 0, 1, 31, 32, 33], [127, 128, 129, 1], [300, 64, 257], [700]]


@pytest.mark.gpu
@pytest.mark.parametrize("lens", LENS, ids=str)
@pytest.mark.parametrize("kind,D,Hq,Hkv", [("bf16", 128, 4, 2), ("bf16", 64, 3, 3), ("bf16", 32, 8, 1), ("bf16", 16, 2, 1),
                                           ("bf16", 256, 2, 1), ("f32", 16, 2, 2), ("f32", 64, 6, 2), ("f32", 128, 2, 1),
                                           ("f32", 256, 2, 1)])
def test_prompt_matches_explicit_weights(kind, D, Hq, Hkv, lens):
    from bwd_la_fwd_gb300 import la
    off = _offsets(lens, start=3)
    T = off[-1] + 5
    q, k, v = _tokens(T, Hq, Hkv, D, kind, seed=D + len(lens))
    state = _state(len(lens), Hkv, D, kind)
    for t in (state.S, state.z, state.a):
        t.fill_(math.nan)  # an unresumed call only writes it
    state.n.fill_(77)
    O = torch.full((T, Hq, D), 9.0, dtype=R.TYPES[kind], device="cuda")
    ws = la.new_prompt_workspace(T, len(lens), Hq, Hkv, D, la.LA_BF16 if kind == "bf16" else la.LA_F32)
    la.la_prompt(q, k, v, torch.tensor(off, dtype=torch.int32, device="cuda"), state, O=O, workspace=ws)
    assert la.la_get_status(ws) == 0
    ref, tol = R.prompt(q, k, v, off, R.empty_state(len(lens), Hkv, D), kind, (kind, D) in TENSOR_CORE)
    _check(O, state, ref, tol, off)
    assert bool((O[:3] == 9.0).all()) and bool((O[off[-1]:] == 9.0).all())  # rows of no sequence stay as they were


@pytest.mark.gpu
@pytest.mark.parametrize("ctas", [1, 2, 3, 7, 40])
@pytest.mark.parametrize("D,Hq,Hkv,resume", [(128, 6, 2, False), (128, 2, 2, True), (64, 4, 1, True), (32, 5, 5, False)])
def test_slices_of_any_number_of_ctas(monkeypatch, D, Hq, Hkv, resume, ctas):
    """The tensor-core form's work split: heads that straddle CTAs, CTAs with many heads, CTAs with nothing."""
    from bwd_la_fwd_gb300 import la
    monkeypatch.setenv("LA_TC_MAX_CTAS", str(ctas))
    lens = [300, 0, 1, 900, 128, 256, 77]
    off = _offsets(lens)
    q, k, v = _tokens(off[-1], Hq, Hkv, D, "bf16", seed=ctas)
    state = _state(len(lens), Hkv, D, "bf16")
    start = R.empty_state(len(lens), Hkv, D)
    if resume:  # a state that some other tokens left
        pq, pk, pv = _tokens(50 * len(lens), Hq, Hkv, D, "bf16", seed=99)
        po = _offsets([50] * len(lens))
        la.la_prompt(pq, pk, pv, torch.tensor(po, dtype=torch.int32, device="cuda"), state)
        start = tuple(t.double().cpu() for t in (state.S, state.z, state.a)) + (state.n.cpu().long(),)
    ws = la.new_prompt_workspace(off[-1], len(lens), Hq, Hkv, D, la.LA_BF16)
    O = la.la_prompt(q, k, v, torch.tensor(off, dtype=torch.int32, device="cuda"), state, resume=resume, workspace=ws)
    assert la.la_get_status(ws) == 0
    ref, tol = R.prompt(q, k, v, off, start, "bf16", True)
    _check(O, state, ref, tol, off)


@pytest.mark.gpu
@pytest.mark.parametrize("lens,D,Hq,Hkv,resume", [([6000], 64, 3, 3, True), ([6000], 128, 2, 1, False),
                                                  ([3000] + [130] * 20, 64, 6, 3, True), ([257] * 60, 32, 2, 2, False),
                                                  ([1500, 1, 0, 1500, 700], 128, 4, 2, True)], ids=str)
def test_heads_that_straddle_many_ctas(lens, D, Hq, Hkv, resume):
    """The tensor-core form's carries: few long chains of CTAs, many short ones, both together; a state to start from."""
    from bwd_la_fwd_gb300 import la
    off = _offsets(lens)
    q, k, v = _tokens(off[-1], Hq, Hkv, D, "bf16", seed=len(lens))
    state = _state(len(lens), Hkv, D, "bf16")
    start = R.empty_state(len(lens), Hkv, D)
    if resume:
        pq, pk, pv = _tokens(40 * len(lens), Hq, Hkv, D, "bf16", seed=98)
        la.la_prompt(pq, pk, pv, torch.tensor(_offsets([40] * len(lens)), dtype=torch.int32, device="cuda"), state)
        start = tuple(t.double().cpu() for t in (state.S, state.z, state.a)) + (state.n.cpu().long(),)
    ws = la.new_prompt_workspace(off[-1], len(lens), Hq, Hkv, D, la.LA_BF16)
    ws[256:].fill_(255)  # what earlier calls left is not read
    O = la.la_prompt(q, k, v, torch.tensor(off, dtype=torch.int32, device="cuda"), state, resume=resume, workspace=ws)
    assert la.la_get_status(ws) == 0
    ref, tol = R.prompt(q, k, v, off, start, "bf16", True)
    _check(O, state, ref, tol, off)


@pytest.mark.gpu
@pytest.mark.parametrize("kind,D", [("bf16", 128), ("bf16", 256), ("f32", 64)])
def test_prompts_without_rows(kind, D):
    """T = 0: sequences start empty and stay so, or keep the state that they continue from."""
    from bwd_la_fwd_gb300 import la
    q, k = torch.empty(0, 4, D, dtype=R.TYPES[kind], device="cuda"), torch.empty(0, 2, D, dtype=R.TYPES[kind], device="cuda")
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    ws = la.new_prompt_workspace(0, 2, 4, 2, D, la.LA_BF16 if kind == "bf16" else la.LA_F32)
    state = _state(2, 2, D, kind)
    parts = (state.S, state.z, state.a, state.n)
    for t in parts:
        t.fill_(5)
    assert la.la_prompt(q, k, k, off, state, resume=True, workspace=ws).shape == (0, 4, D)
    assert all(bool((t == 5).all()) for t in parts)
    la.la_prompt(q, k, k, off, state, workspace=ws)
    assert all(not bool(t.any()) for t in parts) and la.la_get_status(ws) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("D,unit", [(128, 0), (128, 9), (64, 6)])
def test_a_wait_that_runs_out_is_reported_and_leaves_the_next_call_exact(monkeypatch, D, unit):
    """A tile of Q that the walk's first CTA does not ask for (no copy and no arrival): its wait ends after 20 ms, every
    role stops, and the next call on the same workspace has the bits of one that never saw it."""
    from bwd_la_fwd_gb300 import la
    T, Hq, Hkv = 2048, 4, 2
    q, k, v = _tokens(T, Hq, Hkv, D, "bf16", seed=unit)
    off = torch.tensor([0, 900, T], dtype=torch.int32, device="cuda")
    monkeypatch.setenv("LA_TC_MAX_CTAS", "4")
    ws = la.new_prompt_workspace(T, 2, Hq, Hkv, D, la.LA_BF16)
    state = _state(2, Hkv, D, "bf16")
    want = la.la_prompt(q, k, v, off, state, workspace=ws)
    parts = [t.clone() for t in (state.S, state.z, state.a, state.n)]
    assert la.la_get_status(ws) == 0
    monkeypatch.setenv("LA_TEST_WAIT_NS", "20000000")
    monkeypatch.setenv("LA_TEST_DROP_LOAD", str(unit))
    la.la_prompt(q, k, v, off, state, workspace=ws)
    assert la.la_get_status(ws) == 5  # LA_ERR_TIMEOUT
    monkeypatch.delenv("LA_TEST_WAIT_NS")
    monkeypatch.delenv("LA_TEST_DROP_LOAD")
    assert torch.equal(la.la_prompt(q, k, v, off, state, workspace=ws), want) and la.la_get_status(ws) == 0
    assert all(torch.equal(a, b) for a, b in zip(parts, (state.S, state.z, state.a, state.n)))


@pytest.mark.gpu
def test_prompts_on_two_streams_at_once():
    """Calls that overlap, each with a workspace of its own, give the bits of calls one after another."""
    from bwd_la_fwd_gb300 import la
    D, Hq, Hkv, T = 128, 4, 2, 2000
    off = torch.tensor([0, 900, T], dtype=torch.int32, device="cuda")
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    toks = [_tokens(T, Hq, Hkv, D, "bf16", seed=s) for s in (1, 2)]
    ws = [la.new_prompt_workspace(T, 2, Hq, Hkv, D, la.LA_BF16) for _ in streams]
    alone = [la.la_prompt(*t, off, workspace=w) for t, w in zip(toks, ws)]
    outs = [torch.zeros_like(o) for o in alone]
    torch.cuda.synchronize()
    for _ in range(8):
        for s, t, w, o in zip(streams, toks, ws, outs):
            la.la_prompt(*t, off, O=o, workspace=w, stream=s)
    torch.cuda.synchronize()
    assert all(la.la_get_status(w) == 0 for w in ws)
    assert all(torch.equal(a, b) for a, b in zip(alone, outs))


@pytest.mark.gpu
@pytest.mark.parametrize("kind,D,Hq,Hkv", [("bf16", 128, 4, 1), ("bf16", 64, 4, 2), ("bf16", 256, 1, 1), ("f32", 64, 4, 2),
                                           ("f32", 128, 2, 2)])
def test_prompts_in_parts(kind, D, Hq, Hkv):
    """Each sequence in two parts, the second resumed: outputs and states against explicit weights over the whole."""
    from bwd_la_fwd_gb300 import la
    first, second = [200, 3, 0, 128], [150, 129, 40, 0]
    whole = [a + b for a, b in zip(first, second)]
    off = _offsets(whole)
    q, k, v = _tokens(off[-1], Hq, Hkv, D, kind, seed=17)
    ref, tol = R.prompt(q, k, v, off, R.empty_state(4, Hkv, D), kind, (kind, D) in TENSOR_CORE)
    state = _state(4, Hkv, D, kind)
    O = torch.empty(off[-1], Hq, D, dtype=R.TYPES[kind], device="cuda")
    for part, resume in ((0, False), (1, True)):
        rows = torch.cat([torch.arange(off[i] + (first[i] if part else 0), off[i] + (whole[i] if part else first[i]))
                          for i in range(4)]).cuda()
        po = torch.tensor(_offsets(second if part else first), dtype=torch.int32, device="cuda")
        O[rows] = la.la_prompt(q[rows], k[rows], v[rows], po, state, resume=resume)
    _check(O, state, ref, tol, off)


@pytest.mark.gpu
@pytest.mark.parametrize("kind,D", [("bf16", 128), ("bf16", 16), ("f32", 64)])
def test_neighbours_and_outside_rows_have_no_part(kind, D):
    """NaN and infinities in another sequence and in rows of no sequence: the same bits as without them."""
    from bwd_la_fwd_gb300 import la
    lens, Hq, Hkv = [70, 130, 20, 200], 4, 2
    off = _offsets(lens, start=2)
    T = off[-1] + 100
    q, k, v = _tokens(T, Hq, Hkv, D, kind, seed=23)
    o = torch.tensor(off, dtype=torch.int32, device="cuda")
    s1, s2 = _state(4, Hkv, D, kind), _state(4, Hkv, D, kind)
    clean = la.la_prompt(q, k, v, o, s1)
    for t, x in ((q, math.nan), (k, math.inf), (v, math.nan)):
        t[:2] = x
        t[off[1]:off[2]] = x
        t[off[4]:] = x
    dirty = la.la_prompt(q, k, v, o, s2)
    for i in (0, 2, 3):
        assert torch.equal(clean[off[i]:off[i + 1]], dirty[off[i]:off[i + 1]])
        assert torch.equal(s1.S[i], s2.S[i]) and torch.equal(s1.z[i], s2.z[i]) and torch.equal(s1.a[i], s2.a[i])
    assert not torch.isfinite(dirty[off[1]:off[2]]).any()
    assert not dirty[:2].any() and not dirty[off[4]:].any()  # a new O is zero outside


@pytest.mark.gpu
@pytest.mark.parametrize("kind,D", [("bf16", 128), ("f32", 32)])
@pytest.mark.parametrize("bad", [[0, 50, 40, 60], [-1, 10, 20, 30], [0, 10, 20, 61]])
def test_offsets_out_of_order_are_refused(kind, D, bad):
    from bwd_la_fwd_gb300 import la
    q, k, v = _tokens(60, 2, 1, D, kind, seed=1)
    state = _state(3, 1, D, kind)
    state.S.fill_(3.0)
    O = torch.full((60, 2, D), 5.0, dtype=R.TYPES[kind], device="cuda")
    ws = la.new_prompt_workspace(60, 3, 2, 1, D, la.LA_BF16 if kind == "bf16" else la.LA_F32)
    la.la_prompt(q, k, v, torch.tensor(bad, dtype=torch.int32, device="cuda"), state, O=O, workspace=ws)
    assert la.la_get_status(ws) == 6 and la.la_get_status(ws) == 0
    assert bool((O == 5.0).all()) and bool((state.S == 3.0).all()) and not state.n.any()
    la.la_prompt(q, k, v, torch.tensor([0, 10, 20, 60], dtype=torch.int32, device="cuda"), state, O=O, workspace=ws)
    assert la.la_get_status(ws) == 0 and not bool((O == 5.0).all())


@pytest.mark.gpu
@pytest.mark.parametrize("kind,D", [("bf16", 128), ("f32", 64)])
def test_prompt_without_a_state_and_contiguous(kind, D):
    """No state; contiguous operands give the bits of the strided views."""
    from bwd_la_fwd_gb300 import la
    off = torch.tensor([0, 140, 300], dtype=torch.int32, device="cuda")
    q, k, v = _tokens(300, 4, 2, D, kind, seed=6)
    state = _state(2, 2, D, kind)
    want = la.la_prompt(q, k, v, off, state)
    assert torch.equal(la.la_prompt(q.contiguous(), k.contiguous(), v.contiguous(), off), want)
    Oh = torch.empty(4, 300, D, dtype=R.TYPES[kind], device="cuda")  # [H,T,D] through its [T,H,D] view
    la.la_prompt(q, k, v, off, O=Oh.transpose(0, 1))
    assert torch.equal(Oh.transpose(0, 1), want)


@pytest.mark.gpu
@pytest.mark.parametrize("kind,D", [("bf16", 128), ("f32", 64)])
def test_prompt_in_a_graph_follows_its_offsets(kind, D):
    """Lengths live on the device: a captured call replayed with other offsets and tokens; the same bits every time."""
    from bwd_la_fwd_gb300 import la
    q, k, v = _tokens(600, 4, 2, D, kind, seed=8)
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    state, O = _state(3, 2, D, kind), torch.zeros(600, 4, D, dtype=R.TYPES[kind], device="cuda")
    ws = la.new_prompt_workspace(600, 3, 4, 2, D, la.LA_BF16 if kind == "bf16" else la.LA_F32)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        la.la_prompt(q, k, v, off, state, O=O, workspace=ws, stream=side)
    for offsets in ([0, 100, 350, 600], [10, 10, 590, 600], [0, 1, 2, 3]):
        off.copy_(torch.tensor(offsets, dtype=torch.int32))
        O.zero_()
        graph.replay()
        fresh = _state(3, 2, D, kind)
        want = la.la_prompt(q, k, v, off.clone(), fresh)
        assert torch.equal(O, want) and torch.equal(state.S, fresh.S) and torch.equal(state.n, fresh.n)
    assert la.la_get_status(ws) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("B,Hq,Hkv,D", [(1, 4, 1, 128), (2, 3, 3, 64), (3, 16, 2, 16), (2, 14, 2, 32), (2, 4, 2, 256),
                                        (1, 64, 1, 64), (90, 8, 4, 128)])
def test_grouped_decode_matches_explicit_weights(kind, B, Hq, Hkv, D):
    """A few tokens after a prompt, one by one: outputs, normalisers and states."""
    from bwd_la_fwd_gb300 import la
    steps = 3
    prompt_len = 2 if B > 8 else 20
    rows = prompt_len + steps
    q, k, v = _tokens(B * rows, Hq, Hkv, D, kind, seed=B + D)
    off = _offsets([rows] * B)
    ref, tol = R.prompt(q, k, v, off, R.empty_state(B, Hkv, D), kind, False)
    state = _state(B, Hkv, D, kind)
    q, k, v = (t.view(B, rows, *t.shape[1:]) if t.is_contiguous() else t.unflatten(0, (B, rows)) for t in (q, k, v))
    head = [t[:, :prompt_len].flatten(0, 1) for t in (q, k, v)]
    la.la_prompt(*head, torch.tensor(_offsets([prompt_len] * B), dtype=torch.int32, device="cuda"), state)
    Or, ot = (t.unflatten(0, (B, rows)) for t in (ref[0], tol[0]))
    for t in range(prompt_len, rows):
        g = torch.empty(B, Hq, device="cuda")
        o = la.la_decode_step_grouped(state, q[:, t], k[:, t], v[:, t], normaliser=g)
        R.assert_within("o", o, Or[:, t], ot[:, t])
        qd, kd = q[:, t].double().cpu(), k[:, :t + 1].double().cpu()
        W = 1 + torch.einsum("bgrd,btgd->bgrt", qd.unflatten(1, (Hkv, -1)), kd)
        Wm = 1 + torch.einsum("bgrd,btgd->bgrt", qd.abs().unflatten(1, (Hkv, -1)), kd.abs())
        # the prompt's z is rounded to the state's type only; the sums' roundings as in O's denominator
        R.assert_within("g", g, W.sum(-1).flatten(1), (2 * t + 2 * D + 64) * R.U * Wm.sum(-1).flatten(1))
    _check_state = list(zip("Sza", (state.S, state.z, state.a), ref[1], tol[1:]))
    for what, got, want, t in _check_state:
        R.assert_within(what, got, want, t)
    assert torch.equal(state.n.cpu().long(), ref[1][3])


@pytest.mark.gpu
@pytest.mark.parametrize("kind,D", [("bf16", 128), ("f32", 64), ("bf16", 256)])
def test_grouped_decode_of_single_heads_is_the_decode_step(kind, D):
    from bwd_la_fwd_gb300 import la
    B, H = 2, 3
    q, k, v = (t.contiguous() for t in _tokens(B, H, H, D, kind, seed=2))
    s1, s2 = _state(B, H, D, kind), _state(B, H, D, kind)
    for _ in range(3):
        o1, g1 = la.la_decode_step(s1, q, k, v)
        g2 = torch.empty(B, H, device="cuda")
        o2 = la.la_decode_step_grouped(s2, q, k, v, normaliser=g2)
        assert torch.equal(s1.S, s2.S) and torch.equal(s1.z, s2.z) and torch.equal(s1.a, s2.a) and torch.equal(s1.n, s2.n)
        # sums of D products taken in another order: within D half steps of their magnitudes, then the output's rounding
        lim = 2 * D * R.U * (s1.a.abs().double() + torch.einsum("bhd,bhde->bhe", q.double().abs(), s1.S.double().abs()))
        lim = (lim / g1.double()[..., None]).cpu() + 2 * R.half_step(kind) * o1.double().abs().cpu()
        R.assert_within("o", o2, o1, lim)


@pytest.mark.gpu
def test_grouped_decode_in_a_graph():
    from bwd_la_fwd_gb300 import la
    q, k, v = _tokens(4, 8, 2, 128, "bf16", seed=3)
    eager, graphed = _state(4, 2, 128, "bf16"), _state(4, 2, 128, "bf16")
    o = torch.empty(4, 8, 128, dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        la.la_decode_step_grouped(graphed, q, k, v, o=o, stream=side)
    for _ in range(3):
        graph.replay()
        want = la.la_decode_step_grouped(eager, q, k, v)
        assert torch.equal(o, want) and torch.equal(eager.S, graphed.S)
