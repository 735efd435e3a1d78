"""The selective scan where its launches take other shapes than small calls do: two channels to a thread, parts of time for every
number of states, CTAs that walk several sequences of the gradient, several sequences to a block of the step."""
import pytest
import torch

import state_space_testutil as R
from test_selective_scan import GRADS, _case, _check_forward, _cuda, _forward, _options, _rows

pytestmark = pytest.mark.gpu


def _offsets(lens, pad):
    off = [pad]
    for n in lens:
        off.append(off[-1] + n)
    return off


def _check_gradients(c, dy, off, st, dl, kind, opt, extra=0):
    from bwd_la_fwd_gb300 import la
    T, C = c["x"].shape
    S, n, sp = c["A"].shape[1], len(off) - 1, opt.get("softplus", True)
    marks = la.new_selective_scan_marks(T, n, C, S)
    _forward(c, off, st, kind, 0, opt, marks=marks)
    ref, tol = R.scan_backward(*_rows(c), dy, opt.get("D"), opt.get("z"), opt.get("dt_bias"), sp, off, st, dl, extra)
    got = la.la_selective_scan_backward(*_rows(_cuda(c)), dy.cuda(), marks, **{k: v.cuda() if torch.is_tensor(v) else v for k, v in opt.items()},
                                        seq_offsets=torch.tensor(off, dtype=torch.int32, device="cuda"), dstate_out=dl.cuda())
    for name in GRADS + ("dstate_in",):
        if name == "dz" and opt.get("z") is None:
            assert got.dz is None
            continue
        t, typed = getattr(got, name), name in ("dX", "ddt", "dz", "dB", "dC")
        R.assert_within(name, t, ref[name], R.rounded(ref[name], tol[name], kind) if typed else tol[name])


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("S", [8, 16, 32])
def test_two_channels_to_a_thread(S, kind):
    """40 sequences of 5 blocks of channels each: more than the SMs."""
    lens = [(7 * i) % 41 if i % 6 else i % 4 for i in range(40)]
    off = _offsets(lens, 3)
    for C, G, resumed, gated, plain in ((320, 1, True, True, False), (5 * 64 - 16, 2, False, False, True)):
        c, _, st, _ = _case(off[-1] + 3, C, G, S, 40, kind, S + C)
        if plain:
            c["dt"] = c["dt"].abs() * 0.1
        _check_forward(c, off, st if resumed else None, kind, _options(c, gated, plain))


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("S", [8, 16])
def test_two_channels_to_a_thread_in_parts(S, kind):
    """One sequence in 17 parts of 10 blocks of channels."""
    off = [1, 2101]
    c, _, st, _ = _case(2103, 640, 1, S, 1, kind, S)
    _check_forward(c, off, st, kind, _options(c), extra=0.4 * 2100)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("S", [8, 16, 32])
@pytest.mark.parametrize("lens", [[1100], [600, 0, 1, 700]])
def test_gradients_in_parts(lens, S, kind):
    off = _offsets(lens, 2)
    c, dy, st, dl = _case(off[-1] + 2, 16, 1, S, len(lens), kind, S)
    _check_forward(c, off, st, kind, _options(c), extra=0.4 * 1100)
    _check_gradients(c, dy, off, st, dl, kind, _options(c), extra=0.4 * 1100)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("S", [8, 16, 32])
def test_gradients_of_more_sequences_than_walkers(S, kind):
    """90 sequences of 8 or 16 blocks of channels, for which 76 or 38 CTAs walk: what is summed over rows goes on from one
    sequence to the next, what belongs to a sequence does not."""
    lens = [(5 * i) % 8 if i % 7 else 0 for i in range(90)]
    off = _offsets(lens, 1)
    c, dy, st, dl = _case(off[-1] + 1, 1024, 1, S, 90, kind, S)
    _check_gradients(c, dy, off, st, dl, kind, _options(c))


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("S", [8, 16, 32])
def test_gradients_without_options(S, kind):
    off = _offsets([40, 0, 1, 23], 2)
    c, dy, st, dl = _case(off[-1] + 2, 144, 2, S, 4, kind, S)
    c["dt"] = c["dt"].abs() * 0.1
    _check_gradients(c, dy, off, st, dl, kind, _options(c, plain=True))


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("plain", [False, True])
@pytest.mark.parametrize("S,n", [(8, 1219), (16, 611), (32, 307)])
def test_a_token_of_many_sequences(S, n, plain, kind):
    """Four sequences to a block, three to the last."""
    from bwd_la_fwd_gb300 import la
    C = 1024
    c, _, st, _ = _case(n, C, 2, S, n, kind, S)
    if plain:
        c["dt"] = c["dt"].abs() * 0.1
    opt, off = _options(c, plain=plain), list(range(n + 1))
    (y, h), (ey, eh) = R.scan(*_rows(c), opt.get("D"), opt.get("z"), opt.get("dt_bias"), opt.get("softplus", True), off, st)
    state = st.cuda()
    got = la.la_selective_scan_step(state, *_rows(_cuda(c)), **{k: v.cuda() if torch.is_tensor(v) else v for k, v in opt.items()})
    R.assert_within("Y", got, y, R.rounded(y, ey, kind))
    R.assert_within("state", state, h, eh)
