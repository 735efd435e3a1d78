"""The operators together, as a recurrent decoder layer uses them: training (gated recurrence, rotary positions, the
causal head, and the gradients back through all three) and serving (packed prompts, then tokens one by one)."""
import math

import pytest
import torch

import ops_testutil as R

pytestmark = pytest.mark.gpu


def _explicit(q, k, v):
    """Causal head in 64 bits, [B,H,N,D], differentiable."""
    W = torch.tril(1 + q @ k.transpose(-1, -2))
    return W @ v / W.sum(-1, keepdim=True)


def _turn(x, pos, freq):
    th = pos[:, None] * freq
    half = x.shape[-1] // 2
    x1, x2 = x[..., :half], x[..., half:]
    return torch.cat([x1 * th.cos() - x2 * th.sin(), x1 * th.sin() + x2 * th.cos()], -1)


def _scan(x, w, h0):
    a = torch.sigmoid(w)
    h, out = h0, []
    for t in range(x.shape[1]):
        h = a[:, t] * h + (1 - a[:, t]) * x[:, t]
        out.append(h)
    return torch.stack(out, 1)


def test_training_layer_in_fp32():
    """fp32 throughout: the whole chain's outputs and gradients within 1e-4 of 64 bits, norm against norm (three
    operators of some 1e-6 each, the head's own bar being 1e-5 an element)."""
    from bwd_la_fwd_gb300 import la
    B, N, H, D = 2, 150, 2, 32
    gen = torch.Generator().manual_seed(0)
    x, w = (torch.randn(B, N, 3 * H * D, generator=gen) for _ in range(2))
    scale = torch.ones(3 * H * D)
    scale[:2 * H * D] /= math.sqrt(D)
    x = x * scale
    dO = torch.randn(B, H, N, D, generator=gen)
    freqs = la.la_rotary_frequencies(D)
    xc, wc = x.cuda(), w.cuda()
    hs, _ = la.la_gated_scan(xc, wc, "sigmoid")  # [B,N,3HD]: the mixed channels are Q, K and V
    q, k, v = hs.unflatten(-1, (3, H, D)).unbind(2)
    q, k, v = (t.transpose(1, 2) for t in (q, k, v))
    qr, kr = la.la_rotary(q, k, freqs)
    ws = la.new_workspace(B, H, N, D, True, la.LA_F32, True)
    O, _ = la.la_forward(qr, kr, v, True, O=torch.empty_like(qr), workspace=ws)
    dqr, dkr, dv = la.la_backward(qr, kr, v.contiguous(), O, dO.cuda(), True, workspace=ws)
    dh = torch.empty_like(hs)
    dq, dk, dvv = (t.transpose(1, 2) for t in dh.unflatten(-1, (3, H, D)).unbind(2))
    la.la_rotary_backward(dqr, dkr, freqs, dQ_out=dq, dK_out=dk)
    dvv.copy_(dv)
    dx, dw, _ = la.la_gated_scan_backward(xc, wc, hs, dh, "sigmoid")
    assert la.la_get_status(ws) == 0

    xd, wd = x.double().requires_grad_(), w.double().requires_grad_()
    q, k, v = (t.transpose(1, 2) for t in _scan(xd, wd, torch.zeros(B, 3 * H * D, dtype=torch.float64)).unflatten(
        -1, (3, H, D)).unbind(2))
    pos = torch.arange(N, dtype=torch.float64)
    ref = _explicit(_turn(q, pos, R.frequencies(D)), _turn(k, pos, R.frequencies(D)), v)
    ref.backward(dO.double())
    for name, got, want in (("O", O, ref.detach()), ("dX", dx, xd.grad), ("dW", dw, wd.grad)):
        e = float((got.double().cpu() - want).norm() / want.norm())
        assert e <= 1e-4, (name, e)


@pytest.mark.parametrize("kind,bar", [("bf16", 2e-2), ("f32", 1e-5)])
def test_serving_layer(kind, bar):
    """Ragged prompts through rotary, the packed head and its states, then tokens of all sequences together, against the
    explicit head over each whole sequence (the head's bar of largest error against largest value)."""
    from bwd_la_fwd_gb300 import la
    lens, steps, Hq, Hkv, D = [5, 140, 33], 4, 4, 2, 64
    gen = torch.Generator().manual_seed(1)
    dt = R.TYPES[kind]
    seqs = []
    for n in lens:
        x = torch.randn(n + steps, Hq + 2 * Hkv, D, generator=gen)
        x[:, :Hq + Hkv] /= math.sqrt(D)
        seqs.append(x.to(dt))
    freqs = la.la_rotary_frequencies(D)
    packed = torch.cat([x[:n] for x, n in zip(seqs, lens)]).cuda()
    positions = torch.cat([torch.arange(n, dtype=torch.int32) for n in lens]).cuda()
    offsets = torch.tensor([0, 5, 145, 178], dtype=torch.int32, device="cuda")
    state = la.DecodeState(3, Hkv, D, dt)

    def turned(x, pos):  # [T,H,D] rows as one batch entry's [1,H,T,D]
        q, k = x[:, :Hq].transpose(0, 1)[None], x[:, Hq:Hq + Hkv].transpose(0, 1)[None]
        q, k = la.la_rotary(q, k, freqs, positions=pos)
        return q[0].transpose(0, 1), k[0].transpose(0, 1), x[:, Hq + Hkv:]

    O = la.la_prompt(*turned(packed, positions), offsets, state)
    outs = [[O[offsets[i]:offsets[i + 1]]] for i in range(3)]
    for s in range(steps):
        token = torch.stack([x[n + s] for x, n in zip(seqs, lens)]).cuda()
        pos = torch.tensor([n + s for n in lens], dtype=torch.int32, device="cuda")
        o = la.la_decode_step_grouped(state, *turned(token, pos))
        for i in range(3):
            outs[i].append(o[i][None])
    assert state.n.tolist() == [[n + steps] * Hkv for n in lens]
    for i, (x, n) in enumerate(zip(seqs, lens)):
        pos = torch.arange(n + steps, dtype=torch.float64)
        x = x.double().transpose(0, 1)
        q, k = _turn(x[:Hq], pos, R.frequencies(D)), _turn(x[Hq:Hq + Hkv], pos, R.frequencies(D))
        k, v = (t.repeat_interleave(Hq // Hkv, 0) for t in (k, x[Hq + Hkv:]))
        ref = _explicit(q[None], k[None], v[None])[0].transpose(0, 1)
        got = torch.cat(outs[i]).double().cpu()
        assert float((got - ref).abs().max() / ref.abs().max()) <= bar
