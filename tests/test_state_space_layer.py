"""The norm, the short convolution and the selective scan together, as a decoder layer uses them: training (forward and the
gradients back through all three) and serving (packed prompts, then tokens one by one)."""
import math

import pytest
import torch

import state_space_testutil as R

pytestmark = pytest.mark.gpu


def _weights(H, C, S, K, gen):
    want = torch.exp(torch.rand(C, generator=gen) * math.log(100.0) + math.log(0.001))
    return dict(norm=1 + 0.1 * torch.randn(H, generator=gen), w_in=torch.randn(H, 2 * C, generator=gen) / math.sqrt(H),
                taps=torch.randn(C, K, generator=gen) / math.sqrt(K), tap_bias=0.1 * torch.randn(C, generator=gen),
                w_bc=torch.randn(C, 2 * S, generator=gen) / math.sqrt(C), w_dt=0.5 * torch.randn(C, C, generator=gen) / math.sqrt(C),
                A=-torch.arange(1, S + 1).float().repeat(C, 1), D=torch.ones(C), bias=want + torch.log(-torch.expm1(-want)),
                w_out=torch.randn(C, H, generator=gen) / math.sqrt(C))


def _explicit(x, res, w, S):
    """The layer in 64 bits over one sequence [N,H], differentiable: (out, residual)."""
    C = w["D"].numel()
    r = x + res
    y = r * w["norm"] / (r.square().mean(-1, keepdim=True) + 1e-6).sqrt()
    u, z = (y @ w["w_in"]).split(C, -1)
    K = w["taps"].shape[1]
    xs = torch.cat([torch.zeros(K - 1, C, dtype=u.dtype), u])
    u = R.silu(w["tap_bias"] + sum(xs[j:j + u.shape[0]] * w["taps"][:, j] for j in range(K)))
    B, Cm = (u @ w["w_bc"]).split(S, -1)
    d = torch.nn.functional.softplus(u @ w["w_dt"] + w["bias"])
    h, out = torch.zeros(C, S, dtype=u.dtype), []
    for t in range(u.shape[0]):
        h = torch.exp(d[t][:, None] * w["A"]) * h + (d[t] * u[t])[:, None] * B[t]
        out.append(((h * Cm[t]).sum(-1) + w["D"] * u[t]) * R.silu(z[t]))
    return torch.stack(out) @ w["w_out"], r


def test_training_layer_in_fp32():
    """Outputs and all gradients within 1e-4 of 64 bits, norm against norm (operators and products of some 1e-6 each)."""
    from bwd_la_fwd_gb300 import la
    Bt, N, H, C, S, K = 2, 90, 48, 64, 16, 4
    gen = torch.Generator().manual_seed(0)
    x, res, dout, dres = (torch.randn(Bt, N, H, generator=gen) for _ in range(4))
    w = _weights(H, C, S, K, gen)
    g = {k: v.cuda() for k, v in w.items()}
    y, r = la.la_rms_norm(x.cuda(), g["norm"], residual=res.cuda())
    xz = y @ g["w_in"]
    u0, z = xz[..., :C], xz[..., C:]
    u = la.la_short_conv(u0, g["taps"], bias=g["tap_bias"], activation="silu")
    bc = (u @ g["w_bc"]).unflatten(-1, (2, 1, S))
    dt = u @ g["w_dt"]
    marks = la.new_selective_scan_marks(Bt * N, Bt, C, S)
    args = u, dt, g["A"], bc[:, :, 0], bc[:, :, 1]
    opt = dict(D=g["D"], z=z, dt_bias=g["bias"])
    Y = la.la_selective_scan(*args, marks=marks, **opt)
    out = Y @ g["w_out"]
    # back
    dY = dout.cuda() @ g["w_out"].t()
    s = la.la_selective_scan_backward(*args, dY, marks, **opt)
    dbc = torch.cat([s.dB, s.dC], -1).squeeze(2)
    du = s.dX + s.ddt @ g["w_dt"].t() + dbc @ g["w_bc"].t()
    du0, dtaps, dtb = la.la_short_conv_backward(u0, g["taps"], du, bias=g["tap_bias"], activation="silu")
    dy = torch.cat([du0, s.dz], -1) @ g["w_in"].t()
    dx, dnorm = la.la_rms_norm_backward(r, g["norm"], dy, dR=dres.cuda())
    got = dict(out=out, r=r, x=dx, norm=dnorm, taps=dtaps, tap_bias=dtb, A=s.dA, D=s.dD, bias=s.ddt_bias,
               w_dt=torch.einsum("bnc,bnd->cd", u, s.ddt))

    xd, rd = x.double().requires_grad_(), res.double()
    wd = {k: v.double().requires_grad_() for k, v in w.items()}
    both = [_explicit(xd[b], rd[b], wd, S) for b in range(Bt)]
    o, rr = (torch.stack(t) for t in zip(*both))
    ((o * dout.double()).sum() + (rr * dres.double()).sum()).backward()
    want = dict(out=o.detach(), r=rr.detach(), x=xd.grad, **{k: wd[k].grad for k in ("norm", "taps", "tap_bias", "A", "D", "bias", "w_dt")})
    for name, ref in want.items():
        e = float((got[name].double().cpu() - ref).norm() / ref.norm())
        assert e <= 1e-4, (name, e)


@pytest.mark.parametrize("kind,bar", [("bf16", 4e-2), ("f32", 1e-4)])
def test_serving_layer(kind, bar):
    """Ragged prompts through all three with their states, then tokens of all sequences together, against the explicit layer
    over each whole sequence (largest error against largest value; in bf16 five roundings of intermediate tensors, each of
    2^-9, spread through the products)."""
    from bwd_la_fwd_gb300 import la
    lens, steps, H, C, S, K = [5, 70, 2], 4, 64, 128, 16, 4
    gen = torch.Generator().manual_seed(1)
    dt_ = R.TYPES[kind]
    seqs = [(torch.randn(n + steps, H, generator=gen).to(dt_), torch.randn(n + steps, H, generator=gen).to(dt_)) for n in lens]
    w = {k: v.to(dt_).float() if k.startswith("w_") else v for k, v in _weights(H, C, S, K, gen).items()}
    g = {k: v.cuda().to(dt_) if k.startswith("w_") else v.cuda() for k, v in w.items()}
    off = torch.tensor([0, 5, 75, 77], dtype=torch.int32, device="cuda")
    n = len(lens)
    taps, state = torch.empty(n, K - 1, C, dtype=dt_, device="cuda"), torch.empty(n, C, S, device="cuda")

    def layer(x, res, conv, scan):
        y, _ = la.la_rms_norm(x, g["norm"], residual=res)
        xz = y @ g["w_in"]
        u = conv(xz[:, :C])
        bc = (u @ g["w_bc"]).unflatten(-1, (2, 1, S))
        return scan((u, u @ g["w_dt"], g["A"], bc[:, 0], bc[:, 1]), dict(D=g["D"], z=xz[:, C:], dt_bias=g["bias"])) @ g["w_out"]

    rows = layer(*(torch.cat([s[k][:m] for s, m in zip(seqs, lens)]).cuda() for k in range(2)),
                 lambda u: la.la_short_conv(u, g["taps"], bias=g["tap_bias"], activation="silu", seq_offsets=off, state_out=taps),
                 lambda a, o: la.la_selective_scan(*a, **o, seq_offsets=off, state_out=state))
    outs = [[rows[off[i]:off[i + 1]]] for i in range(n)]
    for t in range(steps):
        token = (torch.stack([s[k][m + t] for s, m in zip(seqs, lens)]).cuda() for k in range(2))
        o = layer(*token, lambda u: la.la_short_conv_step(taps, u, g["taps"], bias=g["tap_bias"], activation="silu"),
                  lambda a, o: la.la_selective_scan_step(state, *a, **o))
        for i in range(n):
            outs[i].append(o[i][None])
    for i, (x, res) in enumerate(seqs):
        ref, _ = _explicit(x.double(), res.double(), {k: v.double() for k, v in w.items()}, S)
        got = torch.cat(outs[i]).double().cpu()
        assert float((got - ref).abs().max() / ref.abs().max()) <= bar
