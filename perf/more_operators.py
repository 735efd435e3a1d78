"""A state space layer's operators beside the linear-attention head, as cases that can be timed and compared.

norm   root-mean-square norm with the residual's addition: in the tokens' type, in 8 bits with scales, its gradients
conv   the short causal convolution per channel: packed prompts with their states, gradients, one token
scan   the selective state space scan: training forward, packed prompts with their states, gradients, one token

A case is a dict; `prepare` makes its inputs on the GPU, `run` is one pass in plain torch operations or
(own = True) through this repository's library, `exact` the same from the definition in 64 bits.
"""
import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}
EPS = 1e-6


# ------------------------------------------------------------------------------------------------ cases

def listed():
    return [
        # the norm before a layer for one new token of a small serving batch: latency
        dict(name="norm_token", op="norm", dir="forward", B=8, N=1, C=2048, residual=True, bits=16, type="bf16"),
        # the norm before a layer at the standard training shape's 4 x 4096 tokens of 16 heads x 128 channels
        dict(name="norm_train", op="norm", dir="forward", B=4, N=4096, C=2048, residual=True, bits=16, type="bf16"),
        # a serving batch's prompts on their way into an 8-bit projection, a scale for each 128 channels
        dict(name="norm_8bit", op="norm", dir="forward", B=1, N=12000, C=4096, residual=True, bits=8, group=128, type="bf16"),
        # the norm's gradients at the 24-layer training step's 8 x 2048 tokens
        dict(name="norm_grad", op="norm", dir="backward", B=8, N=2048, C=2048, residual=True, bits=16, type="bf16"),
        # one token of one sequence through the convolution: latency
        dict(name="conv_token", op="conv", dir="step", nseq=1, tokens=1, packed=False, pad=0, C=4096, K=4, silu=True, type="bf16", resume=True),
        # a serving batch's prompts of different lengths, leaving their last inputs
        dict(name="conv_ragged", op="conv", dir="forward", nseq=12, tokens=12000, packed=True, pad=48, C=4096, K=4, silu=True, type="bf16", resume=False),
        # gradients of the convolution, odd length, fp32
        dict(name="conv_grad_f32", op="conv", dir="backward", nseq=2, tokens=4094, packed=False, pad=0, C=2048, K=4, silu=True, type="f32", resume=False),
        # one token for a large decoding batch
        dict(name="scan_step", op="scan", dir="step", nseq=256, tokens=256, packed=False, pad=0, C=4096, G=1, S=16, gated=True, type="bf16", resume=True),
        # the scan's forward at the standard training shape
        dict(name="scan_train", op="scan", dir="forward", nseq=4, tokens=16384, packed=False, pad=0, C=2048, G=1, S=16, gated=True, type="bf16", resume=False),
        # prompts' second parts in fp32, continued from their states, two groups of input and output vectors
        dict(name="scan_resume_f32", op="scan", dir="forward", nseq=7, tokens=1500, packed=True, pad=5, C=1024, G=2, S=16, gated=True, type="f32", resume=True),
        # one long prompt
        dict(name="scan_long", op="scan", dir="forward", nseq=1, tokens=65536, packed=True, pad=0, C=2048, G=1, S=16, gated=True, type="bf16", resume=False),
        # the scan's gradients at the 24-layer training step's 8 x 2048 tokens
        dict(name="scan_grad", op="scan", dir="backward", nseq=8, tokens=16384, packed=False, pad=0, C=2048, G=1, S=16, gated=True, type="bf16", resume=False),
    ]


def _log_between(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "conv", "scan", "scan"])
    kind = rng.choice(["bf16", "bf16", "f32"])
    if op == "norm":
        C = 8 * _log_between(rng, 8, 1024)
        rows = _log_between(rng, 1, 12000 * 4096 * 2 // (C * SIZE[kind]))
        B = rng.randint(1, min(8, rows))
        back = rng.random() < 0.4
        c = dict(op="norm", dir="backward" if back else "forward", B=B, N=rows // B, C=C, residual=rng.random() < 0.7, bits=16, type=kind)
        if not back and rng.random() < 0.5:
            c.update(bits=8, group=rng.choice([0, 128]))
        return c
    what = rng.choice(["step", "forward", "forward", "backward", "backward"])
    C = 16 * _log_between(rng, 4, 256)
    if what == "step":
        n = _log_between(rng, 1, 256)
        packed, tokens = False, n
    else:
        most = 8 * 2048 * 2048 if op == "scan" and what == "backward" else 12000 * 4096
        tokens = _log_between(rng, 16, min(65536, most * 2 // SIZE[kind] // C))
        packed = rng.random() < 0.5
        n = _log_between(rng, 1, min(48 if packed else 8, tokens))
        if not packed:
            tokens -= tokens % n
    c = dict(op=op, dir=what, nseq=n, tokens=tokens, packed=packed, pad=rng.randint(0, 70) if packed else 0, C=C, type=kind,
             resume=what == "step" or rng.random() < 0.5)
    if op == "conv":
        c.update(K=rng.choice([2, 3, 4, 4]), silu=rng.random() < 0.8)
    else:
        S = rng.choice([8, 16, 16, 32])
        c.update(G=rng.choice([1, 1, 2]), S=S, gated=rng.random() < 0.7)
        if S == 32 and what != "step":  # twice the work a channel
            c["C"] = 16 * max(1, C // 32)
        if c["resume"] and what == "backward":
            c["resume"] = False
    return c


def _lengths(case):
    """The sequences' lengths: even, or (packed) uneven, with lengths of one and (from four sequences on) of zero among them."""
    n, total = case["nseq"], case["tokens"]
    if not case["packed"]:
        return [total // n] * n
    if n == 1:
        return [total]
    rng = random.Random(1000003 * n + total)
    part = [rng.uniform(0.2, 1.8) for _ in range(n)]
    if n >= 4:
        part[n // 2] = 0.0
    lens = [int(total * p / sum(part)) for p in part]
    if n >= 3:
        lens[n // 3] = 1
    lens[0] += total - sum(lens)
    return lens


# ----------------------------------------------------------------------------------------------- inputs

def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, kind = case["op"], case["type"]
    dt = TYPES[kind]

    def normal(*shape, scale=1.0, dtype=dt):
        x = torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)
        return (x if scale == 1.0 else x.mul_(scale)).to(dtype)

    s = dict(case=case)
    C = case["C"]
    if op == "norm":
        shape = (case["B"], case["N"], C)
        s["w"] = 1.0 + normal(C, scale=0.1, dtype=torch.float32)
        s["x"] = normal(*shape)
        if case["dir"] == "backward":
            s["x"] = s["x"] * 2
            s["dy"] = normal(*shape)
            if case["residual"]:
                s["dr"] = normal(*shape)
            if own:
                from bwd_la_fwd_gb300 import la
                s["workspace"] = la.new_rms_norm_workspace(C)
        elif case["residual"]:
            s["r"] = normal(*shape, scale=3.0)
        return s
    n, T = case["nseq"], case["tokens"] + case["pad"]
    step = case["dir"] == "step"
    lens = _lengths(case)
    off = [0]
    for m in lens:
        off.append(off[-1] + m)
    s["offsets"] = torch.tensor(off, dtype=torch.int32, device="cuda")

    def rows(t):  # as the call takes it: [nseq, C] for one token, [T, C] packed, [nseq, N, C] otherwise
        return t if step or case["packed"] else t.unflatten(0, (n, T // n))

    xz = normal(T, 2 * C)  # one projection's output: the channels and their gates
    s["x"], s["z"] = rows(xz[:, :C]), rows(xz[:, C:])
    if case["dir"] == "backward":
        s["do"] = rows(normal(T, C))
    elif not step:
        s["o"] = rows(torch.full((T, C), 2.0 ** -6, dtype=dt, device="cuda"))  # rows behind the last prompt stay so
    if op == "conv":
        K = case["K"]
        s["w"] = normal(C, K, scale=1.0 / math.sqrt(K), dtype=torch.float32)
        s["bias"] = normal(C, scale=0.1, dtype=torch.float32)
        s["first"] = normal(n, K - 1, C) if case["resume"] else None
        s["last"] = s["first"] if step else torch.zeros(n, K - 1, C, dtype=dt, device="cuda")
        if own and not step:
            from bwd_la_fwd_gb300 import la
            s["workspace"] = la.new_short_conv_workspace(C, K)
        return s
    S, G = case["S"], case["G"]
    # steps of some 1/1000 to 1/10, decays of 1 to S times that
    want = torch.exp(torch.rand(C, generator=gen, device="cuda") * math.log(100.0) + math.log(0.001))
    s["dt_bias"] = want + torch.log(-torch.expm1(-want))
    s["dt"] = rows(normal(T, C, scale=0.5))
    s["A"] = -(torch.arange(1, S + 1, device="cuda", dtype=torch.float32) * torch.exp(normal(C, S, scale=0.2, dtype=torch.float32)))
    s["D"] = 1.0 + normal(C, scale=0.1, dtype=torch.float32)
    bc = normal(T, 2 * G, S)  # one projection's output as well
    s["B"], s["C"] = rows(bc[:, :G]), rows(bc[:, G:])
    if not case["gated"]:
        s["z"] = None
    s["first"] = normal(n, C, S, scale=0.3, dtype=torch.float32) if case["resume"] else None
    s["last"] = s["first"] if step else torch.zeros(n, C, S, dtype=torch.float32, device="cuda")
    if own and not step:
        from bwd_la_fwd_gb300 import la
        code = la.LA_BF16 if kind == "bf16" else la.LA_F32
        s["workspace"] = la.new_selective_scan_workspace(T, n, C, G, S, code, backward=case["dir"] == "backward")
        s["marks"] = None
        if not case["packed"] or case["dir"] == "backward":  # a training forward leaves what its gradient starts from
            s["marks"] = la.new_selective_scan_marks(T, n, C, S)
        if case["dir"] == "backward":
            la.la_selective_scan(*_scan_inputs(s), **_scan_options(s), marks=s["marks"], workspace=s["workspace"])
    return s


# ------------------------------------------------------------------------------------------ plain forms

def _plain_norm(s):
    c, w = s["case"], s["w"]
    r = s["x"].float()
    if c["dir"] == "backward":
        rstd = torch.rsqrt(r.square().mean(-1, keepdim=True) + EPS)
        dy = s["dy"].float()
        g = w * dy
        dx = rstd * (g - r * rstd.square() * (g * r).mean(-1, keepdim=True))
        if c["residual"]:
            dx = dx + s["dr"].float()
        return dx.to(s["x"].dtype), (dy * r * rstd).double().sum((0, 1)).float()  # a long sum: 64 bits
    if c["residual"]:
        r = r + s["r"].float()
    y = r * torch.rsqrt(r.square().mean(-1, keepdim=True) + EPS) * w
    out = [r.to(s["x"].dtype)] if c["residual"] else []
    if c["bits"] == 16:
        return [y.to(s["x"].dtype)] + out
    G = c["group"] or c["C"]
    pad = -c["C"] % G
    groups = torch.cat([y, torch.zeros_like(y[..., :pad])], -1).unflatten(-1, (-1, G))
    scale = groups.abs().amax(-1).clamp_min(2.0 ** -100) / 448.0
    y8 = (groups / scale[..., None]).clamp(-448.0, 448.0).flatten(-2)[..., :c["C"]]
    return [y8.to(torch.float8_e4m3fn), scale] + out


def _places(s):
    """Rows one behind another: each row's sequence and its place in it, and whether it has one; all on the device."""
    off = s["offsets"].long()
    T = s["case"]["tokens"] + s["case"]["pad"]
    at = torch.arange(T, device=off.device)
    seq = torch.searchsorted(off[1:], at, right=True).clamp_max(off.numel() - 2)
    return off, seq, at - off[seq], at < off[-1]


def _flat(t, tail=1):
    """[nseq, N, ...] or [T, ...] as rows."""
    return t.flatten(0, 1) if t is not None and t.dim() == tail + 2 else t


def _silu_grad(p):
    g = torch.sigmoid(p)
    return g * (1 + p * (1 - g))


def _taps(x, s, seq, pos, j):
    """The inputs under tap j: j - K + 1 rows back, from the state (or zero) before a sequence's first row."""
    K = s["case"]["K"]
    back = K - 1 - j
    at = torch.arange(x.shape[0], device=x.device)
    here = x[(at - back).clamp_min(0)]
    before = s["first"].float()[seq, (pos + j).clamp(0, K - 2)] if s["first"] is not None else torch.zeros_like(here)
    return torch.where((pos >= back)[:, None], here, before)


def _plain_conv(s):
    c, w, K = s["case"], s["w"], s["case"]["K"]
    if c["dir"] == "step":
        x = s["x"].float()
        taps = torch.cat([s["first"].float(), x[:, None]], 1)
        p = s["bias"] + (taps * w.t()).sum(1)
        s["first"].copy_(torch.cat([s["first"][:, 1:], s["x"][:, None]], 1))
        return (p * torch.sigmoid(p) if c["silu"] else p).to(s["x"].dtype), s["first"]
    off, seq, pos, live = _places(s)
    x = _flat(s["x"]).float()
    taps = [_taps(x, s, seq, pos, j) for j in range(K)]
    p = s["bias"] + sum(t * w[:, j] for j, t in enumerate(taps))
    if c["dir"] == "backward":
        dp = _flat(s["do"]).float()
        if c["silu"]:
            dp = dp * _silu_grad(p)
        dp = torch.where(live[:, None], dp, 0.0)
        left = (off[seq + 1] - off[seq] - pos)  # rows from this one to the sequence's end
        at = torch.arange(x.shape[0], device=x.device)
        dx = sum(w[:, j] * torch.where((left > K - 1 - j)[:, None], dp[(at + K - 1 - j).clamp_max(x.shape[0] - 1)], 0.0) for j in range(K))
        dx = torch.where(live[:, None], dx, 0.0).to(s["x"].dtype)
        dw = torch.stack([(dp * t).double().sum(0) for t in taps], 1).float()  # long sums: 64 bits
        return dx.view(s["x"].shape), dw, dp.double().sum(0).float()
    o = (p * torch.sigmoid(p) if c["silu"] else p).to(s["o"].dtype)
    flat = _flat(s["o"])
    flat.copy_(torch.where(live[:, None], o, flat))
    # the last K - 1 inputs: from the rows, or from the state before where there are fewer
    m = torch.arange(K - 1, device=x.device)
    place = (off[1:] - off[:-1])[:, None] - (K - 1) + m
    from_rows = _flat(s["x"])[(off[:-1, None] + place).clamp(0, x.shape[0] - 1)]
    before = torch.zeros_like(from_rows)
    if s["first"] is not None:
        before = s["first"].gather(1, (place + K - 1).clamp(0, K - 2)[..., None].expand(-1, -1, x.shape[1]))
    s["last"].copy_(torch.where((place >= 0)[..., None], from_rows, before))
    return s["o"], s["last"]


def _scan(a, x):
    """h_t = a_t h_{t-1} + x_t along dimension 0, by doubling; nothing stands before the first row."""
    d, n = 1, x.shape[0]
    while d < n:
        x = torch.cat([x[:d], torch.addcmul(x[d:], a[d:], x[:-d])])
        a = torch.cat([a[:d], a[d:] * a[:-d]])
        d *= 2
    return x


def _softplus(v):
    return v.clamp_min(0) + torch.log1p(torch.exp(-v.abs()))


def _by_channel(v, C):
    """[T, G, S] as each channel's [T, C, S]."""
    return v[:, :, None].expand(-1, -1, C // v.shape[1], -1).reshape(v.shape[0], C, v.shape[2])


def _plain_scan(s):
    c, A, D, C = s["case"], s["A"], s["D"], s["case"]["C"]
    x, z = _flat(s["x"]).float(), _flat(s["z"])
    z = z.float() if z is not None else None
    v = _flat(s["dt"]).float() + s["dt_bias"]
    d = _softplus(v)
    Bc, Cc = (_by_channel(_flat(s[k], 2).float(), C) for k in ("B", "C"))
    a = torch.exp(d[..., None] * A)
    u = (d * x)[..., None] * Bc
    gate = z * torch.sigmoid(z) if z is not None else 1.0
    if c["dir"] == "step":
        s["first"].copy_(a * s["first"] + u)
        y = (s["first"] * Cc).sum(-1) + D * x
        return (y * gate).to(s["x"].dtype), s["first"]
    off, seq, pos, live = _places(s)
    begins = off[:-1][off[1:] > off[:-1]]  # sequences that have rows
    have = off[1:] > off[:-1]
    if s["first"] is not None:
        u[begins] += a[begins] * s["first"][have]
    cut = a.clone()
    cut[begins] = 0.0
    h = _scan(cut, u)
    y = (h * Cc).sum(-1) + D * x
    if c["dir"] == "forward":
        flat = _flat(s["o"])
        flat.copy_(torch.where(live[:, None], (y * gate).to(flat.dtype), flat))
        s["last"].copy_(s["first"] if s["first"] is not None else torch.zeros_like(s["last"]))
        s["last"][have] = h[off[1:][have] - 1]
        return s["o"], s["last"]
    do = torch.where(live[:, None], _flat(s["do"]).float(), 0.0)
    g = do * gate
    later = torch.cat([cut[1:], torch.zeros_like(cut[:1])])
    Gr = _scan(later.flip(0), (g[..., None] * Cc).flip(0)).flip(0)
    before = torch.cat([torch.zeros_like(h[:1]), h[:-1]])  # gradients start from empty states
    before[begins] = 0.0
    e = a * before * Gr
    dd = (e * A).sum(-1) + x * (Gr * Bc).sum(-1)
    dt = s["x"].dtype
    grouped = lambda t: t.unflatten(1, (c["G"], -1)).sum(2).to(dt)  # noqa: E731
    out = dict(dx=(d * (Gr * Bc).sum(-1) + D * g).to(dt), ddt=torch.where(live[:, None], dd * torch.sigmoid(v), 0.0))
    out.update(dA=(e * d[..., None]).double().sum(0).float(), dB=grouped(Gr * (d * x)[..., None]), dC=grouped(g[..., None] * h),
               dD=(g * x).double().sum(0).float(), dbias=out["ddt"].double().sum(0).float())
    out["ddt"] = out["ddt"].to(dt)
    if z is not None:
        out["dz"] = (do * y * _silu_grad(z)).to(dt)
    for k in ("dx", "ddt", "dz"):
        if k in out:
            out[k] = out[k].view(s["x"].shape)
    out["dB"], out["dC"] = out["dB"].view(s["B"].shape), out["dC"].view(s["B"].shape)
    return out


# ----------------------------------------------------------------------------------- through the library

def _scan_inputs(s):
    return s["x"], s["dt"], s["A"], s["B"], s["C"]


def _scan_options(s):
    return dict(D=s["D"], z=s["z"], dt_bias=s["dt_bias"], softplus=True, seq_offsets=s["offsets"] if s["case"]["packed"] else None)


def _own(s):
    from bwd_la_fwd_gb300 import la
    c = s["case"]
    if c["op"] == "norm":
        if c["dir"] == "backward":
            return la.la_rms_norm_backward(s["x"], s["w"], s["dy"], dR=s.get("dr"), eps=EPS, workspace=s["workspace"])
        if c["bits"] == 8:
            y8, scale, r = la.la_rms_norm_8bit(s["x"], s["w"], residual=s.get("r"), group=c["group"], eps=EPS)
            return [y8, scale] + ([r] if c["residual"] else [])
        y, r = la.la_rms_norm(s["x"], s["w"], residual=s.get("r"), eps=EPS)
        return [y] + ([r] if c["residual"] else [])
    if c["op"] == "conv":
        act = "silu" if c["silu"] else "none"
        if c["dir"] == "step":
            return la.la_short_conv_step(s["first"], s["x"], s["w"], bias=s["bias"], activation=act), s["first"]
        off = s["offsets"] if c["packed"] else None
        if c["dir"] == "backward":
            return la.la_short_conv_backward(s["x"], s["w"], s["do"], bias=s["bias"], activation=act, seq_offsets=off,
                                             state_in=s["first"], workspace=s["workspace"])
        o = la.la_short_conv(s["x"], s["w"], bias=s["bias"], activation=act, seq_offsets=off, state_in=s["first"],
                             state_out=s["last"], O=s["o"], workspace=s["workspace"])
        return o, s["last"]
    if c["dir"] == "step":
        y = la.la_selective_scan_step(s["first"], *_scan_inputs(s), D=s["D"], z=s["z"], dt_bias=s["dt_bias"], softplus=True)
        return y, s["first"]
    if c["dir"] == "backward":
        got = la.la_selective_scan_backward(*_scan_inputs(s), s["do"], s["marks"], **_scan_options(s), workspace=s["workspace"])
        out = dict(dx=got.dX, ddt=got.ddt, dA=got.dA, dB=got.dB, dC=got.dC, dD=got.dD, dbias=got.ddt_bias)
        return out if s["z"] is None else {**out, "dz": got.dz}
    y = la.la_selective_scan(*_scan_inputs(s), **_scan_options(s), state_in=s["first"], state_out=s["last"], marks=s["marks"],
                             Y=s["o"], workspace=s["workspace"])
    return y, s["last"]


def run(state):
    if own:
        return _own(state)
    return {"norm": _plain_norm, "conv": _plain_conv, "scan": _plain_scan}[state["case"]["op"]](state)


# ----------------------------------------------------------------------------------------------- the floor

def work(case):
    e, C = SIZE[case["type"]], case["C"]
    if case["op"] == "norm":
        n = case["B"] * case["N"] * C
        if case["dir"] == "backward":
            return {"bytes": n * e * (4 if case["residual"] else 3) + 8 * C, "flops": 12 * n}
        y = e if case["bits"] == 16 else 1
        scales = 0 if case["bits"] == 16 else case["B"] * case["N"] * (-(-C // case["group"]) if case["group"] else 1) * 4
        return {"bytes": n * (e * (3 if case["residual"] else 1) + y) + scales + 4 * C, "flops": 6 * n}
    T, n = case["tokens"], case["nseq"]
    states = 2 if case["resume"] else 1
    if case["op"] == "conv":
        K = case["K"]
        held = n * (K - 1) * C * e * (states if case["dir"] != "backward" else states - 1)
        return {"bytes": T * C * e * (3 if case["dir"] == "backward" else 2) + held + C * 4 * (K + 1) * (2 if case["dir"] == "backward" else 1),
                "flops": T * C * 2 * K * (3 if case["dir"] == "backward" else 1)}
    S, G = case["S"], case["G"]
    held = n * C * S * 4 * states
    params = C * 4 * (S + 2)
    gate = 1 if case["gated"] else 0
    if case["dir"] == "backward":  # x, dt, dout, z in; dx, ddt, dz out; B, C and their gradients
        return {"bytes": T * C * e * (5 + 2 * gate) + 4 * T * G * S * e + 2 * params, "flops": 26 * T * C * S}
    return {"bytes": T * C * e * (3 + gate) + 2 * T * G * S * e + params + held, "flops": 8 * T * C * S}


# ------------------------------------------------------------------------------------------- in 64 bits

def _exact_norm(s):
    c, w, x = s["case"], s["w"].double(), s["x"].double()
    if c["dir"] == "backward":
        ms = (x * x).sum(-1, keepdim=True) / c["C"] + EPS
        xhat = x / ms.sqrt()
        g = s["dy"].double() * w
        dx = (g - xhat * ((g * xhat).sum(-1, keepdim=True) / c["C"])) / ms.sqrt()
        if c["residual"]:
            dx = dx + s["dr"].double()
        return dx, (s["dy"].double() * xhat).sum((0, 1))
    if c["residual"]:
        x = x + s["r"].double()
    y = w * x / ((x * x).sum(-1, keepdim=True) / c["C"] + EPS).sqrt()
    out = [x] if c["residual"] else []
    if c["bits"] == 16:
        return [y] + out
    G = c["group"] or c["C"]
    parts = y.split(G, -1)
    scale = torch.stack([p.abs().amax(-1) for p in parts], -1).clamp_min(2.0 ** -100) / 448
    y8 = torch.cat([p / scale[..., i, None] for i, p in enumerate(parts)], -1)
    return [y8, scale] + out


def _padded(s):
    """Row indices [nseq, longest] of each sequence (0 where it has none), and where it has one."""
    off = s["offsets"].long().cpu()
    lens = off[1:] - off[:-1]
    at = torch.arange(max(1, int(lens.max())))
    live = at[None] < lens[:, None]
    return torch.where(live, off[:-1, None] + at, 0).cuda(), live.cuda()


def _exact_conv(s):
    c, K, w = s["case"], s["case"]["K"], s["w"].double()
    n, C = c["nseq"], c["C"]
    act = (lambda p: p / (1 + torch.exp(-p))) if c["silu"] else (lambda p: p)
    if c["dir"] == "step":
        taps = torch.cat([s["first"].double(), s["x"].double()[:, None]], 1)
        return act(s["bias"].double() + torch.einsum("bkc,ck->bc", taps, w)), taps[:, 1:]
    index, live = _padded(s)
    L = index.shape[1]
    x = torch.where(live[..., None], _flat(s["x"]).double()[index], 0.0)
    first = s["first"].double() if s["first"] is not None else torch.zeros(n, K - 1, C, dtype=torch.float64, device="cuda")
    xs = torch.cat([first, x], 1)  # row t of a sequence stands at t + K - 1
    p = s["bias"].double() + sum(xs[:, j:j + L] * w[:, j] for j in range(K))
    if c["dir"] == "backward":
        dp = torch.where(live[..., None], _flat(s["do"]).double()[index], 0.0)
        if c["silu"]:
            e = torch.exp(-p)
            dp = dp * (1 / (1 + e) + p * e / (1 + e) ** 2)
        after = torch.cat([dp, torch.zeros(n, K - 1, C, dtype=torch.float64, device="cuda")], 1)
        dx = sum(after[:, K - 1 - j:K - 1 - j + L] * w[:, j] for j in range(K))
        full = torch.zeros(c["tokens"] + c["pad"], C, dtype=torch.float64, device="cuda")
        full[index[live]] = dx[live]
        dw = torch.stack([(dp * xs[:, j:j + L]).sum((0, 1)) for j in range(K)], 1)
        return full.view(s["x"].shape), dw, dp.sum((0, 1))
    full = _flat(s["o"]).double()
    full[index[live]] = act(p)[live]
    lens = live.sum(1)
    last = xs.gather(1, (lens[:, None] + torch.arange(K - 1, device="cuda"))[..., None].expand(-1, -1, C))
    return full.view(s["o"].shape), last


def _exact_scan(s):
    c, A, D = s["case"], s["A"].double(), s["D"].double()
    n, C, S, G = c["nseq"], c["C"], c["S"], c["G"]
    r = C // G
    v = _flat(s["dt"]).double() + s["dt_bias"].double()
    d = torch.logaddexp(v, torch.zeros_like(v))
    x = _flat(s["x"]).double()
    z = _flat(s["z"]).double() if s["z"] is not None else None
    Bm, Cm = (_flat(s[k], 2).double() for k in ("B", "C"))
    gate = z / (1 + torch.exp(-z)) if z is not None else torch.ones_like(x)
    h = s["first"].double() if s["first"] is not None else torch.zeros(n, C, S, dtype=torch.float64, device="cuda")
    if c["dir"] == "step":
        h = torch.exp(d[..., None] * A) * h + (d * x)[..., None] * Bm.repeat_interleave(r, 1)
        return ((h * Cm.repeat_interleave(r, 1)).sum(-1) + D * x) * gate, h
    index, live = _padded(s)
    L, on = index.shape[1], live.t()[..., None]

    def by_time(t):  # [T, ...] as [longest, nseq, ...]; zero where a sequence has no row: nothing happens there
        t = t[index.t()]
        return torch.where(on if t.dim() == 3 else on[..., None], t, 0.0)

    dp, up, Bp, Cp = by_time(d), by_time(d * x), by_time(Bm), by_time(Cm)
    back = c["dir"] == "backward"
    y = torch.empty(L, n, C, dtype=torch.float64, device="cuda")
    kept = []
    for t in range(L):
        if back:
            kept.append(h)
        u = (up[t].view(n, G, r, 1) * Bp[t][:, :, None]).view(n, C, S)
        h = torch.addcmul(u, torch.exp(dp[t][..., None] * A), h)
        torch.matmul(h.view(n, G, r, S), Cp[t][..., None], out=y[t].view(n, G, r, 1))
    at = index.t()[live.t()]
    full = torch.zeros_like(x)
    full[at] = y[live.t()]
    full = full + D * x
    if not back:
        out = _flat(s["o"]).double()
        out[at] = (full * gate)[at]
        return out.view(s["o"].shape), h
    inside = torch.zeros(x.shape[0], 1, dtype=torch.bool, device="cuda")
    inside[at] = True
    do = torch.where(inside, _flat(s["do"]).double(), 0.0)
    g = do * gate
    gp = by_time(g)
    dBp, dCp, W, E = torch.empty_like(Bp), torch.empty_like(Cp), torch.empty_like(dp), torch.empty_like(dp)
    dA = torch.zeros_like(A)
    P = torch.zeros(n, C, S, dtype=torch.float64, device="cuda")  # a_{t+1} G_{t+1}
    for t in range(L - 1, -1, -1):
        Gt = (gp[t].view(n, G, r, 1) * Cp[t][:, :, None]).view(n, C, S) + P
        u = (up[t].view(n, G, r, 1) * Bp[t][:, :, None]).view(n, C, S)
        a = torch.exp(dp[t][..., None] * A)
        P = a * Gt
        e = P * kept[t]
        by_group = Gt.view(n, G, r, S)
        torch.matmul(by_group, Bp[t][..., None], out=W[t].view(n, G, r, 1))
        torch.matmul(up[t].view(n, G, 1, r), by_group, out=dBp[t].view(n, G, 1, S))
        torch.matmul(gp[t].view(n, G, 1, r), torch.addcmul(u, a, kept[t]).view(n, G, r, S), out=dCp[t].view(n, G, 1, S))
        torch.sum(e * A, -1, out=E[t])
        dA += (e * dp[t][..., None]).sum(0)

    def by_row(t):
        out = torch.zeros(x.shape[0], *t.shape[2:], dtype=torch.float64, device="cuda")
        out[at] = t[live.t()]
        return out

    W, E, dB, dC = by_row(W), by_row(E), by_row(dBp), by_row(dCp)
    dx, dd = d * W + D * g, E + x * W
    ddt = torch.where(inside, dd / (1 + torch.exp(-v)), 0.0)
    shape = s["x"].shape
    out = dict(dx=dx.view(shape), ddt=ddt.view(shape), dA=dA, dB=dB.view(s["B"].shape), dC=dC.view(s["C"].shape),
               dD=(g * x).sum(0), dbias=ddt.sum(0))
    if z is not None:
        e = torch.exp(-z)
        out["dz"] = (do * full * (1 / (1 + e) + z * e / (1 + e) ** 2)).view(shape)
    return out


def exact(case, seed):
    if case["op"] == "scan" and case["dir"] == "backward" and max(_lengths(case)) > 20000:
        return None  # row by row it takes too long
    s = prepare(case, seed)
    return {"norm": _exact_norm, "conv": _exact_conv, "scan": _exact_scan}[case["op"]](s)
