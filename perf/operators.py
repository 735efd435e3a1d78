"""The operators around the linear-attention head, as cases that can be timed and compared.

rotary   positions rotated into Q and K (training: whole sequences and their gradients; decoding: one token)
scan     the gated linear recurrence h_t = a_t h_{t-1} + b_t x_t: forward, backward, one step
prompt   the causal head over packed prompts with grouped heads, leaving (or resuming) the recurrent state
decode   one token per sequence for grouped heads, the state advanced in place

A case is a dict; `prepare` makes its inputs on the GPU, `run` is one pass in plain torch operations or
(own = True) through this repository's library, `exact` the same from the definition in 64 bits.
"""
import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}


# ------------------------------------------------------------------------------------------------ cases

def listed():
    return [
        # the position of one new token in Q and K of a small serving batch, far into its context
        dict(name="rotary_token", op="rotary", B=8, N=1, Hq=16, Hk=4, D=128, R=128, interleaved=False, inverse=False,
             scaling="by_turns", type="bf16", far=1000000),
        # the standard training shape: Q and K slices of one fused projection
        dict(name="rotary_train", op="rotary", B=4, N=4096, Hq=16, Hk=16, D=128, R=128, interleaved=False, inverse=False,
             scaling="none", type="bf16", far=0),
        # gradients through a rotation of half of each head, odd length, fp32
        dict(name="rotary_grad_f32", op="rotary", B=2, N=2047, Hq=16, Hk=4, D=128, R=64, interleaved=True, inverse=True,
             scaling="linear", type="f32", far=0),
        # one token of the recurrence for a serving batch
        dict(name="scan_step", op="scan", dir="step", B=256, N=1, C=2048, gate="sigmoid", type="bf16"),
        # the recurrence over the standard training shape's 4 x 4096 tokens, 16 heads of 128 channels
        dict(name="scan_train", op="scan", dir="forward", B=4, N=4096, C=2048, gate="sigmoid", type="bf16"),
        # one long sequence, few channels, packed with restarts
        dict(name="scan_long_f32", op="scan", dir="forward", B=1, N=65536, C=512, gate="log", type="f32"),
        # the gradients at the 24-layer training step's 8 x 2048 tokens
        dict(name="scan_grad", op="scan", dir="backward", B=8, N=2048, C=2048, gate="log", type="bf16"),
        # a serving batch's prompts of different lengths
        dict(name="prompt_ragged", op="prompt", nseq=12, tokens=12000, pad=48, Hq=16, Hkv=4, D=128, type="bf16", resume=False),
        # one long prompt
        dict(name="prompt_long", op="prompt", nseq=1, tokens=65536, pad=0, Hq=16, Hkv=4, D=128, type="bf16", resume=False),
        # short prompts' second parts in fp32, narrow heads, continued from their states
        dict(name="prompt_resume_f32", op="prompt", nseq=7, tokens=1500, pad=5, Hq=8, Hkv=4, D=64, type="f32", resume=True),
        # one sequence decoded: latency
        dict(name="decode_one", op="decode", B=1, Hq=16, Hkv=4, D=128, type="bf16"),
        # a large decoding batch
        dict(name="decode_batch", op="decode", B=256, Hq=32, Hkv=8, D=128, type="bf16"),
    ]


def _log_between(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotary", "scan", "scan", "prompt", "prompt", "decode"])
    kind = rng.choice(["bf16", "bf16", "f32"])
    if op == "rotary":
        D = rng.choice([32, 64, 128, 256])
        Hk = rng.choice([1, 2, 4, 8, 16])
        Hq = Hk * rng.choice([1, 2, 4]) if Hk < 16 else 16
        tokens = _log_between(rng, 1, 4 * 4096 * 32 * 128 // ((Hq + Hk) * D * (SIZE[kind] // 2)))
        B = rng.randint(1, min(8, tokens))
        return dict(op="rotary", B=B, N=max(1, tokens // B), Hq=Hq, Hk=Hk, D=D, R=D if rng.random() < 0.5 else 2 * rng.randint(1, D // 2),
                    interleaved=rng.random() < 0.5, inverse=rng.random() < 0.5, scaling=rng.choice(["none", "linear", "by_turns"]),
                    type=kind, far=rng.choice([0, rng.randint(1, 1000000)]))
    if op == "scan":
        C = 8 * _log_between(rng, 2, 512)
        what = rng.choice(["step", "forward", "forward", "backward", "backward"])
        most = 8 * 2048 * 2048 // C * 2 // SIZE[kind]
        if what == "step":
            return dict(op="scan", dir="step", B=_log_between(rng, 1, 512), N=1, C=C, gate=rng.choice(["log", "sigmoid"]), type=kind)
        N = _log_between(rng, 1, min(most, 65536))
        return dict(op="scan", dir=what, B=rng.randint(1, max(1, min(16, most // N))), N=N, C=C, gate=rng.choice(["log", "sigmoid"]), type=kind)
    Hkv = rng.choice([1, 2, 4, 8])
    r = rng.choice([1, 2, 4, 8]) if Hkv < 8 else rng.choice([1, 2, 4])
    D = rng.choice([32, 64, 128, 128])
    if op == "decode":
        return dict(op="decode", B=_log_between(rng, 1, 256 if kind == "bf16" else 64), Hq=Hkv * r, Hkv=Hkv, D=D, type=kind)
    nseq = _log_between(rng, 1, 64)
    tokens = _log_between(rng, max(nseq, 16), 65536 * 16 // max(16, Hkv * r) if kind == "bf16" else 2000)
    return dict(op="prompt", nseq=nseq, tokens=tokens, pad=rng.randint(0, 70), Hq=Hkv * r, Hkv=Hkv, D=D, type=kind,
                resume=rng.random() < 0.5)


def _lengths(case):
    """The sequences' lengths: uneven, with lengths of one and (from four sequences on) of zero among them."""
    n, total = case["nseq"], case["tokens"]
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

def _frequencies(case):
    """Radians per position of each pair, in 64 bits."""
    R = case["R"]
    f = [10000.0 ** (-2.0 * i / R) for i in range(R // 2)]
    if case["scaling"] == "linear":
        f = [x / 4.0 for x in f]
    if case["scaling"] == "by_turns":  # pairs of few turns over 8192 positions slow down, those of many stay
        out = []
        for x in f:
            t = min(1.0, max(0.0, (8192.0 * x / (2.0 * math.pi) - 1.0) / (32.0 - 1.0)))
            out.append((1.0 - t) * x / 8.0 + t * x)
        f = out
    return f


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, kind = case["op"], case["type"]
    dt = TYPES[kind]

    def normal(*shape, scale=1.0, dtype=dt):
        x = torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)
        return (x if scale == 1.0 else x * scale).to(dtype)

    s = dict(case=case)
    if op == "rotary":
        B, N, Hq, Hk, D = (case[x] for x in ("B", "N", "Hq", "Hk", "D"))
        # one projection's output [B, N, Hq + 2 Hk, D]; Q and K are views of it (their gradients likewise)
        x = normal(B, N, Hq + 2 * Hk, D, scale=1.0 / math.sqrt(D))
        s["q"] = x[:, :, :Hq].transpose(1, 2)
        s["k"] = x[:, :, Hq:Hq + Hk].transpose(1, 2)
        first = torch.randint(0, case["far"] + 1, (B, 1), generator=gen, device="cuda", dtype=torch.int32)
        s["positions"] = first + torch.arange(N, device="cuda", dtype=torch.int32)
        s["frequencies"] = torch.tensor(_frequencies(case), dtype=torch.float64, device="cuda")
        s["magnitude"] = 1.25 if case["scaling"] == "by_turns" else 1.0
        if own:
            from bwd_la_fwd_gb300 import la
            scaled = {"none": {}, "linear": dict(factor=4.0),
                      "by_turns": dict(factor=8.0, original_length=8192, low_turns=1.0, high_turns=32.0)}[case["scaling"]]
            s["plan"] = la.la_rotary_frequencies(case["R"], 10000.0, case["scaling"], **scaled)
    elif op == "scan":
        B, N, C = (case[x] for x in ("B", "N", "C"))
        x = normal(B, N, C)
        if case["gate"] == "log":  # decays over some ten to a thousand tokens; one gate in 997 starts anew
            w = (-torch.exp(normal(B, N, C, scale=1.2, dtype=torch.float32) - 4.0)).to(dt)
            cut = torch.rand(B, N, 1, generator=gen, device="cuda") < 1.0 / 997.0
            w = torch.where(cut, torch.full_like(w, -math.inf), w)
        else:
            w = (normal(B, N, C, scale=1.5, dtype=torch.float32) + 3.0).to(dt)
        h0 = normal(B, C, dtype=torch.float32)
        s.update(x=x, w=w, h0=h0)
        if case["dir"] == "step":
            s.update(x=x[:, 0], w=w[:, 0])
        if case["dir"] == "backward":
            a, b = _gates(w.float(), case["gate"])
            s["h"] = _scan(a, b * x.float(), h0).to(dt)
            s["dh"] = normal(B, N, C)
            s["dh_last"] = normal(B, C, dtype=torch.float32)
    else:
        Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
        acc = torch.float32 if kind == "bf16" else torch.float64
        B = case["nseq"] if op == "prompt" else case["B"]
        T = case["tokens"] + case["pad"] if op == "prompt" else B
        qkv = normal(T, Hq + 2 * Hkv, D)
        qkv[:, :Hq + Hkv] /= math.sqrt(D)
        s.update(q=qkv[:, :Hq], k=qkv[:, Hq:Hq + Hkv], v=qkv[:, Hq + Hkv:])
        if op == "prompt":
            lens = _lengths(case)
            off = [0]
            for n in lens:
                off.append(off[-1] + n)
            s.update(offsets=torch.tensor(off, dtype=torch.int32, device="cuda"), longest=max(lens))
            s["o"] = torch.full((T, Hq, D), 2.0 ** -6, dtype=dt, device="cuda")  # rows behind the last prompt stay so
        # what some thousand earlier tokens leave; a prompt that is not resumed overwrites it
        n0 = torch.randint(1, 4000, (B, Hkv), generator=gen, device="cuda", dtype=torch.int32)
        if op == "prompt":
            n0 = n0[:, :1].repeat(1, Hkv)
        root = n0.double().sqrt()
        s["S"] = (normal(B, Hkv, D, D, dtype=torch.float32).to(acc) * (root / math.sqrt(D))[..., None, None].to(acc)).contiguous()
        s["z"] = (normal(B, Hkv, D, dtype=torch.float32).to(acc) * (root / math.sqrt(D))[..., None].to(acc)).contiguous()
        s["a"] = (normal(B, Hkv, D, dtype=torch.float32).to(acc) * root[..., None].to(acc)).contiguous()
        s["n"] = n0.contiguous()
        if own:
            from bwd_la_fwd_gb300 import la
            state = la.DecodeState(B, Hkv, D, dt, tensors=(s["S"], s["z"], s["a"], s["n"]))
            s["state"] = state
            if op == "prompt":
                s["workspace"] = la.new_prompt_workspace(T, B, Hq, Hkv, D, la.LA_BF16 if kind == "bf16" else la.LA_F32)
    return s


# ------------------------------------------------------------------------------------------ plain forms

def _rotate(x, cos, sin, R, interleaved):
    """x [B, H, N, D] in 32 bits; cos, sin [B, 1, N, R / 2]."""
    y = x.clone()
    if interleaved:
        x1, x2 = x[..., 0:R:2], x[..., 1:R:2]
        y[..., 0:R:2] = x1 * cos - x2 * sin
        y[..., 1:R:2] = x1 * sin + x2 * cos
    else:
        x1, x2 = x[..., :R // 2], x[..., R // 2:R]
        y[..., :R // 2] = x1 * cos - x2 * sin
        y[..., R // 2:R] = x1 * sin + x2 * cos
    return y


def _plain_rotary(s):
    c = s["case"]
    angle = s["positions"].double()[:, None, :, None] * s["frequencies"]  # far positions: 64 bits
    if c["inverse"]:
        angle = -angle
    cos, sin = (angle.cos() * s["magnitude"]).float(), (angle.sin() * s["magnitude"]).float()
    return [_rotate(x.float(), cos, sin, c["R"], c["interleaved"]).to(x.dtype) for x in (s["q"], s["k"])]


def _gates(w, gate):
    """a and b of h_t = a_t h_{t-1} + b_t x_t."""
    if gate == "log":
        return torch.exp(w), torch.ones((), dtype=w.dtype, device=w.device)
    return torch.sigmoid(w), torch.sigmoid(-w)


def _scan(a, x, h0):
    """h_t = a_t h_{t-1} + x_t along dimension 1, by doubling."""
    x = torch.cat([(x[:, 0] + a[:, 0] * h0)[:, None], x[:, 1:]], 1)
    d, n = 1, x.shape[1]
    while d < n:
        x = torch.cat([x[:, :d], x[:, d:] + a[:, d:] * x[:, :-d]], 1)
        a = torch.cat([a[:, :d], a[:, d:] * a[:, :-d]], 1)
        d *= 2
    return x


def _plain_scan(s):
    c = s["case"]
    x, w, h0 = s["x"].float(), s["w"].float(), s["h0"]
    a, b = _gates(w, c["gate"])
    if c["dir"] == "step":
        h0.copy_(a * h0 + b * x)
        return h0.to(s["x"].dtype), h0
    if c["dir"] == "forward":
        h = _scan(a, b * x, h0)
        return h.to(s["x"].dtype), h[:, -1].contiguous()
    h, dh = s["h"].float(), s["dh"].float()
    before = torch.cat([h0[:, None], h[:, :-1]], 1)
    # G_t = dh_t + a_{t+1} G_{t+1}, from the back; behind the end stands dh_last
    later = torch.cat([torch.ones_like(a[:, :1]), a.flip(1)[:, :-1]], 1)
    G = _scan(later, dh.flip(1), s["dh_last"]).flip(1)
    dw = a * before * G if c["gate"] == "log" else a * b * (before - x) * G
    return (b * G).to(s["x"].dtype), dw.to(s["x"].dtype), a[:, 0] * G[:, 0]


CHUNK = 128


def _plain_prompt(s):
    """Sequences padded to whole chunks; within a chunk the weights, between chunks the summed state."""
    c = s["case"]
    n, Hq, G, D = c["nseq"], c["Hq"], c["Hkv"], c["D"]
    r, chunks = Hq // G, max(1, -(-s["longest"] // CHUNK))
    off = s["offsets"].long()
    at = torch.arange(chunks * CHUNK, device=off.device)
    inside = at[None] < (off[1:] - off[:-1])[:, None]
    index = torch.where(inside, off[:-1, None] + at, 0)
    acc = s["S"].dtype
    live = inside[..., None, None]
    q = torch.where(live, s["q"][index].float(), 0.0).view(n, chunks, CHUNK, G, r, D).permute(0, 1, 3, 4, 2, 5)
    k = torch.where(live, s["k"][index].float(), 0.0).view(n, chunks, CHUNK, G, D).transpose(2, 3)
    v = torch.where(live, s["v"][index].float(), 0.0).view(n, chunks, CHUNK, G, D).transpose(2, 3)
    count = inside.view(n, chunks, CHUNK).sum(2)[..., None].expand(n, chunks, G)
    keep = 1 if c["resume"] else 0

    def carried(first, sums):
        """The state before each chunk and after the last, sums over long sequences in 64 bits."""
        run = torch.cat([keep * first[:, None].double(), sums.double()], 1).cumsum(1)
        return run[:, :-1].float(), run[:, -1].to(first.dtype)

    S, S1 = carried(s["S"], k.to(acc).transpose(-1, -2) @ v.to(acc))
    z, z1 = carried(s["z"], k.to(acc).sum(-2))
    a, a1 = carried(s["a"], v.to(acc).sum(-2))
    m, m1 = carried(s["n"], count)
    weight = torch.tril(1.0 + q @ k[:, :, :, None].transpose(-1, -2))
    g = weight.sum(-1) + m[..., None, None] + (q @ z[:, :, :, None, :, None])[..., 0]
    o = weight @ v[:, :, :, None] + q @ S[:, :, :, None] + a[:, :, :, None, None]
    o = (o / g[..., None]).permute(0, 1, 4, 2, 3, 5).reshape(n, chunks * CHUNK, Hq, D)
    s["o"][index[inside]] = o[inside].to(s["o"].dtype)
    s["S"].copy_(S1), s["z"].copy_(z1), s["a"].copy_(a1), s["n"].copy_(m1)
    return s["o"], s["S"], s["z"], s["a"], s["n"]


def _plain_decode(s):
    c = s["case"]
    B, G, D = c["B"], c["Hkv"], c["D"]
    acc = s["S"].dtype
    q, k, v = (s[x].to(acc) for x in ("q", "k", "v"))
    q = q.reshape(B, G, -1, D)
    s["S"] += k[..., :, None] * v[..., None, :]
    s["z"] += k
    s["a"] += v
    s["n"] += 1
    g = s["n"][..., None].to(acc) + (q * s["z"][:, :, None]).sum(-1)
    o = (s["a"][:, :, None] + q @ s["S"]) / g[..., None]
    return o.reshape(B, G * q.shape[2], D).to(s["q"].dtype), s["S"], s["z"], s["a"], s["n"]


def _own(s):
    from bwd_la_fwd_gb300 import la
    c = s["case"]
    if c["op"] == "rotary":
        call = la.la_rotary_backward if c["inverse"] else la.la_rotary
        return list(call(s["q"], s["k"], s["plan"], positions=s["positions"], interleaved=c["interleaved"], magnitude=s["magnitude"]))
    if c["op"] == "scan":
        if c["dir"] == "step":
            return la.la_gated_scan_step(s["h0"], s["x"], s["w"], c["gate"]), s["h0"]
        if c["dir"] == "forward":
            return la.la_gated_scan(s["x"], s["w"], c["gate"], h0=s["h0"])
        return la.la_gated_scan_backward(s["x"], s["w"], s["h"], s["dh"], c["gate"], h0=s["h0"], dh_last=s["dh_last"])
    st = s["state"]
    if c["op"] == "prompt":
        o = la.la_prompt(s["q"], s["k"], s["v"], s["offsets"], st, resume=c["resume"], O=s["o"], workspace=s["workspace"])
    else:
        o = la.la_decode_step_grouped(st, s["q"], s["k"], s["v"])
    return o, st.S, st.z, st.a, st.n


def run(state):
    if own:
        return _own(state)
    return {"rotary": _plain_rotary, "scan": _plain_scan, "prompt": _plain_prompt, "decode": _plain_decode}[state["case"]["op"]](state)


# ------------------------------------------------------------------------------- what a pass cannot avoid

def work(case):
    e = SIZE[case["type"]]
    if case["op"] == "rotary":
        x = case["B"] * case["N"] * (case["Hq"] + case["Hk"])
        return {"bytes": 2 * x * case["D"] * e + case["B"] * case["N"] * 4, "flops": 3 * x * case["R"]}
    if case["op"] == "scan":
        x, line = case["B"] * case["N"] * case["C"], case["B"] * case["C"]
        if case["dir"] == "step":
            return {"bytes": 3 * x * e + 8 * line, "flops": 2 * x}
        if case["dir"] == "forward":
            return {"bytes": 3 * x * e + 8 * line, "flops": 2 * x}
        return {"bytes": (5 if case["gate"] == "log" else 6) * x * e + 12 * line, "flops": 4 * x}
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    acc = 4 if case["type"] == "bf16" else 8
    B, tokens = (case["nseq"], case["tokens"]) if case["op"] == "prompt" else (case["B"], case["B"])
    states = B * Hkv * ((D * D + 2 * D) * acc + 4) * (1 if case["op"] == "prompt" and not case["resume"] else 2)
    return {"bytes": tokens * 2 * (Hq + Hkv) * D * e + states, "flops": tokens * 2 * (Hq + Hkv) * D * D}


# ------------------------------------------------------------------- from the definitions, in 64 bits

def _exact_rotary(s):
    c = s["case"]
    turn = torch.polar(torch.full_like(s["frequencies"], s["magnitude"]).expand(*s["positions"].shape, -1).contiguous(),
                       (-1.0 if c["inverse"] else 1.0) * s["positions"].double()[..., None] * s["frequencies"])[:, None]
    R, out = c["R"], []
    for x in (s["q"], s["k"]):
        x = x.double()
        if c["interleaved"]:
            u = torch.view_as_complex(x[..., :R].reshape(*x.shape[:-1], R // 2, 2).contiguous()) * turn
            y = torch.view_as_real(u).flatten(-2)
        else:
            u = torch.complex(x[..., :R // 2].contiguous(), x[..., R // 2:R].contiguous()) * turn
            y = torch.cat([u.real, u.imag], -1)
        out.append(torch.cat([y, x[..., R:]], -1))
    return out


def _exact_scan(s):
    c = s["case"]
    log = c["gate"] == "log"
    x, w, h = s["x"].double(), s["w"].double(), s["h0"].double()
    a = w.exp() if log else 1.0 / (1.0 + (-w).exp())
    b = torch.ones_like(a) if log else 1.0 / (1.0 + w.exp())
    if c["dir"] == "step":
        h = a * h + b * x
        return h, h
    if c["dir"] == "forward":
        u = b * x
        out = torch.empty_like(x)
        for t in range(c["N"]):
            h = torch.addcmul(u[:, t], a[:, t], h)
            out[:, t] = h
        return out, h
    hs, dh = s["h"].double(), s["dh"].double()
    G = s["dh_last"].double()
    Gs = torch.empty_like(dh)
    for t in range(c["N"] - 1, -1, -1):
        G = dh[:, t] + G  # G holds a_{t+1} G_{t+1} here
        Gs[:, t] = G
        G = a[:, t] * G
    before = torch.cat([s["h0"].double()[:, None], hs[:, :-1]], 1)
    dw = Gs * a * (before if log else b * (before - x))
    return b * Gs, dw, G


def _exact_heads(s):
    """Prompt and decode, sequence by sequence in blocks of rows: explicit weights within a block, the state of
    all rows before it."""
    c = s["case"]
    G, r, D = c["Hkv"], c["Hq"] // c["Hkv"], c["D"]
    if c["op"] == "prompt":
        off, o = s["offsets"].tolist(), s["o"].double()
    else:
        off, o = list(range(c["B"] + 1)), torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    keep = 1.0 if c["op"] == "decode" or c["resume"] else 0.0
    S, z, a = (keep * s[x].double() for x in ("S", "z", "a"))
    n = int(keep) * s["n"]
    for i in range(len(off) - 1):
        for lo in range(off[i], off[i + 1], 512):
            hi = min(lo + 512, off[i + 1])
            q = s["q"][lo:hi].double().reshape(hi - lo, G, r, D).permute(1, 2, 0, 3)
            k, v = (s[x][lo:hi].double().transpose(0, 1) for x in ("k", "v"))
            seen = torch.arange(hi - lo, device="cuda")
            W = (1.0 + torch.einsum("grid,gjd->grij", q, k)) * (seen[:, None] >= seen[None])
            g = W.sum(-1) + torch.einsum("grid,gd->gri", q, z[i]) + n[i].double()[:, None, None]
            num = torch.einsum("grij,gje->grie", W, v) + torch.einsum("grid,gde->grie", q, S[i]) + a[i][:, None, None]
            o[lo:hi] = (num / g[..., None]).permute(2, 0, 1, 3).reshape(hi - lo, G * r, D)
            S[i] += torch.einsum("gjd,gje->gde", k, v)
            z[i] += k.sum(1)
            a[i] += v.sum(1)
            n[i] += hi - lo
    return o, S, z, a, n


def exact(case, seed):
    global own
    was, own = own, False  # the inputs alone: no plan of the library
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return {"rotary": _exact_rotary, "scan": _exact_scan, "prompt": _exact_heads, "decode": _exact_heads}[case["op"]](s)
