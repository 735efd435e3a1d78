"""Plain 64-bit forms of the operators around the head, with the error that fp32 arithmetic and the output's rounding
may leave in each element.

Half a step of a type is eps / 2 relative to the value; U below is fp32's, 2^-24.  Bounds are worst cases: every
rounding counted with its full half step against the sum of the magnitudes it applies to.
"""
from __future__ import annotations

import math

import torch

U = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def half_step(kind: str) -> float:
    return torch.finfo(TYPES[kind]).eps / 2


def assert_within(name, got, ref, tol):
    """|got - ref| <= tol element by element, with NaN and infinities in the same places."""
    got, ref = got.detach().double().cpu(), ref.double().cpu()
    tol = torch.as_tensor(tol, dtype=torch.float64).cpu().expand_as(ref)
    assert got.shape == ref.shape, f"{name}: shape {tuple(got.shape)} != {tuple(ref.shape)}"
    fine = torch.isfinite(ref)
    assert torch.equal(fine, torch.isfinite(got)), f"{name}: non-finite values in other places"
    over = ((got - ref).abs() - tol)[fine]
    assert over.numel() == 0 or float(over.max()) <= 0, \
        f"{name}: off by up to {float(over.max()):.3e} more than allowed at {int((over > 0).sum())} of {over.numel()}"


# ---------------------------------------------------------------------------------------------- rotary

def frequencies(R, base=10000.0, scaling="none", factor=1.0, original_length=0.0, low=1.0, high=32.0):
    out = []
    for i in range(R // 2):
        f = base ** (-2.0 * i / R)
        if scaling == "linear":
            f /= factor
        elif scaling == "by_turns":
            n = original_length * f / (2 * math.pi)
            t = min(1.0, max(0.0, (n - low) / (high - low)))
            f = (1 - t) * f / factor + t * f
        out.append(f)
    return torch.tensor(out, dtype=torch.float64)


def rotary(x, positions, freq, R, interleaved, magnitude=1.0, inverse=False):
    """x [B,H,N,D], positions [B,N] -> (y, bound on the fp32 error before the output's rounding).

    Counted per output: the phase's conversion to fp32 (2^-24 of at most pi), sincospif within 2 ulp, the products with the
    magnitude, the two products and their sum: under 12 half steps of m (|x1| + |x2|); and F's rounding with the 64-bit
    angle's own, under 4 half steps of fp64 each of p f (f <= 1), and p times the fixed point's pi 2^-64."""
    x = x.double().cpu()
    th = positions.double().cpu()[:, None, :, None] * freq * (-1 if inverse else 1)
    c, s = th.cos() * magnitude, th.sin() * magnitude
    y = x.clone()
    tol = torch.zeros_like(x)
    lo, hi = (slice(0, R, 2), slice(1, R, 2)) if interleaved else (slice(0, R // 2), slice(R // 2, R))
    x1, x2 = x[..., lo], x[..., hi]
    y[..., lo] = x1 * c - x2 * s
    y[..., hi] = x1 * s + x2 * c
    e = abs(magnitude) * (x1.abs() + x2.abs()) * (12 * U + 8 * 2.0 ** -53 * th.abs() +
                                                     math.pi * 2.0 ** -64 * positions.double().cpu().abs()[:, None, :, None])
    tol[..., lo] = e
    tol[..., hi] = e
    return y, tol


# --------------------------------------------------------------------------------------- gated recurrence

def gates(w, gate):
    if gate == "log":
        return torch.exp(w), torch.ones_like(w)
    return 1 / (1 + torch.exp(-w)), 1 / (1 + torch.exp(w))


def cut_product(a, h):
    return torch.where(a == 0, torch.zeros_like(a), a * h)


def scan(X, W, gate, h0):
    """-> h [B,N,C] in 64 bits and a bound on its error in fp32.

    A gate is off by at most 10 half steps (expf 2 ulp; sigmoid: expf, 1 + e, the quotient's 2 ulp, a product), a product
    of gates by 11 for each; a term that is t steps old passes t products and at most t / 8 + 64 sums.  With M the sum of
    the terms' magnitudes and A the sum of magnitude times age: 12 A + 72 M half steps."""
    x, w = X.double().cpu(), W.double().cpu()
    a, b = gates(w, gate)
    u = torch.where(b == 0, torch.zeros_like(x), b * x)
    h = h0.double().cpu() if h0 is not None else torch.zeros_like(x[:, 0])
    M, A = h.abs(), torch.zeros_like(h)
    hs, tol = [], []
    for t in range(x.shape[1]):
        h = cut_product(a[:, t], h) + u[:, t]
        A = cut_product(a[:, t], A + M)
        M = cut_product(a[:, t], M) + u[:, t].abs()
        hs.append(h)
        tol.append(U * (12 * A + 72 * M))
    return torch.stack(hs, 1), torch.stack(tol, 1)


def scan_backward(X, W, H, dH, gate, h0, dh_last):
    """-> (dX, dW, dh0) in 64 bits and bounds on their errors in fp32 (as for scan; dW passes five more products)."""
    x, w, h, dh = (t.double().cpu() for t in (X, W, H, dH))
    a, b = gates(w, gate)
    first = h0.double().cpu() if h0 is not None else torch.zeros_like(x[:, 0])
    before = torch.cat([first[:, None], h[:, :-1]], 1)
    P = dh_last.double().cpu() if dh_last is not None else torch.zeros_like(first)
    M, A = P.abs(), torch.zeros_like(P)
    dx, dw, ex, ew = [], [], [], []
    for t in range(x.shape[1] - 1, -1, -1):
        G, M = dh[:, t] + P, dh[:, t].abs() + M
        e = U * (12 * A + 72 * M)
        bt, at = b[:, t], a[:, t]
        dx.append(torch.where(bt == 0, torch.zeros_like(G), bt * G))
        ex.append(bt * e + 12 * U * (bt * G).abs())
        P, A, M = cut_product(at, G), cut_product(at, A + M), cut_product(at, M)
        if gate == "log":
            dw.append(torch.where(at == 0, torch.zeros_like(G), before[:, t] * P))
            f = (at * before[:, t]).abs()
        else:
            shut = (at == 0) | (bt == 0)
            dw.append(torch.where(shut, torch.zeros_like(G), at * bt * (before[:, t] - x[:, t]) * G))
            f = at * bt * (before[:, t].abs() + x[:, t].abs())
        ew.append(torch.nan_to_num(f * (e + 24 * U * G.abs()), nan=0.0))
    return [torch.stack(t[::-1], 1) for t in (dx, dw)] + [P], [torch.stack(t[::-1], 1) for t in (ex, ew)] + [
        U * (12 * A + 72 * M)]


# ------------------------------------------------------------------------------------- packed prompts, decoding

def empty_state(nseq, Hkv, D):
    z = lambda *s: torch.zeros(*s, dtype=torch.float64)  # noqa: E731
    return z(nseq, Hkv, D, D), z(nseq, Hkv, D), z(nseq, Hkv, D), torch.zeros(nseq, Hkv, dtype=torch.int64)


def prompt(Q, K, V, offsets, state, kind, tensor_cores):
    """-> (O [T,Hq,D] with zeros outside the sequences, state after), (bound of O, of S, of z, of a), by explicit weights.

    O's magnitudes: every product and sum of the numerator lies under Mag = |a| + |q|.|S| + sum_j (1 + |q_i|.|k_j|) |v_j|,
    the denominator's under Den (the same without v).  Sums of up to n + 2 D + 64 terms in fp32; on the tensor cores W and
    S are rounded once to bf16 (half a step each, so one of Mag) and z to two bf16 parts (2^-16)."""
    Q, K, V = (t.double().cpu() for t in (Q, K, V))
    S, z, a, n = (t.clone() for t in state)
    Sm, zm, am = S.abs(), z.abs(), a.abs()
    T, Hq, D = Q.shape
    r = Hq // K.shape[1]
    O, tol = torch.zeros_like(Q), torch.zeros_like(Q)
    off = [int(x) for x in offsets]
    for i in range(len(off) - 1):
        lo, hi = off[i], off[i + 1]
        for h in range(Hq):
            g = h // r
            q, k, v = Q[lo:hi, h], K[lo:hi, g], V[lo:hi, g]
            mask = torch.tril(torch.ones(hi - lo, hi - lo, dtype=torch.float64))
            W, Wm = mask * (1 + q @ k.T), mask * (1 + q.abs() @ k.T.abs())
            den = W.sum(1) + q @ z[i, g] + float(n[i, g])
            Den = Wm.sum(1) + q.abs() @ zm[i, g] + float(n[i, g])
            o = W @ v + q @ S[i, g] + a[i, g]
            Mag = Wm @ v.abs() + q.abs() @ Sm[i, g] + am[i, g]
            O[lo:hi, h] = o / den[:, None]
            c = (int(n[i, g]) + (hi - lo) + 2 * D + 64) * U
            cn, cd = (c + 2.0 ** -8, c + 2.0 ** -16) if tensor_cores else (c, c)
            tol[lo:hi, h] = (cn * Mag + cd * Den[:, None] * O[lo:hi, h].abs()) / den.abs()[:, None]
        for g in range(K.shape[1]):
            k, v = K[lo:hi, g], V[lo:hi, g]
            S[i, g] += k.T @ v
            Sm[i, g] += k.T.abs() @ v.abs()
            z[i, g] += k.sum(0)
            zm[i, g] += k.abs().sum(0)
            a[i, g] += v.sum(0)
            am[i, g] += v.abs().sum(0)
            n[i, g] += hi - lo
    tol = tol + half_step(kind) * O.abs()
    # the state: sums of n terms, in fp32 (bf16 tokens) or as pairs of floats (fp32 tokens)
    per = (U if kind == "bf16" else 2.0 ** -44) * (n.double() + 1)
    return (O, (S, z, a, n)), (tol, per[..., None, None] * Sm, per[..., None] * zm, per[..., None] * am)


def normal(gen, *shape, scale=1.0, kind="bf16"):
    return (torch.randn(*shape, generator=gen) * scale).to(TYPES[kind])
