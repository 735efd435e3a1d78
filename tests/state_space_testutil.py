"""Plain 64-bit forms of the norm, the short convolution and the selective scan, with the error that fp32 arithmetic may
leave in each element before the output's rounding.

U is half a step of fp32, 2^-24.  Bounds are worst cases: every rounding counted with its full half step against the
magnitude it applies to.  What the kernels' functions leave, in half steps of the result: e^x and 1 / (1 + e^-x) |x| + 8
(the product x log2 e, the hardware's 2^x within 2 ulp, the sum, the reciprocal), log1p 4, rsqrt 4."""
from __future__ import annotations

import torch

from ops_testutil import TYPES, U, assert_within, half_step  # noqa: F401

# What is below 2^-126 the hardware's 2^x gives as 0: a decay lost so leaves at most 2^-126 of what it multiplies, a state and
# a gradient of less than 2^8 each in these tests.
LOST = 2.0 ** -110
SUM = 200  # roundings of a sum over a row's, or a call's, blocks, beside its terms: the threads', warps' and blocks' sums


def rounded(ref, tol, kind):
    """The bound with the output's rounding to its type."""
    return tol + half_step(kind) * (ref.abs() + tol)


# ------------------------------------------------------------------------------------------------ norm

def norm(x, residual, w, eps):
    """-> (r, y) and their bounds.  r: one sum.  y: r's half step (twice, in r and in the squares), the squares' sum (a
    thread adds at most 64 of them, then come SUM others: each of them counts half under the root), the root's 4, three
    products."""
    x, w = x.double(), w.double()
    r = x + residual.double() if residual is not None else x
    y = r * w / (r.square().mean(-1, keepdim=True) + eps).sqrt()
    return (r, y), (U * r.abs(), U * ((64 + SUM) / 2 + 10) * y.abs())


def norm_backward(R, w, dY, dR, eps):
    """-> (dX, dw) and their bounds, as for norm; the sum of g R is off by its roundings times the magnitudes."""
    r, w, dy = R.double(), w.double(), dY.double()
    rstd = 1 / (r.square().mean(-1, keepdim=True) + eps).sqrt()
    g = w * dy
    m = (g * r).mean(-1, keepdim=True) * rstd.square()
    dx = rstd * (g - r * m)
    size = rstd * (g.abs() + r.abs() * rstd.square() * (g * r).abs().mean(-1, keepdim=True))
    if dR is not None:
        dx = dx + dR.double()
        size = size + dR.double().abs()
    t = dy * r * rstd
    rows = t.reshape(-1, t.shape[-1])
    n = rows.shape[0]
    return (dx, rows.sum(0)), (U * 2 * (64 + SUM) * size, U * (n + 2 * SUM) * rows.abs().sum(0))


# -------------------------------------------------------------------------------------------- convolution

def silu(p):
    return p / (1 + torch.exp(-p))


def silu_grad(p):
    s = 1 / (1 + torch.exp(-p))
    return s * (1 + p * (1 - s))


def spans(offsets):
    off = [int(o) for o in offsets]
    return [(a, b) for a, b in zip(off[:-1], off[1:])]


def conv(X, W, bias, act, offsets, state):
    """X [T,C] packed -> (O, state after) with zeros outside the sequences, and O's bound: K + 1 roundings of p, which O
    follows with a slope of at most 1.1, and the logistic function."""
    x, w = X.double(), W.double()
    K, C = w.shape[1], w.shape[0]
    b = bias.double() if bias is not None else torch.zeros(C, dtype=torch.float64)
    O, tol = torch.zeros_like(x), torch.zeros_like(x)
    last = []
    for i, (lo, hi) in enumerate(spans(offsets)):
        first = state[i].double() if state is not None else torch.zeros(K - 1, C, dtype=torch.float64)
        xs = torch.cat([first, x[lo:hi]])
        n = hi - lo
        p = b + sum(xs[j:j + n] * w[:, j] for j in range(K))
        M = b.abs() + sum((xs[j:j + n] * w[:, j]).abs() for j in range(K))
        O[lo:hi] = silu(p) if act == "silu" else p
        tol[lo:hi] = U * (1.1 * (K + 1) * M + ((p.abs() + 10) * O[lo:hi].abs() if act == "silu" else 0))
        last.append(xs[n:])
    return (O, torch.stack(last) if last else torch.zeros(0, K - 1, C, dtype=torch.float64)), tol


def conv_backward(X, W, dO, bias, act, offsets, state):
    """-> (dX, dW, dbias) and their bounds.  The activation's slope is off by half the error of p (its own slope is at most
    1/2), and by the logistic function's in s and in p (1 - s)."""
    x, w, d = X.double(), W.double(), dO.double()
    K, C = w.shape[1], w.shape[0]
    b = bias.double() if bias is not None else torch.zeros(C, dtype=torch.float64)
    z = lambda *s: torch.zeros(*s, dtype=torch.float64)  # noqa: E731
    dX, eX, dW, eW, db, eb = z(*x.shape), z(*x.shape), z(C, K), z(C, K), z(C), z(C)
    rows = 0
    for i, (lo, hi) in enumerate(spans(offsets)):
        n = hi - lo
        rows += n
        first = state[i].double() if state is not None else z(K - 1, C)
        xs = torch.cat([first, x[lo:hi]])
        p = b + sum(xs[j:j + n] * w[:, j] for j in range(K))
        M = b.abs() + sum((xs[j:j + n] * w[:, j]).abs() for j in range(K))
        slope = silu_grad(p) if act == "silu" else torch.ones_like(p)
        dp = d[lo:hi] * slope
        e = U * d[lo:hi].abs() * ((0.5 * (K + 1) * M + (1 + p.abs()) * (p.abs() + 12)) if act == "silu" else 0 * M)
        after, eafter = (torch.cat([t, z(K - 1, C)]) for t in (dp, e))
        for j in range(K):
            s = slice(K - 1 - j, K - 1 - j + n)
            dX[lo:hi] += after[s] * w[:, j]
            eX[lo:hi] += (eafter[s] + U * (K + 1) * after[s].abs()) * w[:, j].abs()
            dW[:, j] += (dp * xs[j:j + n]).sum(0)
            eW[:, j] += (e * xs[j:j + n].abs()).sum(0)
        db += dp.sum(0)
        eb += e.sum(0)
    # sums of `rows` terms: each rounding against the sum of their magnitudes
    for i, (lo, hi) in enumerate(spans(offsets)):
        n = hi - lo
        first = state[i].double() if state is not None else z(K - 1, C)
        xs = torch.cat([first, x[lo:hi]])
        p = b + sum(xs[j:j + n] * w[:, j] for j in range(K))
        dp = (d[lo:hi] * (silu_grad(p) if act == "silu" else 1)).abs()
        for j in range(K):
            eW[:, j] += U * (rows + SUM) * (dp * xs[j:j + n].abs()).sum(0)
        eb += U * (rows + SUM) * dp.sum(0)
    return (dX, dW, db), (eX, eW, eb)


# --------------------------------------------------------------------------------------------------- scan

def _steps(dt, bias, softplus):
    """d, its slope and its bound: the sum dt + bias, the exponential (|v| + 8), log1p and the last sum."""
    v = dt.double() + (bias.double() if bias is not None else 0)
    if not softplus:
        return v, torch.ones_like(v), U * v.abs(), v
    d = torch.logaddexp(v, torch.zeros_like(v))
    return d, 1 / (1 + torch.exp(-v)), U * (2 * v.clamp_min(0) + (2 * v.abs() + 16) * d), v


def _wide(t, C):
    return t.double().repeat_interleave(C // t.shape[1], 1)  # [T, C, S]


def _states(x, d, ed, A, B, h, E, Hm, extra):
    """The states before and after each row, their bounds, and each row's decay with its relative bound.

    A decay is off by A's part of d's error, three roundings of the exponent and the 2 ulp (four half steps) of 2^x; the
    input by d's error and two products; the step by one rounding.  `extra`: where time is cut into parts, a
    part's decay e^(A sum d) has a sum that is off by a half step for each of its n rows, so what stood before it by n half
    steps of x e^-x <= 0.4, x = |A| sum d: 0.4 n half steps of the largest state so far, wherever in the part."""
    Hx = Hm
    before, after, eb, ea, decay, rho = [], [], [], [], [], []
    for t in range(x.shape[0]):
        a = torch.exp(d[t][:, None] * A)
        r = A.abs() * ed[t][:, None] + U * (3 * (d[t][:, None] * A).abs() + 5)
        u = (d[t] * x[t])[:, None] * B[t]
        before.append(h), eb.append(E + extra * U * Hx), decay.append(a), rho.append(r)
        E = a * E + a * Hm * (r + U) + (x[t].abs() * ed[t])[:, None] * B[t].abs() + 3 * U * u.abs()
        h = a * h + u
        Hm = a * Hm + u.abs()
        Hx = torch.maximum(Hx, Hm)
        after.append(h), ea.append(E + extra * U * Hx)
    return before, after, eb, ea, decay, rho, h, E + extra * U * Hx, Hm


def scan(x, dt, A, B, C, D, z, bias, softplus, offsets, state, extra=0):
    """Packed [T,...] -> (Y, state after) with zeros outside the sequences, and their bounds."""
    x, A = x.double(), A.double()
    T, Ch = x.shape
    S = A.shape[1]
    Bw, Cw = _wide(B, Ch), _wide(C, Ch)
    d, _, ed, _ = _steps(dt, bias, softplus)
    Dv = D.double() if D is not None else torch.zeros(Ch, dtype=torch.float64)
    Y, tol = torch.zeros_like(x), torch.zeros_like(x)
    last, elast = [], []
    for i, (lo, hi) in enumerate(spans(offsets)):
        h = state[i].double() if state is not None else torch.zeros(Ch, S, dtype=torch.float64)
        s = slice(lo, hi)
        _, after, _, ea, _, _, h, E, _ = _states(x[s], d[s], ed[s], A, Bw[s], h, torch.zeros_like(h), h.abs(), extra)
        if hi > lo:
            hs, es = torch.stack(after), torch.stack(ea)
            y = (hs * Cw[s]).sum(-1) + Dv * x[s]
            M = (hs.abs() * Cw[s].abs()).sum(-1) + (Dv * x[s]).abs()
            e = (es * Cw[s].abs()).sum(-1) + U * (S + 2) * M
            if z is not None:
                zz = z[s].double()
                gate = silu(zz)
                y, e = y * gate, e * gate.abs() + U * (zz.abs() + 11) * (M * gate.abs())
            Y[s], tol[s] = y, e
        last.append(h), elast.append(E)
    empty = torch.zeros(0, Ch, S, dtype=torch.float64)
    return (Y, torch.stack(last) if last else empty), (tol + LOST, torch.stack(elast) + LOST if last else empty)


def scan_backward(x, dt, A, B, C, dY, D, z, bias, softplus, offsets, state, dlast, extra=0):
    """-> dicts of the gradients and of their bounds (the states' bounds as in scan; G's in the same way, from g's (the gate's
    |z| + 11 half steps) and the decays'; `extra`: half steps of G behind a part's end, as of the state in scan)."""
    x, A, dY = x.double(), A.double(), dY.double()
    T, Ch = x.shape
    S, G = A.shape[1], B.shape[1]
    Bw, Cw = _wide(B, Ch), _wide(C, Ch)
    d, slope, ed, v = _steps(dt, bias, softplus)
    Dv = D.double() if D is not None else torch.zeros(Ch, dtype=torch.float64)
    zero = lambda *s: torch.zeros(*s, dtype=torch.float64)  # noqa: E731
    g = {"dX": zero(T, Ch), "ddt": zero(T, Ch), "dz": zero(T, Ch), "dA": zero(Ch, S), "dB": zero(T, Ch, S), "dC": zero(T, Ch, S),
         "dD": zero(Ch), "ddt_bias": zero(Ch), "dstate_in": zero(len(offsets) - 1, Ch, S)}
    e = {k: torch.zeros_like(t) for k, t in g.items()}
    m = {k: torch.zeros_like(t) for k, t in g.items()}  # magnitudes of what is summed over rows or channels
    for i, (lo, hi) in enumerate(spans(offsets)):
        h = state[i].double() if state is not None else zero(Ch, S)
        s = slice(lo, hi)
        before, after, eb, ea, decay, rho, _, _, _ = _states(x[s], d[s], ed[s], A, Bw[s], h, torch.zeros_like(h), h.abs(), extra)
        gate = silu(z.double()) if z is not None else torch.ones_like(x)
        P = dlast[i].double() if dlast is not None else zero(Ch, S)  # a_{t+1} G_{t+1}
        EP, MP, Gx = torch.zeros_like(P), P.abs(), P.abs()
        for t in range(hi - 1, lo - 1, -1):
            k = t - lo
            gt = dY[t] * gate[t]
            egt = U * ((z[t].double().abs() + 11) if z is not None else 0) * gt.abs()
            Gt, Gm = gt[:, None] * Cw[t] + P, (gt[:, None] * Cw[t]).abs() + MP
            EG = egt[:, None] * Cw[t].abs() + EP + U * Gm
            carried = EG  # without what a part's end leaves, which does not grow
            Gx = torch.maximum(Gx, Gm)
            EG = EG + extra * U * Gx
            a, r = decay[k], rho[k]
            P, MP = a * Gt, a * Gm
            EP = a * carried + MP * (r + U)
            w, wm = (Gt * Bw[t]).sum(-1), (Gm * Bw[t].abs()).sum(-1)
            ew = (EG * Bw[t].abs()).sum(-1) + U * (S + 1) * wm
            g["dX"][t] = d[t] * w + Dv * gt
            e["dX"][t] = d[t].abs() * ew + ed[t] * wm + 3 * U * (d[t].abs() * wm + (Dv * gt).abs()) + Dv.abs() * egt
            q, qm = P * before[k], MP * before[k].abs()
            eq = EP * before[k].abs() + MP * eb[k] + U * qm
            dd = (q * A).sum(-1) + x[t] * w
            dm = (qm * A.abs()).sum(-1) + x[t].abs() * wm
            edd = (eq * A.abs()).sum(-1) + x[t].abs() * ew + U * (S + 6) * dm
            g["ddt"][t] = dd * slope[t]
            e["ddt"][t] = edd * slope[t] + U * (v[t].abs() + 10) * dm * slope[t]
            m["ddt"][t] = dm * slope[t]
            g["dA"] += q * d[t][:, None]
            e["dA"] += eq * d[t].abs()[:, None] + qm * ed[t][:, None]
            m["dA"] += qm * d[t].abs()[:, None]
            u = d[t] * x[t]
            g["dB"][t] = Gt * u[:, None]
            e["dB"][t] = EG * u.abs()[:, None] + Gm * (x[t].abs() * ed[t] + 2 * U * u.abs())[:, None]
            m["dB"][t] = Gm * u.abs()[:, None]
            g["dC"][t] = gt[:, None] * after[k]
            e["dC"][t] = gt.abs()[:, None] * ea[k] + (egt + U * gt.abs())[:, None] * after[k].abs()
            m["dC"][t] = (gt[:, None] * after[k]).abs()
            g["dD"] += gt * x[t]
            e["dD"] += egt * x[t].abs()
            m["dD"] += (gt * x[t]).abs()
            if z is not None:
                zz = z[t].double()
                y = (after[k] * Cw[t]).sum(-1) + Dv * x[t]
                M = (after[k].abs() * Cw[t].abs()).sum(-1) + (Dv * x[t]).abs()
                ey = (ea[k] * Cw[t].abs()).sum(-1) + U * (S + 2) * M
                sg = silu_grad(zz)
                g["dz"][t] = dY[t] * y * sg
                e["dz"][t] = dY[t].abs() * (ey * sg.abs() + U * ((1 + zz.abs()) * (zz.abs() + 12) + 3) * M)
        g["dstate_in"][i], e["dstate_in"][i] = P, EP + extra * U * Gx
    g["ddt_bias"] = g["ddt"].sum(0)
    e["ddt_bias"] = e["ddt"].sum(0) + U * (T + SUM) * m["ddt"].sum(0)
    e["dA"] += U * (T + SUM) * m["dA"]
    e["dD"] += U * (T + SUM) * m["dD"]
    for k in ("dB", "dC"):  # over the group's channels
        by = lambda t: t.view(T, G, Ch // G, S).sum(2)  # noqa: E731
        g[k], e[k] = by(g[k]), by(e[k]) + U * (Ch // G + SUM) * by(m[k])
    return g, {k: t + LOST for k, t in e.items()}
