"""The root-mean-square norm with the residual's addition, its 8-bit form and its gradients, against their definitions in
64 bits (bounds in state_space_testutil)."""
import ctypes
import math

import pytest
import torch

import state_space_testutil as R
from ops_testutil import normal

EPS = 1e-6


# ------------------------------------------------------------------------------------------------ without a GPU

def test_the_gradient_formulas_against_differences():
    gen = torch.Generator().manual_seed(1)
    r, w, dy = (torch.randn(*s, generator=gen).double() for s in ((3, 5), (5,), (3, 5)))

    def loss(r, w):
        return float((R.norm(r, None, w, EPS)[0][1] * dy).sum())

    grads, _ = R.norm_backward(r, w, dy, None, EPS)
    for k, g in enumerate(grads):
        for at in range(g.numel()):
            ends = []
            for s in (1e-5, -1e-5):
                args = [t.clone() for t in (r, w)]
                args[k].view(-1)[at] += s
                ends.append(loss(*args))
            assert abs((ends[0] - ends[1]) / 2e-5 - float(g.reshape(-1)[at])) < 1e-8


def test_refuses_on_the_host():
    from bwd_la_fwd_gb300 import la
    lib = la.load_library()

    def call(x=1 << 20, res=None, w=2 << 20, s=None, y=3 << 20, B=1, N=4, C=64, eps=EPS, dtype=1, strides=None):
        st = None if strides is None else (ctypes.c_longlong * 8)(*strides)
        return lib.la_rms_norm(x, res, w, s, y, B, N, C, eps, dtype, st, None)

    assert call(dtype=2) == 1 and call(N=-1) == 1 and call(C=0) == 1 and call(B=-1) == 1
    assert call(eps=-1.0) == 1 and call(eps=math.nan) == 1 and call(eps=math.inf) == 1
    assert call(C=16392) == 2
    assert call(x=None) == 1 and call(y=None) == 1 and call(w=None) == 1 and call(x=(1 << 20) + 8) == 1 and call(w=(2 << 20) + 4) == 1
    assert call(res=4 << 20) == 1 and call(s=4 << 20) == 1           # a residual and its sum come together
    assert call(C=33) == 1                                            # rows of 66 bytes: strides are whole 16-byte vectors
    assert call(strides=[256, 32] + [256, 64] * 3) == 1               # rows overlap
    assert call(y=(1 << 20) + 128) == 1 and call(y=2 << 20) == 1      # the output meets x (shifted), the weight
    assert call(res=4 << 20, s=3 << 20) == 1                          # the outputs meet
    assert call(N=2 ** 31 - 1) == 1 and call(B=0) == 0 and call(N=0) == 0

    def eight(y8=3 << 20, scales=4 << 20, group=128, x=1 << 20, B=1, N=4, C=64):
        return lib.la_rms_norm_8bit(x, None, 2 << 20, None, y8, scales, group, B, N, C, EPS, 1, None, None)

    assert eight(group=64) == 1 and eight(y8=None) == 1 and eight(scales=None) == 1 and eight(scales=3 << 20) == 1
    assert eight(y8=1 << 20) == 1 and eight(y8=(3 << 20) + 8) == 1 and eight(N=0) == 0 and eight(y8=None, B=0) == 0

    def back(r=1 << 20, w=2 << 20, dy=3 << 20, dr=None, dx=4 << 20, dw=5 << 20, ws=6 << 20, size=None, B=1, N=4, C=64):
        size = lib.la_rms_norm_workspace_bytes(C) if size is None else size
        return lib.la_rms_norm_backward(r, w, dy, dr, dx, dw, B, N, C, EPS, 1, None, ws, size, None)

    assert lib.la_rms_norm_workspace_bytes(0) == 0 and lib.la_rms_norm_workspace_bytes(16385) == 0
    assert back(ws=None) == 3 and back(size=512) == 3 and back(ws=(6 << 20) + 16) == 3
    assert back(dw=None) == 1 and back(dw=2 << 20) == 1 and back(dx=(1 << 20) + 128) == 1 and back(dw=4 << 20) == 1
    assert back(dx=6 << 20) == 1 and back(r=None) == 1 and back(dy=None) == 1


def test_binding_refuses():
    from bwd_la_fwd_gb300 import la
    x, w = torch.empty(4, 64, dtype=torch.bfloat16), torch.empty(64)
    with pytest.raises(ValueError, match="weight"):
        la.la_rms_norm(x, w.double())
    with pytest.raises(ValueError, match="CUDA"):
        la.la_rms_norm(x, w)
    with pytest.raises(ValueError, match="residual"):
        la.la_rms_norm(x, w, sum=x)
    with pytest.raises(ValueError):
        la.la_rms_norm(x, w, residual=x.float())
    with pytest.raises(ValueError, match="contiguous"):
        la.la_rms_norm(torch.empty(64, 4, dtype=torch.bfloat16).t(), w)
    with pytest.raises(ValueError, match="group"):
        la.la_rms_norm_8bit(x, w, group=32)
    with pytest.raises(ValueError, match="scales"):
        la.la_rms_norm_8bit(x, w, scales=torch.empty(4))
    with pytest.raises(TypeError):
        la.la_rms_norm(x.half(), w)
    with pytest.raises(ValueError):
        la.la_rms_norm(torch.empty(64), w)


# --------------------------------------------------------------------------------------------------- on the GPU

# channels on both sides of each kernel shape's width, rows around a block's; the widest rows
SHAPES = [(1, 1, 8), (2, 5, 64), (1, 33, 200), (1, 9, 256), (3, 7, 264), (1, 17, 520), (2, 9, 1032), (1, 5, 2048), (1, 70, 2056),
          (1, 3, 4104), (1, 3, 8200), (1, 2, 16384)]


def _case(B, N, C, kind, seed):
    gen = torch.Generator().manual_seed(seed)
    x, res = normal(gen, B, N, C, kind=kind), normal(gen, B, N, C, scale=3.0, kind=kind)
    return gen, x, res, 1 + 0.2 * torch.randn(C, generator=gen)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("B,N,C", SHAPES)
def test_norm(B, N, C, kind):
    from bwd_la_fwd_gb300 import la
    _, x, res, w = _case(B, N, C, kind, N + C)
    for residual in (None, res):
        (r, y), (er, ey) = R.norm(x, residual, w, EPS)
        Y, got = la.la_rms_norm(x.cuda(), w.cuda(), residual=None if residual is None else residual.cuda(), eps=EPS)
        R.assert_within("y", Y, y, R.rounded(y, ey, kind))
        R.assert_within("r", got, r, R.rounded(r, er, kind))


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("B,N,C", SHAPES)
def test_norm_in_8_bits(B, N, C, group, kind):
    """y8 scale is y within half a step of e4m3, 2^-4 of it (2^-10 of the scale where it is subnormal), and y's bound twice
    (in y and in the scale)."""
    from bwd_la_fwd_gb300 import la
    _, x, res, w = _case(B, N, C, kind, N + C + 1)
    (r, y), (er, ey) = R.norm(x, res, w, EPS)
    Y8, scales, got = la.la_rms_norm_8bit(x.cuda(), w.cuda(), residual=res.cuda(), group=group, eps=EPS)
    G = group or C
    parts = y.split(G, -1)
    want = torch.stack([p.abs().amax(-1) for p in parts], -1) / 448
    assert Y8.dtype == torch.float8_e4m3fn and scales.shape == want.shape
    R.assert_within("scales", scales, want, want * (ey / y.abs().clamp_min(1e-30)).max() + 4 * R.U * want)
    wide = scales.double().cpu().repeat_interleave(G, -1)[..., :C]
    # the value 448 stands at the largest; nothing saturates beyond the rounding of y / s
    R.assert_within("y8", Y8.float().double().cpu() * wide, y, 2.0 ** -4 * y.abs() * (1 + 2.0 ** -10) + 2.0 ** -10 * wide + 2 * ey)
    R.assert_within("r", got, r, R.rounded(r, er, kind))


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("B,N,C", SHAPES + [(2, 3000, 136)])
def test_norm_backward(B, N, C, kind):
    from bwd_la_fwd_gb300 import la
    gen, r, dr, w = _case(B, N, C, kind, N + C + 2)
    dy = normal(gen, B, N, C, kind=kind)
    for other in (None, dr):
        (dx, dw), (ex, ew) = R.norm_backward(r, w, dy, other, EPS)
        dX, dW = la.la_rms_norm_backward(r.cuda(), w.cuda(), dy.cuda(), dR=None if other is None else other.cuda(), eps=EPS)
        R.assert_within("dX", dX, dx, R.rounded(dx, ex, kind))
        R.assert_within("dw", dW, dw, ew)


@pytest.mark.gpu
def test_gradients_against_differences():
    """fp32 gradients along random directions against central differences of the 64-bit forward."""
    from bwd_la_fwd_gb300 import la
    gen, r, _, w = _case(2, 50, 72, "f32", 3)
    dy = torch.randn(2, 50, 72, generator=gen)
    got = la.la_rms_norm_backward(r.cuda(), w.cuda(), dy.cuda(), eps=EPS)
    _, tols = R.norm_backward(r, w, dy, None, EPS)
    for k, t in enumerate((r, w)):
        d = torch.randn(t.shape, generator=gen, dtype=torch.float64)
        ends = []
        for s in (1e-6, -1e-6):
            args = [u.double() for u in (r, w)]
            args[k] = args[k] + s * d
            ends.append(float((R.norm(args[0], None, args[1], EPS)[0][1] * dy.double()).sum()))
        want, have = (ends[0] - ends[1]) / 2e-6, float((got[k].double().cpu() * d).sum())
        size = float((d.abs() * (tols[k] + 2 * R.U * got[k].double().cpu().abs())).sum())
        assert abs(have - want) <= size + 1e-6 * (1 + abs(want))


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_strided_views_odd_channels_and_in_place(kind):
    """Slices of wider rows with channels that are no whole vector equal the packed call; in place too; nothing around them is
    written."""
    from bwd_la_fwd_gb300 import la
    B, N, C, wide = 2, 7, 203, 480
    gen = torch.Generator().manual_seed(5)
    x, res = (normal(gen, B, N, wide, kind=kind).cuda() for _ in range(2))
    w = torch.randn(C, generator=gen).cuda()
    xs, rs = x[:, :, 16:16 + C], res[:, :, 240:240 + C]
    (r, y), (er, ey) = R.norm(xs.cpu(), rs.cpu(), w.cpu(), EPS)
    out = torch.full((B, N, wide), 7.0, dtype=x.dtype, device="cuda")
    keep, keep_res = x.clone(), res.clone()
    Y, S = la.la_rms_norm(xs, w, residual=rs, eps=EPS, Y=out[:, :, 32:32 + C], sum=rs)
    R.assert_within("y", Y, y, R.rounded(y, ey, kind))
    R.assert_within("r", res[:, :, 240:240 + C], r, R.rounded(r, er, kind))
    assert torch.equal(x, keep) and torch.equal(res[:, :, :240], keep_res[:, :, :240]) and torch.equal(res[:, :, 240 + C:], keep_res[:, :, 240 + C:])
    assert (out[:, :, :32] == 7).all() and (out[:, :, 32 + C:] == 7).all()
    sums = torch.empty_like(out)[:, :, :C]  # (contiguous rows of 203 channels are no whole vectors apart)
    a, sa, _ = la.la_rms_norm_8bit(xs, w, residual=keep_res[:, :, 240:240 + C], eps=EPS, sum=sums)
    b, sb, _ = la.la_rms_norm_8bit(xs[1], w, residual=keep_res[1, :, 240:240 + C], eps=EPS, sum=sums[0])
    with pytest.raises(la.LAError):
        la.la_rms_norm_8bit(xs, w, residual=keep_res[:, :, 240:240 + C], eps=EPS)
    assert torch.equal(a[1].view(torch.uint8), b.view(torch.uint8)) and torch.equal(sa[1], sb)
    assert S.data_ptr() == rs.data_ptr()
    la.la_rms_norm(xs, w, eps=EPS, Y=xs)
    (_, y), (_, ey) = R.norm(keep[:, :, 16:16 + C].cpu(), None, w.cpu(), EPS)
    R.assert_within("in place", xs, y, R.rounded(y, ey, kind))
    # the gradient into one of its inputs
    r0, dy = normal(gen, N, 96, kind=kind).cuda(), normal(gen, N, 96, kind=kind).cuda()
    want = la.la_rms_norm_backward(r0, w[:96].contiguous(), dy, dR=r0, eps=EPS)
    have = la.la_rms_norm_backward(r0, w[:96].contiguous(), dy, dR=r0, eps=EPS, dX=dy)
    assert torch.equal(want[0], have[0]) and torch.equal(want[1], have[1]) and torch.equal(dy, want[0])


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_batches_with_rows_between_them(kind):
    """Entries whose rows do not follow one another evenly: as the packed call on copies, forward and backward."""
    from bwd_la_fwd_gb300 import la
    gen = torch.Generator().manual_seed(8)
    big = [normal(gen, 3, 12, 72, kind=kind).cuda() for _ in range(3)]
    w = torch.randn(72, generator=gen).cuda()
    x, res, dy = (t[:, 1:11] for t in big)
    a = la.la_rms_norm(x, w, residual=res)
    b = la.la_rms_norm(x.contiguous(), w, residual=res.contiguous())
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    a, b = la.la_rms_norm_8bit(x, w), la.la_rms_norm_8bit(x.contiguous(), w)
    assert torch.equal(a[0].view(torch.uint8), b[0].view(torch.uint8)) and torch.equal(a[1], b[1])
    a, b = la.la_rms_norm_backward(x, w, dy, dR=res), la.la_rms_norm_backward(x.contiguous(), w, dy.contiguous(), dR=res.contiguous())
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    one = la.la_rms_norm(big[0][:, 5:6], w)[0]  # a row from each entry
    assert torch.equal(one, la.la_rms_norm(big[0], w)[0][:, 5:6])


@pytest.mark.gpu
def test_rows_of_zeros_infinities_and_nan():
    """A zero row stays zero (eps > 0), its scale the least; a row with an infinity or NaN spoils itself alone."""
    from bwd_la_fwd_gb300 import la
    for kind in ("bf16", "f32"):
        gen = torch.Generator().manual_seed(6)
        x = normal(gen, 40, 256, kind=kind)
        x[3] = 0
        clean = x.clone()
        x[5, 7], x[11, 200] = math.inf, math.nan
        w = torch.ones(256).cuda()
        Y, _ = la.la_rms_norm(x.cuda(), w)
        Z, _ = la.la_rms_norm(clean.cuda(), w)
        rest = [i for i in range(40) if i not in (5, 11)]
        assert torch.equal(Y[rest], Z[rest]) and not Y[3].any() and torch.isnan(Y[5, 7]) and torch.isnan(Y[11]).all()
        for group in (0, 128):
            a, s, _ = la.la_rms_norm_8bit(x.cuda(), w, group=group)
            b, t, _ = la.la_rms_norm_8bit(clean.cuda(), w, group=group)
            assert torch.equal(a[rest].view(torch.uint8), b[rest].view(torch.uint8)) and torch.equal(s[rest], t[rest])
            assert not a[3].float().any() and torch.isfinite(s[3]).all() and torch.isnan(a[11].float()).all()
            assert torch.isnan(a[5, :128].float()).all()


@pytest.mark.gpu
def test_no_rows():
    from bwd_la_fwd_gb300 import la
    x, w = torch.empty(0, 64, device="cuda"), torch.ones(64, device="cuda")
    assert la.la_rms_norm(x, w)[0].shape == (0, 64)
    assert la.la_rms_norm_8bit(x, w)[0].shape == (0, 64)
    _, dw = la.la_rms_norm_backward(x, w, x, dweight=torch.ones(64, device="cuda"))
    assert not dw.any()


@pytest.mark.gpu
def test_gradients_are_the_same_bits_and_captured():
    """The weight's gradient does not change from run to run, nor in a captured graph on another stream."""
    from bwd_la_fwd_gb300 import la
    gen, r, dr, w = _case(1, 5000, 512, "bf16", 7)
    r, dr, w = r.cuda(), dr.cuda(), w.cuda()
    ws = la.new_rms_norm_workspace(512)
    first = la.la_rms_norm_backward(r, w, dr, workspace=ws)
    for _ in range(3):
        again = la.la_rms_norm_backward(r, w, dr, workspace=ws)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    out = torch.empty_like(r), torch.empty_like(w)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        la.la_rms_norm_backward(r, w, dr, dX=out[0], dweight=out[1], workspace=ws)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[0], first[0]) and torch.equal(out[1], first[1])
