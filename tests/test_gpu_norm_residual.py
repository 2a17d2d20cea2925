"""The norms around a block with its gate and residual scale, against 64 bits: lengths from one
token, rows of one warp, of a part of a CTA, odd multiples of 8 and the longest; gates for one,
some and all tokens; every optional input left out. The gradients are autograd's in 64 bits,
which are checked against differences in turn."""

import pytest
import torch

from bit_quantized_lora_03_b200 import binding as B

from block_util import U16, U32, assert_within, norm_fwd64, randn
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


SHAPES = [(1, 8), (5, 72), (33, 256), (40, 264), (1000, 512), (3, 520), (64, 1000), (301, 4096), (7, 8192),
          (150, 8200), (2, 16384), (160, 16384)]
PARTS = [  # y, w_post, rows per gate (0 none, -1 all tokens), w_pre
    (True, True, 0, True), (True, True, -1, True), (True, False, 3, True), (True, True, 1, False),
    (False, False, 0, True), (True, False, 0, False), (True, True, 5, True),
]


def _inputs(t, h, y, post, rows, pre, seed):
    d = lambda v: None if v is None else v.cuda()  # noqa: E731
    rows = t if rows < 0 else rows
    x = randn((t, h), 2.0, seed)
    yy = randn((t, h), 0.7, seed + 1) if y else None
    wo = (1 + randn((h,), 0.2, seed + 2)) if post else None
    wi = (1 + randn((h,), 0.2, seed + 3)) if pre else None
    g = randn((-(-t // rows), h), 0.6, seed + 4) if rows else None
    return d(x), d(yy), d(wo), d(g), d(wi), rows


@pytest.mark.parametrize("t,h", SHAPES)
@pytest.mark.parametrize("y,post,rows,pre", PARTS)
def test_forward(t, h, y, post, rows, pre):
    x, yy, wo, g, wi, rows = _inputs(t, h, y, post, rows, pre, 10 * t + h)
    scale, eps = 0.7, 1e-5
    xo, n, ro, ri = B.qlora_norm_residual_fwd(x, yy, w_post=wo, gate=g, w_pre=wi, scale=scale, eps=eps,
                                              rows_per_gate=rows or None)
    rx, rn, rro, rri = norm_fwd64(x, yy, wo, g, wi, scale, eps, rows)
    # a row's sum of squares: h positive terms, so rstd is off by h 2^-25 at most, and 8 roundings
    st = h * U32 / 2 + 8 * U32
    part = (rx - x.double()).abs()
    ex = (st + 8 * U32) * part + 2 * U32 * (x.double().abs() + part)
    assert_within(xo, rx, U16 * (rx.abs() + ex) + ex, "x'")
    if post:
        assert_within(ro, rro, st * rro, "rstd_post")
    if pre:
        # an error e of x' moves a row's rstd by sum |x'| e / sum x'^2 <= max e / mean |x'| of itself
        rel = st + 16 * U32 + ex.amax(1) / rx.abs().mean(1)
        assert_within(ri, rri, rel * rri, "rstd_pre")
        en = rri[:, None] * wi.double().abs() * ex + rel[:, None] * rn.abs()
        assert_within(n, rn, U16 * (rn.abs() + en) + en, "n")
    else:
        assert n is None and ri is None
    assert B.last_status() == 0


@pytest.mark.parametrize("t,h", SHAPES)
@pytest.mark.parametrize("y,post,rows,pre", PARTS)
def test_backward(t, h, y, post, rows, pre):
    x, yy, wo, g, wi, rows = _inputs(t, h, y, post, rows, pre, 20 * t + h)
    scale, eps = 0.7, 1e-5
    xo, n, ro, ri = B.qlora_norm_residual_fwd(x, yy, w_post=wo, gate=g, w_pre=wi, scale=scale, eps=eps,
                                              rows_per_gate=rows or None)
    if pre:     # the statistics of the x' that is passed, as the reference takes them
        ri = (xo.double().square().mean(1) + eps).rsqrt().float()
    dxo = randn((t, h), 0.5, 31).cuda()
    dn = randn((t, h), 0.5, 32).cuda() if pre else None
    dx, dy, dwo, dg, dwi = B.qlora_norm_residual_bwd(dxo, dn, xo, yy, ro, ri, w_post=wo, gate=g, w_pre=wi,
                                                     scale=scale, rows_per_gate=rows or None)
    # autograd in 64 bits, the second norm at the saved (rounded) x', as the call is given it
    leaf = lambda v: None if v is None else v.double().requires_grad_(True)  # noqa: E731
    ly, lo, lg, li = leaf(yy), leaf(wo), leaf(g), leaf(wi)
    lx = xo.double().requires_grad_(True)
    loss = (lx * dxo.double()).sum()
    if pre:
        _, ln, _, _ = norm_fwd64(lx, None, None, None, li, 1.0, eps, 0)
        loss = loss + (ln * dn.double()).sum()
    loss.backward()
    gx = lx.grad
    st = (h + 16) * U32      # sums of h terms and a few roundings, relative to the terms' magnitudes
    big, ex = dxo.double().abs(), 8 * U32 * dxo.double().abs()
    if pre:
        r = ri.double()[:, None]
        xh = (xo.double() * r).abs()
        dh = (dn.double() * wi.double()).abs()
        big = big + r * (dh + xh * (dh * xh).mean(1, keepdim=True))
        ex = 8 * U32 * big + st * r * xh * (dh * xh).mean(1, keepdim=True)
    assert_within(dx, gx, U16 * (gx.abs() + ex) + ex, "dx")
    terms = None
    if pre:
        terms = (dn.double() * xo.double() * ri.double()[:, None]).abs()
        assert_within(dwi, li.grad, terms.sum(0) * (t * U32 + st), "dw_pre")
    else:
        assert dwi is None
    if not y:
        assert dy is None and dwo is None and dg is None
        return
    out, _, _, _ = norm_fwd64(torch.zeros_like(lx), ly, lo, lg, None, scale, eps, rows)
    (out * gx).sum().backward()
    one = torch.ones((), dtype=torch.float64, device="cuda")
    gate = g.double()[torch.arange(t, device="cuda") // rows].abs() if rows else one
    wod = wo.double().abs() if post else one
    yh = (yy.double() * ro.double()[:, None]).abs() if post else yy.double().abs()
    rr = ro.double()[:, None] if post else one
    small = (16 + 0.5 * h) * U32
    du = scale * gate * gx.abs()
    edu = scale * gate * ex + small * du
    e = du * wod
    ee = edu * wod
    ey = rr * (ee + small * e)
    if post:
        k = scale * gate * wod * yh
        sums = (k * (gx.abs() + 2 * big)).mean(1, keepdim=True) * st + (k * ex).mean(1, keepdim=True)
        ey = ey + rr * yh * (sums + small * (e * yh).mean(1, keepdim=True))
        assert_within(dwo, lo.grad, ((edu + du * (t * U32 + small)) * yh).sum(0), "dw_post")
    else:
        assert dwo is None
    assert_within(dy, ly.grad, U16 * (ly.grad.abs() + ey) + ey, "dy")
    if rows:
        tg = scale * (ex + gx.abs() * (t * U32 + small)) * yh * wod
        idx = torch.arange(t, device="cuda") // rows
        assert_within(dg, lg.grad, torch.zeros_like(lg.grad).index_add_(0, idx, tg), "dgate")
    else:
        assert dg is None
    assert B.last_status() == 0


def test_reference_gradient_against_differences():
    """The 64-bit form's gradient is the derivative of the 64-bit form (central differences: error
    of order step^2 = 1e-10 times third derivatives of order 1)."""
    t, h, rows = 4, 16, 3
    x, y, wo, g, wi = (v.double() for v in (randn((t, h), 1.0, 1), randn((t, h), 1.0, 2), 1 + randn((h,), 0.2, 3),
                                            randn((2, h), 0.6, 4), 1 + randn((h,), 0.2, 5)))
    cx, cn = randn((t, h), 1.0, 6).double(), randn((t, h), 1.0, 7).double()

    def f(v):
        xo, n, _, _ = norm_fwd64(v[0], v[1], v[2], v[3], v[4], 0.7, 1e-5, rows)
        return (xo * cx + n * cn).sum()
    leaves = [v.clone().requires_grad_(True) for v in (x, y, wo, g, wi)]
    f(leaves).backward()
    for i, v in enumerate(leaves):
        d = randn(tuple(v.shape), 1.0, 60 + i).double()
        up, dn = list(leaves), list(leaves)
        up[i], dn[i] = v + 1e-5 * d, v - 1e-5 * d
        diff = (f(up) - f(dn)) / 2e-5
        assert abs(diff - (v.grad * d).sum()) <= 1e-6 * (1 + abs(diff))


def test_values_that_are_not_finite_stay_in_their_rows():
    t, h = 6, 1000
    x, y, wo, g, wi, rows = _inputs(t, h, True, True, -1, True, 5)
    x[2, 7], y[4, 3] = float("nan"), float("inf")
    xo, n, _, _ = B.qlora_norm_residual_fwd(x, y, w_post=wo, gate=g, w_pre=wi)
    clean = [0, 1, 3, 5]
    assert torch.isfinite(xo[clean]).all() and torch.isfinite(n[clean]).all()
    assert torch.isnan(n[2]).all() and torch.isnan(xo[4, 3])


def test_zero_rows_are_finite():
    x = torch.zeros(3, 4096, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(4096, dtype=torch.bfloat16, device="cuda")
    xo, n, ro, ri = B.qlora_norm_residual_fwd(x, x, w_post=w, w_pre=w, eps=1e-6)
    assert not xo.any() and not n.any()
    assert_within(ri, torch.full((3,), 1e3), torch.full((3,), 1.0), "rstd of zeros")   # 1 / sqrt(1e-6)


def test_same_bits_on_every_run_in_place_and_on_another_stream():
    t, h = 700, 4096
    x, y, wo, g, wi, rows = _inputs(t, h, True, True, 100, True, 9)
    dxo, dn = randn((t, h), 0.5, 1).cuda(), randn((t, h), 0.5, 2).cuda()

    def both(stream=None):
        f = B.qlora_norm_residual_fwd(x, y, w_post=wo, gate=g, w_pre=wi, rows_per_gate=100, stream=stream)
        b = B.qlora_norm_residual_bwd(dxo, dn, f[0], y, f[2], f[3], w_post=wo, gate=g, w_pre=wi,
                                      rows_per_gate=100, stream=stream)
        return [*f, *b]
    a = both()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    b, c = both(), both(side)
    torch.cuda.synchronize()
    for u, v, w in zip(a, b, c):
        assert torch.equal(u, v) and torch.equal(u, w)
    z = x.clone()
    B.qlora_norm_residual_fwd(z, y, w_post=wo, gate=g, w_pre=wi, rows_per_gate=100, x_out=z)
    assert torch.equal(z, a[0])
