"""The norms with gradients or outputs left out: each gives what the full call gives with zeros in their
place, in every kernel (rows of a warp, of a CTA that stays, with and without all operands, the longest)."""

import pytest
import torch

from bit_quantized_lora_03_b200 import binding as B

from block_util import randn
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu
SHAPES = [(1, 8), (9, 256), (3000, 264), (700, 4096), (40, 4104), (700, 1000), (20, 16384)]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _case(t, h):
    c = lambda shape, s, i: randn(shape, s, i).cuda()  # noqa: E731
    rows = max(1, t // 3)
    return (c((t, h), 2.0, 1), c((t, h), 0.7, 2), 1 + c((h,), 0.2, 3), c((-(-t // rows), h), 0.6, 4), 1 + c((h,), 0.2, 5),
            c((t, h), 0.5, 6), c((t, h), 0.5, 7), rows)


def _equal(got, want):
    for a, b in zip(got, want):
        assert (a is None) == (b is None)
        assert a is None or torch.equal(a, b)


@pytest.mark.parametrize("t,h", SHAPES)
def test_a_gradient_left_out_is_zero(t, h):
    x, y, wo, g, wi, dxo, dn, rows = _case(t, h)
    xo, _, ro, ri = B.qlora_norm_residual_fwd(x, y, w_post=wo, gate=g, w_pre=wi, rows_per_gate=rows)

    def bwd(d, e, **k):
        return B.qlora_norm_residual_bwd(d, e, xo, y, ro, ri, w_post=wo, gate=g, w_pre=wi, rows_per_gate=rows, **k)
    zero = torch.zeros_like(x)
    _equal(bwd(None, dn), bwd(zero, dn))
    got, want = bwd(dxo, None), bwd(dxo, zero)
    _equal(got, want)
    assert not got[4].any()
    # and x' and its statistics are then not needed
    _equal(B.qlora_norm_residual_bwd(dxo, None, None, y, ro, None, w_post=wo, gate=g, rows_per_gate=rows)[:4], want[:4])
    assert B.last_status() == 0


@pytest.mark.parametrize("t,h", SHAPES)
def test_an_output_left_out_changes_no_other(t, h):
    x, y, wo, g, wi, _, _, rows = _case(t, h)
    xo, n, ro, ri = B.qlora_norm_residual_fwd(x, y, w_post=wo, gate=g, w_pre=wi, rows_per_gate=rows)
    xo2, n2, none, none2 = B.qlora_norm_residual_fwd(x, y, w_post=wo, gate=g, w_pre=wi, rows_per_gate=rows, want_rstd=False)
    assert none is None and none2 is None and torch.equal(xo, xo2) and torch.equal(n, n2)
    only = torch.empty_like(x)
    a = lambda v: v.data_ptr()  # noqa: E731
    rc = B.lib().qlora_norm_residual_fwd(a(x), a(y), t, h, a(wo), a(g), rows, 1.0, a(wi), 1e-6, None, a(only), None, None,
                                         torch.cuda.current_stream().cuda_stream)
    assert rc == 0 and torch.equal(only, n)
    assert torch.equal(B.qlora_norm_residual_fwd(x, y, w_post=wo, gate=g, rows_per_gate=rows)[0], xo)
    # more tokens to a gate row than there are tokens: one row
    one = g[:1].contiguous()
    _equal(B.qlora_norm_residual_fwd(x, y, w_post=wo, gate=one, w_pre=wi, rows_per_gate=1 << 40),
           B.qlora_norm_residual_fwd(x, y, w_post=wo, gate=one, w_pre=wi))
    assert B.last_status() == 0
