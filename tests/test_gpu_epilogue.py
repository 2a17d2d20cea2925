"""The linear with bias, activation and residual in its epilogue, and that epilogue's backward,
against 64 bits: both token paths (decode GEMV up to 16 tokens, tcgen05 GEMM above), ragged tokens,
outputs and ranks, every activation and every combination of the optional parts."""

import numpy as np
import pytest
import torch

from bit_quantized_lora_03_b200 import binding as B
from bit_quantized_lora_03_b200 import inputs
from oracle import nf4_oracle as O

from block_util import ACT, U16, U32, act_grad, assert_within, randn
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _linear64(li):
    """(Z without bias, error bound of the kernels' Z) in 64 bits from the oracle's weight."""
    W = torch.from_numpy(np.array(O.nf4_dequantize(O.nf4_quantize(li.Wt.numpy())))).double()
    W = W.t() if W.shape == (li.o, li.h) else W
    X, L1, L2 = li.X.double(), li.L1.double(), li.L2.double()
    sT = li.s * (X @ L1)
    Z = X @ W + sT @ L2
    # sT is rounded to bf16 (by contract); the accumulator adds h + r exact products, each addition
    # truncating at most 2^-23 of the magnitudes' sum
    mags = X.abs() @ W.abs() + sT.abs() @ L2.abs()
    est = U16 * sT.abs() + li.h * 2 * U32 * abs(li.s) * (X.abs() @ L1.abs())
    return Z, est @ L2.abs() + (li.h + li.r + 64) * 2 * U32 * mags


CASES = [  # t, h, o, r, act, bias, residual, Z kept
    (1, 320, 576, 16, "gelu_tanh", True, False, False), (3, 192, 64, 48, "silu", False, True, True),
    (9, 320, 576, 32, "none", True, True, False), (16, 1024, 96 * 2, 256, "gelu", True, True, True),
    (17, 320, 576, 48, "relu", True, True, True), (300, 320, 576, 48, "silu", True, False, True),
    (513, 640, 320, 80, "none", False, True, False), (257, 64, 64, 16, "gelu", True, True, False),
    (1030, 192, 832, 64, "gelu_tanh", False, False, True), (40, 128, 256, 16, "none", True, False, True),
    # K split over the card: one and two accumulators, shares of unequal length, two row tiles
    (23, 4096, 512, 64, "silu", True, True, True), (300, 2112, 320, 16, "gelu", True, True, False),
    (700, 1984, 192, 48, "none", False, True, True), (12, 8192, 4096, 32, "silu", True, True, True), (129, 11008, 256, 80, "relu", True, False, False),
    # a large weight for 9 to 16 tokens, K whole
    (9, 1024, 8256, 48, "gelu", True, True, True),
]


@pytest.mark.parametrize("t,h,o,r,act,bias,residual,keep", CASES)
def test_forward(t, h, o, r, act, bias, residual, keep):
    li = inputs.random_linear(t, h, o, r, 0.5, seed=t + h, with_grad=False)
    b = randn((o,), 0.5, 3) if bias else None
    R = randn((t, o), 2.0, 4) if residual else None
    p = B.nf4_quantize(li.Wt.cuda())
    c = lambda v: None if v is None else v.cuda()  # noqa: E731
    Y, Z, sT = B.qlora_linear_fwd_epilogue(c(li.X), p, c(li.L1), c(li.L2), li.s, bias=c(b), act=act,
                                           residual=c(R), want_Z=keep)
    assert B.last_status() == 0
    z, ez = _linear64(li)
    if bias:
        z, ez = z + b.double(), ez + U32 * (z.abs() + b.double().abs())
    y = ACT[act](z)
    ey = 1.13 * ez + 8 * U32 * (z.abs() + 1)       # |act'| <= 1.13; a few units in exp, erf, divide
    if residual:
        y = y + R.double()
        ey = ey + U32 * y.abs()
    assert_within(Y, y, U16 * (y.abs() + ey) + ey, "Y")
    if keep:
        assert_within(Z, z, U16 * (z.abs() + ez) + ez, "Z")
    else:
        assert Z is None
    if li.h * li.o < 1 << 23:       # the rank-r product is the plain forward's
        _, sT0 = B.qlora_linear_fwd(c(li.X), p, c(li.L1), c(li.L2), li.s)
        assert torch.equal(sT, sT0)
    else:                           # (up to the order of its fp32 sum: then half a step of bf16 either way)
        want = li.s * (li.X.double() @ li.L1.double())
        e = li.h * 2 * U32 * abs(li.s) * (li.X.double().abs() @ li.L1.double().abs())
        assert_within(sT, want, U16 * (want.abs() + e) + e, "sT")


@pytest.mark.parametrize("t", [5, 64])
def test_without_any_part_it_is_the_plain_linear(t):
    li = inputs.random_linear(t, 320, 576, 16, 1.0, seed=2, with_grad=False)
    p = B.nf4_quantize(li.Wt.cuda())
    X, L1, L2 = li.X.cuda(), li.L1.cuda(), li.L2.cuda()
    Y0, _ = B.qlora_linear_fwd(X, p, L1, L2, li.s)
    Y, Z, _ = B.qlora_linear_fwd_epilogue(X, p, L1, L2, li.s, want_Z=True)
    if t > 16:      # the decode sums' order may differ between calls
        assert torch.equal(Y, Y0)
    assert torch.equal(Y, Z)


def test_residual_in_place():
    li = inputs.random_linear(300, 320, 576, 16, 1.0, seed=3, with_grad=False)
    p = B.nf4_quantize(li.Wt.cuda())
    X, L1, L2 = li.X.cuda(), li.L1.cuda(), li.L2.cuda()
    R = randn((300, 576), 1.0, 8).cuda()
    Y, _, _ = B.qlora_linear_fwd_epilogue(X, p, L1, L2, li.s, act="silu", residual=R)
    S = R.clone()
    B.qlora_linear_fwd_epilogue(X, p, L1, L2, li.s, act="silu", residual=S, Y=S)
    assert torch.equal(Y, S)


@pytest.mark.parametrize("t,o", [(1, 8), (2, 264), (33, 4096), (64, 72), (65, 256), (1000, 1000), (4099, 328)])
@pytest.mark.parametrize("act", list(ACT))
def test_backward(t, o, act):
    dY, Z = randn((t, o), 1.0, t), randn((t, o), 1.5, o)
    Z[0, 0] = 0.0
    dZ, db = B.qlora_epilogue_bwd(dY.cuda(), Z.cuda() if act != "none" else None, act)
    want = dY.double() * act_grad(Z, act)
    # act' combines terms of magnitude up to |z| phi and 1, each off by a few units
    e = dY.double().abs() * (16 * U32 * (1 + Z.double().abs()))
    assert_within(dZ, want, U16 * (want.abs() + e) + e, "dZ")
    assert_within(db, want.sum(0), (e + want.abs() * t * U32).sum(0), "dbias")
    only, none = B.qlora_epilogue_bwd(dY.cuda(), Z.cuda(), act, want_dbias=False)
    assert none is None and torch.equal(only, dZ)
    none, again = B.qlora_epilogue_bwd(dY.cuda(), Z.cuda(), act, want_dZ=False)
    assert none is None and torch.equal(again, db)
    D = dY.cuda()
    B.qlora_epilogue_bwd(D, Z.cuda(), act, dZ=D)
    assert torch.equal(D, dZ)
    assert B.last_status() == 0


@pytest.mark.parametrize("act", list(ACT))
def test_activation_gradient_against_differences(act):
    """The kernels' act' is the slope of the kernels' own act: through a linear that is the identity
    on its bias (zero weights), Y = act(b); central differences of 64-bit act bound the middle."""
    z = torch.linspace(-6, 6, 512, dtype=torch.float64).to(torch.bfloat16)
    step = 1e-4
    slope = (ACT[act](z.double() + step) - ACT[act](z.double() - step)) / (2 * step)
    _, db = B.qlora_epilogue_bwd(torch.ones(1, 512, dtype=torch.bfloat16, device="cuda"), z[None].cuda(), act)
    # differences: third derivatives below 2 times step^2 / 6; the kink of relu lies off the grid
    assert_within(db, slope, torch.full_like(slope, 1e-8 + 16 * U32 * 7), "act'")


def test_large_pre_activations():
    z = torch.tensor([[-1e30, -500.0, -90.0, -40.0, 40.0, 90.0, 500.0, 1e30]], dtype=torch.bfloat16)
    for act in ("relu", "gelu", "gelu_tanh", "silu"):
        dZ, db = B.qlora_epilogue_bwd(torch.ones(1, 8, dtype=torch.bfloat16, device="cuda"), z.cuda(), act)
        want = torch.tensor([[0.0, 0, 0, 0, 1, 1, 1, 1]])
        assert_within(dZ, want, torch.full((1, 8), 1e-14), f"{act}'")   # 40 exp(-40) is 2e-16
