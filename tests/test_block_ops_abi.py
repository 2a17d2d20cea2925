"""Refusals of the operators around the linear, on the host: nothing here launches anything, and
the addresses are never dereferenced."""

import ctypes

import pytest
import torch

from bit_quantized_lora_03_b200 import binding as B
from bit_quantized_lora_03_b200 import build as build_mod

P, BIG = 0x10000, 1 << 40
INVALID, SHAPE, ALIGN, WS = (B.QLORA_ERR_INVALID_ARG, B.QLORA_ERR_BAD_SHAPE, B.QLORA_ERR_MISALIGNED,
                             B.QLORA_ERR_WORKSPACE)


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return B.lib()


def test_linear_epilogue(lib):
    d = B.NF4WeightDesc(P, P, P, 128, 128)

    def f(X=P, t=4, r=16, s=1.0, bias=P, act=1, R=P, Y=P, Z=P, ws=P, n=BIG, w=d):
        return lib.qlora_linear_fwd_epilogue(X, t, ctypes.byref(w), P, P, r, s, bias, act, R, Y, Z, None, ws, n, None)
    assert f(act=-1) == f(act=5) == f(X=None) == f(t=0) == f(r=24) == f(s=float("inf")) == f(Y=None) == INVALID
    assert f(w=B.NF4WeightDesc(P, P, P, 100, 128)) == SHAPE
    assert f(bias=P + 2) == f(R=P + 8) == f(Z=P + 4) == f(X=P + 2) == ALIGN
    assert f(ws=None) == f(n=64) == WS
    # a few hundred tokens split K: their fp32 shares lie behind the plain forward's workspace
    assert lib.qlora_fwd_epilogue_workspace_bytes(4, 128, 128, 16) == lib.qlora_fwd_workspace_bytes(4, 128, 128, 16)
    assert lib.qlora_fwd_epilogue_workspace_bytes(64, 4096, 4096, 64) >= 2 * 64 * 4096 * 4
    assert lib.qlora_fwd_epilogue_workspace_bytes(64, 100, 128, 16) == 0


def test_epilogue_backward(lib):
    def f(dY=P, Z=P, t=4, o=128, act=2, dZ=P, db=P, ws=P, n=BIG):
        return lib.qlora_epilogue_bwd(dY, Z, t, o, act, dZ, db, ws, n, None)
    assert f(dY=None) == f(Z=None) == f(act=9) == f(t=0) == f(dZ=None, db=None) == INVALID
    assert f(o=0) == f(o=100) == f(t=1 << 31) == SHAPE
    assert f(dY=P + 2) == f(Z=P + 8) == f(dZ=P + 4) == f(db=P + 4) == f(ws=P + 8) == ALIGN
    assert f(ws=None) == f(n=16) == WS
    assert lib.qlora_epilogue_bwd_workspace_bytes(4, 100) == 0
    assert lib.qlora_epilogue_bwd_workspace_bytes(0, 128) == 0
    assert lib.qlora_epilogue_bwd_workspace_bytes(4096, 11008) >= 64 * 11008 * 4


def test_norm_forward(lib):
    def f(x=P, y=P, t=4, h=128, wo=P, g=P, rows=1, scale=1.0, wi=P, eps=1e-6, xo=P, n=P, ro=P, ri=P):
        return lib.qlora_norm_residual_fwd(x, y, t, h, wo, g, rows, scale, wi, eps, xo, n, ro, ri, None)
    assert f(x=None) == f(y=None) == f(y=None, g=None, ro=None) == f(n=None) == f(wi=None) == INVALID
    assert f(xo=None, n=None, wi=None, ri=None) == f(wo=None) == f(wi=None, n=None) == f(rows=0) == INVALID
    assert f(scale=float("nan")) == f(eps=-1.0) == f(eps=float("inf")) == f(t=0) == INVALID
    assert f(h=0) == f(h=12) == f(h=16392) == f(t=1 << 31) == SHAPE
    for k in ("x", "y", "wo", "g", "wi", "xo", "n"):
        assert f(**{k: P + 8}) == ALIGN, k
    assert f(ro=P + 2) == f(ri=P + 1) == ALIGN


def test_norm_backward(lib):
    def f(dxo=P, dn=P, xo=P, y=P, t=4, h=128, wo=P, g=P, rows=1, scale=1.0, wi=P, ro=P, ri=P, dx=P, dy=P,
          dwo=P, dg=P, dwi=P, ws=P, n=BIG):
        return lib.qlora_norm_residual_bwd(dxo, dn, xo, y, t, h, wo, g, rows, scale, wi, ro, ri, dx, dy, dwo, dg,
                                           dwi, ws, n, None)
    for k in ("dn", "xo", "y", "wo", "g", "wi", "ro", "ri", "dx", "dy", "dwo", "dg", "dwi"):
        assert f(**{k: None}) == INVALID, k
    assert f(dxo=None, dn=None, wi=None, dwi=None) == f(rows=0) == f(t=0) == f(scale=float("inf")) == INVALID
    assert f(h=20) == f(h=20000) == SHAPE
    for k in ("dxo", "dn", "xo", "y", "wo", "g", "wi", "dx", "dy", "dwo", "dg", "dwi", "ws"):
        assert f(**{k: P + 8}) == ALIGN, k
    assert f(ro=P + 2) == ALIGN
    assert f(ws=None) == f(n=64) == WS
    assert lib.qlora_norm_residual_bwd_workspace_bytes(4, 20000) == 0


def test_vocabulary_loss(lib):
    base = dict(X=P, W=P, t=4, h=64, v=100, y=P, ignore=-100)

    def fwd(loss=P, lse=P, ws=P, n=BIG, **k):
        return lib.qlora_vocab_loss_fwd(*{**base, **k}.values(), loss, lse, ws, n, None)

    def bwd(lse=P, dloss=P, dlse=P, dX=P, ws=P, n=BIG, **k):
        return lib.qlora_vocab_loss_bwd(*{**base, **k}.values(), lse, dloss, dlse, dX, ws, n, None)

    def both(dloss=P, loss=P, lse=P, dX=P, ws=P, n=BIG, **k):
        return lib.qlora_vocab_loss_fwd_bwd(*{**base, **k}.values(), dloss, loss, lse, dX, ws, n, None)
    for f in (fwd, bwd, both):
        for k in ("X", "W", "y", "lse"):
            assert f(**{k: None}) == INVALID, (f, k)
        assert f(t=0) == f(v=0) == INVALID
        assert f(h=0) == f(h=12) == f(t=1 << 31) == f(v=(1 << 24) + 1) == SHAPE
        for k in ("X", "W"):
            assert f(**{k: P + 8}) == ALIGN
        assert f(y=P + 4) == f(lse=P + 2) == f(ws=P + 8) == ALIGN
        assert f(ws=None) == f(n=8) == WS
    assert fwd(loss=None) == both(loss=None) == both(dloss=None) == bwd(dloss=None) == bwd(dX=None) == INVALID
    assert bwd(dX=P + 8) == bwd(dlse=P + 1) == both(loss=P + 2) == ALIGN
    for name in ("fwd", "bwd", "fwd_bwd"):
        f = getattr(lib, f"qlora_vocab_loss_{name}_workspace_bytes")
        assert f(4, 12, 100) == f(0, 64, 100) == f(4, 64, 0) == 0
    # the gradient's workspace is bounded whatever the batch: 256 MiB of factors, partial tiles, statistics
    bound = (256 << 20) + 160 * 256 * 256 * 4 + (8 << 20)
    assert lib.qlora_vocab_loss_fwd_bwd_workspace_bytes(1 << 20, 4096, 32000) <= bound
    assert lib.qlora_vocab_loss_bwd_workspace_bytes(1 << 20, 4096, 32000) <= bound


def test_vocabulary_loss_workspace_is_bounded(lib):
    """The loss alone holds 8 bytes per token and 128 words (or 32, for few tokens) of one run."""
    size = lib.qlora_vocab_loss_fwd_workspace_bytes
    assert size(1 << 20, 4096, 1 << 17) <= (256 << 20) + 4 * 4 * (1 << 18) + 4096
    assert size(1 << 30, 8, 1 << 24) <= (256 << 20) + 4 * 4 * 256 + 4096
    assert size(4096, 4096, 32000) >= 4096 * 250 * 8
    # 256 tokens where those need more than 256 MiB
    assert lib.qlora_vocab_loss_bwd_workspace_bytes(1 << 20, 8, 1 << 24) >= 256 * (1 << 24) * 2


def test_binding_refuses_host_tensors_shapes_and_unknown_activations():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    p = B.PackedNF4(64, 64, "cpu")
    for call in (lambda: B.qlora_linear_fwd_epilogue(x, p, x, x, 1.0), lambda: B.qlora_epilogue_bwd(x, x, "relu"),
                 lambda: B.qlora_norm_residual_fwd(x), lambda: B.qlora_norm_residual_bwd(x, None, x, None, None, None),
                 lambda: B.qlora_norm_residual_bwd(None, None, x, None, None, None),
                 lambda: B.qlora_norm_residual_fwd(x[0])):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(ValueError, match="unknown activation"):
        B._act_id("swish")
