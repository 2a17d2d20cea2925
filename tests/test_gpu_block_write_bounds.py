"""Guard bytes around every output and workspace of the operators around the linear, on shapes that
end inside tiles, shares, units and rows (as test_gpu_write_bounds does for the linear and codec)."""

import pytest
import torch

from bit_quantized_lora_03_b200 import binding as B
from bit_quantized_lora_03_b200 import inputs

from block_util import randn
from gpu_util import require_gpu
from test_gpu_write_bounds import Guarded

pytestmark = pytest.mark.gpu
bf16, f32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _stream():
    return torch.cuda.current_stream().cuda_stream


def _check(rc, **buffers):
    assert rc == 0 and B.last_status() == 0
    for name, g in buffers.items():
        g.check(name)


@pytest.mark.parametrize("t,h,o,r", [(3, 320, 576, 48), (13, 8192, 1088, 16), (23, 4096, 576, 16), (257, 192, 320, 80),
                                     (700, 1984, 192, 48)])
def test_linear_epilogue(t, h, o, r):
    li = inputs.random_linear(t, h, o, r, 0.5, seed=t, with_grad=False)
    p = B.nf4_quantize(li.Wt.cuda())
    Y, Z, sT = Guarded((t, o), bf16), Guarded((t, o), bf16), Guarded((t, r), bf16)
    ws = Guarded((int(B.lib().qlora_fwd_epilogue_workspace_bytes(t, h, o, r)),), torch.uint8)
    B.qlora_linear_fwd_epilogue(li.X.cuda(), p, li.L1.cuda(), li.L2.cuda(), 0.5, bias=randn((o,), 1.0, 1).cuda(),
                                act="silu", residual=randn((t, o), 1.0, 2).cuda(), Y=Y.t, Z=Z.t, sT=sT.t, ws=ws.t)
    _check(0, Y=Y, Z=Z, sT=sT, ws=ws)
    assert torch.isfinite(Y.t).all() and torch.isfinite(Z.t).all()


@pytest.mark.parametrize("t,o", [(1, 8), (70, 264), (1001, 1000)])
def test_epilogue_backward(t, o):
    dZ, db = Guarded((t, o), bf16), Guarded((o,), f32)
    ws = Guarded((int(B.lib().qlora_epilogue_bwd_workspace_bytes(t, o)),), torch.uint8)
    B.qlora_epilogue_bwd(randn((t, o), 1.0, 1).cuda(), randn((t, o), 1.0, 2).cuda(), "gelu", dZ=dZ.t, dbias=db.t, ws=ws.t)
    _check(0, dZ=dZ, db=db, ws=ws)


@pytest.mark.parametrize("t,h,rows", [(1, 8, 1), (9, 72, 2), (300, 520, 7), (31, 8192, 31), (299, 1000, 64),
                                      (5, 16384, 3), (160, 8200, 160)])
def test_norms(t, h, rows):
    x, y, dxo, dn = (randn((t, h), 1.0, i).cuda() for i in range(4))
    wo, wi, g = randn((h,), 1.0, 5).cuda(), randn((h,), 1.0, 6).cuda(), randn((-(-t // rows), h), 1.0, 7).cuda()
    xo, n, ro, ri = Guarded((t, h), bf16), Guarded((t, h), bf16), Guarded((t,), f32), Guarded((t,), f32)
    L = B.lib()
    a = lambda v: (v.t if isinstance(v, Guarded) else v).data_ptr()  # noqa: E731
    _check(L.qlora_norm_residual_fwd(a(x), a(y), t, h, a(wo), a(g), rows, 0.7, a(wi), 1e-6, a(xo), a(n), a(ro), a(ri),
                                     _stream()), xo=xo, n=n, ro=ro, ri=ri)
    dx, dy = Guarded((t, h), bf16), Guarded((t, h), bf16)
    dwo, dg, dwi = Guarded((h,), f32), Guarded(tuple(g.shape), f32), Guarded((h,), f32)
    ws = Guarded((int(L.qlora_norm_residual_bwd_workspace_bytes(t, h)),), torch.uint8)
    _check(L.qlora_norm_residual_bwd(a(dxo), a(dn), a(xo), a(y), t, h, a(wo), a(g), rows, 0.7, a(wi), a(ro), a(ri),
                                     a(dx), a(dy), a(dwo), a(dg), a(dwi), a(ws), ws.t.numel(), _stream()),
           dx=dx, dy=dy, dwo=dwo, dg=dg, dwi=dwi, ws=ws)
    for v in (xo, n, dx, dy, dwo, dg, dwi):     # every element was written
        assert torch.isfinite(v.t).all() and (v.t != torch.tensor(0).to(v.t)).any()


@pytest.mark.parametrize("t,h,v", [(1, 8, 1), (5, 72, 1000), (79, 200, 333), (81, 200, 333), (300, 136, 2049),
                                   (600, 64, 262147)])
def test_vocabulary_loss(t, h, v):
    X, W = randn((t, h), 1.0, 1).cuda(), randn((v, h), 0.2, 2).cuda()
    y = (torch.arange(t) % v).cuda()
    d = torch.ones(t, device="cuda")
    L = B.lib()
    loss, lse, dX = Guarded((t,), f32), Guarded((t,), f32), Guarded((t, h), bf16)
    ws = Guarded((int(L.qlora_vocab_loss_fwd_workspace_bytes(t, h, v)),), torch.uint8)
    B.qlora_vocab_loss_fwd(X, W, y, loss=loss.t, lse=lse.t, ws=ws.t)
    _check(0, loss=loss, lse=lse, ws=ws)
    ws = Guarded((int(L.qlora_vocab_loss_bwd_workspace_bytes(t, h, v)),), torch.uint8)
    B.qlora_vocab_loss_bwd(X, W, y, lse.t, d, dX=dX.t, ws=ws.t)
    _check(0, dX=dX, ws=ws)
    ws = Guarded((int(L.qlora_vocab_loss_fwd_bwd_workspace_bytes(t, h, v)),), torch.uint8)
    B.qlora_vocab_loss_fwd_bwd(X, W, y, d, loss=loss.t, lse=lse.t, dX=dX.t, ws=ws.t)
    _check(0, loss=loss, lse=lse, dX=dX, ws=ws)
