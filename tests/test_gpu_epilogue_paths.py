"""Which kernels the linear with the fused epilogue runs for 9 to 16 tokens, and both against 64 bits: the
decode GEMV for wide weights of few inputs, the tcgen05 GEMM for small weights (but the smallest)."""

import pytest
import torch

from bit_quantized_lora_03_b200 import binding as B

import test_gpu_block_write_bounds as bounds
import test_gpu_epilogue as epilogue
from block_util import randn
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu
GEMV, GEMM = "nf4_gemv_kernel", "nf4_gemm_kernel<fwd>"


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _kernels(t, h, o, r):
    p = B.PackedNF4(o, h)
    p.codes.random_(0, 256)
    p.absmax_q8.random_(1, 256)
    p.absmax_s2.fill_(3e-4)
    args = (randn(s, 1.0, i).cuda() for i, s in enumerate(((t, h), (h, r), (r, o))))
    x, l1, l2 = args
    with B.KernelProfile() as prof:
        B.qlora_linear_fwd_epilogue(x, p, l1, l2, 0.5)
    return {k for k, n in prof.launches.items() if n}


@pytest.mark.parametrize("t,h,o,r,kernel", [
    (1, 4096, 1024, 64, GEMV), (8, 512, 512, 16, GEMV), (9, 4096, 1024, 64, GEMM), (16, 2048, 2048, 16, GEMM),
    (12, 512, 512, 16, GEMM), (12, 256, 512, 16, GEMV), (16, 512, 19008, 16, GEMV), (9, 4096, 11008, 16, GEMV), (17, 512, 19008, 16, GEMM)])
def test_path(t, h, o, r, kernel):
    assert kernel in _kernels(t, h, o, r)


@pytest.mark.parametrize("t,h,o,r,act,bias,residual,keep", [
    (9, 512, 19008, 16, "gelu", True, True, True), (16, 512, 19008, 16, "silu", True, False, False),
    (13, 512, 19008, 16, "none", False, True, False), (9, 576, 512, 16, "gelu_tanh", True, True, True),
    (16, 4096, 256, 64, "relu", True, True, True), (11, 192, 1088, 240, "silu", False, True, True)])
def test_forward(t, h, o, r, act, bias, residual, keep):
    if o > 1088:
        assert GEMV in _kernels(t, h, o, r)
    epilogue.test_forward(t, h, o, r, act, bias, residual, keep)


@pytest.mark.parametrize("t,h,o,r", [(13, 512, 19008, 16), (9, 576, 512, 16), (16, 4096, 320, 48)])
def test_write_bounds(t, h, o, r):
    bounds.test_linear_epilogue(t, h, o, r)
