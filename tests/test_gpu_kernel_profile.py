"""The kernel profile sees every launch of the operators around the linear, the ones that join or finish
another kernel's partial results among them."""

import pytest
import torch

from bit_quantized_lora_03_b200 import binding as B

from block_util import randn
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _launches(call):
    with B.KernelProfile() as prof:
        call()
    return {k: n for k, n in prof.launches.items() if n}


def _c(shape, seed, dtype=torch.bfloat16):
    return randn(shape, 1.0, seed, dtype).cuda()


def test_every_launch_is_recorded():
    t, h, o, r = 40, 4096, 512, 16
    p = B.nf4_quantize(_c((o, h), 1, torch.float32))
    x, l1, l2 = _c((t, h), 2), _c((h, r), 3), _c((r, o), 4)
    got = _launches(lambda: B.qlora_linear_fwd_epilogue(x, p, l1, l2, 0.5))       # K split over the card
    assert got == {"tc_gemm_kernel": 1, "nf4_gemm_kernel<fwd>": 1, "nf4_gemm_join_kernel": 1}
    d = _c((2000, o), 5)
    assert _launches(lambda: B.qlora_epilogue_bwd(d, d, "silu")) == {"epilogue_bwd_kernel": 2}
    assert _launches(lambda: B.qlora_epilogue_bwd(d, d, "silu", want_dbias=False)) == {"epilogue_bwd_kernel": 1}
    n = _c((64, 1024), 6)
    w, one = _c((1024,), 7), torch.ones(64, device="cuda")
    assert _launches(lambda: B.qlora_norm_residual_fwd(n, n, w_post=w, w_pre=w)) == {"norm_residual_kernels": 1}
    assert _launches(lambda: B.qlora_norm_residual_bwd(n, n, n, n, one, one, w_post=w, w_pre=w)) == {
        "norm_residual_kernels": 2}
    W = _c((3000, 256), 8)
    for t, joins in ((30, 1), (300, 1)):     # both forms split dX's sum
        X, y, d = _c((t, 256), 9), torch.zeros(t, dtype=torch.int64, device="cuda"), torch.ones(t, device="cuda")
        assert _launches(lambda: B.qlora_vocab_loss_fwd(X, W, y)) == {"vocab_gemm_kernel": 1, "vocab_row_kernels": 1}
        assert _launches(lambda: B.qlora_vocab_loss_fwd_bwd(X, W, y, d)) == {
            "vocab_gemm_kernel": 3, "vocab_row_kernels": 2 + joins}
        assert _launches(lambda: B.qlora_vocab_loss_bwd(X, W, y, d, d)) == {
            "vocab_gemm_kernel": 2, "vocab_row_kernels": joins}
