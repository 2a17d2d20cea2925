"""What the vocabulary loss has to keep that a comparison at ordinary sizes and weights does not show."""

import pytest
import torch

from bit_quantized_lora_03_b200 import binding as B

from block_util import U16, U32, assert_within
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


@pytest.mark.parametrize("t", [24, 300])
@pytest.mark.parametrize("dloss", [1.0, 1e-12, 1e-20, 1e-30])
def test_small_upstream_gradients_of_large_losses(t, dloss):
    """A loss of 50 to 59, and one of 60 to 64 whose largest logit is 59 above the target's: dloss.exp(-loss)
    underflows, the gradient dloss.(p - [target]).W does not."""
    h, v = 16, 512
    W = torch.zeros(v, h)
    W[:, 1:] = torch.linspace(-1, 1, v)[:, None] * torch.linspace(0.5, 1.5, h - 1)
    W[:, 0] = 0
    W[0, 0] = 1.0       # one word high above the others (even rows)
    W = W.bfloat16()
    X = torch.zeros(t, h)
    X[0::2, 0] = torch.linspace(50, 58.5, (t + 1) // 2)
    X[1::2, 1] = -118.0     # word 0 at 59, word v - 1 at -59: targets near the middle (odd rows)
    X = X.bfloat16()
    y = torch.full((t,), v - 1)
    z = X.double() @ W.double().T
    rows = torch.arange(t)
    y[1::2] = ((z[1::2].amax(1, keepdim=True) - z[1::2] - 59).abs()).argmin(1)
    assert (z.amax(1) - z[rows, y] <= 60).all()     # one product of the logits serves
    lse = torch.logsumexp(z, 1)
    assert (lse - z[rows, y] >= 49).all()
    p = (z - lse[:, None]).exp()
    hot = torch.zeros_like(z)
    hot[rows, y] = 1
    want = dloss * (p - hot) @ W.double()
    d = torch.full((t,), dloss, device="cuda")
    _, _, dX = B.qlora_vocab_loss_fwd_bwd(X.cuda(), W.cuda(), y.cuda(), d)
    # p's exponentials are rounded to bf16, and the logits (h exact products of magnitudes up to 160) move them by
    # 2^-24 of those each
    e = dloss * (p + hot) @ W.double().abs() * (U16 + (h + 8) * 2 * U32 * 160)
    assert_within(dX, want, U16 * (want.abs() + e) + e, "dX")
    assert B.last_status() == 0
