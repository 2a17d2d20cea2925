"""What the vocabulary loss has to keep that a comparison at ordinary sizes and weights does not show."""

import pytest
import torch

from bit_quantized_lora_03_b200 import binding as B

from block_util import U16, U32, assert_within, randn
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


@pytest.mark.parametrize("t,h,v", [(300, 64, 1 << 22), (20, 2048, 1 << 21), (100, 4096, 1 << 20)])
def test_gradient_over_a_long_vocabulary_is_summed_in_pieces(t, h, v):
    """X = 0, so that p is 2^-k for every word, and the target's row of W is the mean of all rows in bf16:
    dX is what is left of the mean, and shows the sum's own error. The tensor core truncates its fp32 sum
    after every 16 words; at most 8192 words are summed there, 512 truncations of 2^-23 of the magnitudes
    and 16 more for the products of one step. The pieces' sums, v / 8192 of them, and up to 16 shares of a
    split sum are added in fp32, each to 2^-24 of the whole."""
    g = torch.Generator("cuda")
    g.manual_seed(v)
    W = torch.empty(v, h, dtype=torch.bfloat16, device="cuda")
    total = torch.zeros(h, dtype=torch.float64, device="cuda")
    step = (1 << 26) // h
    for i in range(0, v, step):
        W[i:i + step] = torch.rand(step, h, generator=g, device="cuda").bfloat16()
        total += W[i:i + step].double().sum(0)
    y = torch.full((t,), v // 3, device="cuda")
    total -= W[v // 3].double()
    W[v // 3] = (total / (v - 1)).bfloat16()
    total += W[v // 3].double()
    mean = total / v
    want = (mean - W[v // 3].double()).expand(t, h)
    X = torch.zeros(t, h, dtype=torch.bfloat16, device="cuda")
    d = torch.ones(t, device="cuda")
    loss, lse, dX = B.qlora_vocab_loss_fwd_bwd(X, W, y, d)
    back = B.qlora_vocab_loss_bwd(X, W, y, lse, d)
    # lse, and with it the row's factor, is off by a few units of fp32 and the 600 roundings of a row's sum
    # of exponentials (p from lse, 2^-k but for that, is 2^-k again in bf16)
    e = mean * ((512 + 16) * 2 + v / 8192 + 16 + 600 + 64) * U32
    for got, name in ((dX, "dX"), (back, "dX from lse")):
        assert_within(got, want, U16 * (want.abs() + e) + e, name)
    assert B.last_status() == 0


@pytest.mark.parametrize("word", [float("-inf"), float("nan")])
@pytest.mark.parametrize("t", [30, 300])
def test_rows_that_count_for_nothing_get_zero_whatever_the_words_hold(t, word):
    """Also in the gradient from lse, and in the one-call form where a loss above 60 has the run computed again."""
    h, v = 64, 700
    X, W = torch.ones(t, h), torch.zeros(v, h)
    W[7] = word
    y = torch.arange(t) % 500 + 20
    off = torch.arange(t) % 3 == 0
    y[off] = -100
    X, W, y, off = X.bfloat16().cuda(), W.bfloat16().cuda(), y.cuda(), off.cuda()
    d = torch.ones(t, device="cuda")
    W[9] = 2.0      # a word of logit 128: every loss is
    _, lse, dX = B.qlora_vocab_loss_fwd_bwd(X, W, y, d)
    assert not dX[off].any()
    assert not B.qlora_vocab_loss_bwd(X, W, y, lse, d)[off].any()
    e = torch.where(torch.arange(t, device="cuda") % 6 == 0, 0.0, 1.0)
    back = B.qlora_vocab_loss_bwd(X, W, y, lse, d, dlse=e)
    assert not back[::6].any()      # neither counted nor with a gradient of lse
    assert torch.isnan(back[3::6]).all()    # the formula's zero times -inf, or NaN


@pytest.mark.parametrize("t", [30, 300])
def test_gradients_of_loss_and_lse_that_cancel(t):
    """dlse = -dloss leaves a = 0 and b = dloss: dX is -b W[y], exactly."""
    h, v = 72, 700
    X, W, y = randn((t, h), 1.0, 1).cuda(), randn((v, h), 0.5, 2).cuda(), (torch.arange(t) % v).cuda()
    d = torch.full((t,), 0.25, device="cuda")
    _, lse = B.qlora_vocab_loss_fwd(X, W, y)
    assert torch.equal(B.qlora_vocab_loss_bwd(X, W, y, lse, d, dlse=-d), -0.25 * W[y])
