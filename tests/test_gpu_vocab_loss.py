"""The vocabulary loss and its gradient against 64 bits: one token to several runs of the workspace,
vocabularies of one word to more than a run's worth, hidden widths that end inside a K-step, targets
at both ends, repeated and not counted, and logits that are not finite."""

import pytest
import torch

from bit_quantized_lora_03_b200 import binding as B

from block_util import U16, U32, assert_within, randn
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


SHAPES = [(1, 64, 1), (1, 64, 300), (3, 8, 257), (17, 72, 64), (16, 2048, 1500), (255, 128, 1000), (256, 64, 256),
          (257, 136, 513), (100, 136, 5003), (128, 64, 513), (129, 264, 1025), (48, 4096, 777), (300, 320, 2049), (1000, 64, 5000), (33, 1024, 33001), (2500, 512, 700),
          (600, 64, 262147)]


def _inputs(t, h, v, seed, sigma=3.0):
    X, W = randn((t, h), 1.0, seed).cuda(), randn((v, h), sigma / h ** 0.5, seed + 1).cuda()
    g = torch.Generator("cpu")
    g.manual_seed(seed + 2)
    y = torch.randint(0, v, (t,), generator=g)
    y[0] = v - 1
    if t > 2:
        y[1], y[2] = 0, -100
    y[5::7] = -100
    y[6::7] = v // 2
    return X, W, y.cuda()


def _reference(X, W, y, dloss=None, dlse=None, ignore=-100):
    """(loss, lse, dX, and the magnitudes the bounds need) in 64 bits, by rows to bound the memory."""
    x, w = X.double(), W.double()
    out = [[] for _ in range(6)]
    for j in torch.arange(X.shape[0], device="cuda").split(256):
        z = x[j] @ w.T
        el = (X.shape[1] + 64) * 2 * U32 * (x[j].abs() @ w.abs().T)   # sums of h exact products
        lse = torch.logsumexp(z, 1)
        hot = torch.zeros_like(z)
        n = y[j] != ignore
        hot[n, y[j][n]] = 1
        loss = torch.where(n, lse - (z * hot).sum(1), 0)
        p = (z - lse[:, None]).exp()
        # the mean error of the logits under the softmax, a few units of exp, log and of the maximum
        e_lse = (p * el).sum(1) + 16 * U32 * (1 + z.abs().amax(1) + lse.abs())
        for o, val in zip(out, (loss, lse, e_lse, e_lse + (el * hot).sum(1))):
            o.append(val)
        if dloss is not None:
            b = torch.where(n, dloss[j].double(), 0)
            a = b + (dlse[j].double() if dlse is not None else 0)
            g = a[:, None] * p - b[:, None] * hot
            eg = (a.abs()[:, None] * p) * (el + e_lse[:, None] + 16 * U32 * (1 + z.abs()))
            out[4].append(g @ w)
            # g is rounded to bf16 once, and before that its exponential once in the one-call form
            out[5].append((eg * 1.01 + U16 * 1.01 * (g.abs() + (a.abs()[:, None] * p) * (1 - hot))) @ w.abs())
    return [torch.cat(o) if o else None for o in out]


def _check_forward(loss, lse, ref):
    assert_within(lse, ref[1], ref[2] + U32 * ref[1].abs(), "lse")
    assert_within(loss, ref[0], ref[3] + U32 * ref[0].abs(), "loss")


def _check_gradient(dX, ref, h, v):
    e = ref[5] + 2 * v * U32 * ref[5]      # and sums of v products
    assert_within(dX, ref[4], U16 * (ref[4].abs() + e) + e, "dX")


@pytest.mark.parametrize("t,h,v", SHAPES)
def test_forward_backward_and_both_at_once(t, h, v):
    X, W, y = _inputs(t, h, v, t + v)
    g = torch.Generator("cpu")
    g.manual_seed(9)
    dloss = (torch.rand(t, generator=g) / t).cuda()
    dlse = (torch.randn(t, generator=g) / t).cuda()
    ref = _reference(X, W, y, dloss)
    loss, lse = B.qlora_vocab_loss_fwd(X, W, y)
    _check_forward(loss, lse, ref)
    assert not loss[y == -100].any()
    loss2, lse2, dX = B.qlora_vocab_loss_fwd_bwd(X, W, y, dloss)
    _check_forward(loss2, lse2, ref)
    _check_gradient(dX, ref, h, v)
    assert not dX[y == -100].any()
    _check_gradient(B.qlora_vocab_loss_bwd(X, W, y, lse, dloss), ref, h, v)
    ref = _reference(X, W, y, dloss, dlse)
    _check_gradient(B.qlora_vocab_loss_bwd(X, W, y, lse, dloss, dlse=dlse), ref, h, v)
    assert B.last_status() == 0


@pytest.mark.parametrize("t,v,rows", [(3, 1 << 24, [0, 1, 2]), (260, 1 << 24, [0, 3, 255, 256, 259]),
                                      (4100, 1 << 20, [0, 4095, 4096, 4099])])
def test_long_vocabularies(t, v, rows):
    """The largest vocabulary (g and the statistics pass 2^32 bytes, t x v passes 2^32), and the loss
    alone in more than one run. Some rows are compared. A row's sum of exponentials goes through 64
    additions in a piece of 128 and at most 512 + 8 of pieces in a lane, and 13 joins: 600 roundings."""
    h = 8
    X, W, y = _inputs(t, h, v, 11)
    if t > 3:
        y[3] = 5
    dloss = torch.full((t,), 1.0 / t, device="cuda")
    at = torch.tensor(rows, device="cuda")
    ref = _reference(X[at], W, y[at], dloss[at])
    ref[2], ref[3] = ref[2] + 600 * U32, ref[3] + 600 * U32
    ref[5] = ref[5] + 600 * U32 * (dloss[at].double()[:, None] * W.double().abs().amax(0))
    loss, lse = B.qlora_vocab_loss_fwd(X, W, y)
    _check_forward(loss[at], lse[at], ref)
    loss2, lse2, dX = B.qlora_vocab_loss_fwd_bwd(X, W, y, dloss)
    _check_forward(loss2[at], lse2[at], ref)
    _check_gradient(dX[at], ref, h, v)
    _check_gradient(B.qlora_vocab_loss_bwd(X, W, y, lse, dloss)[at], ref, h, v)
    assert B.last_status() == 0


@pytest.mark.parametrize("t", [20, 300])
@pytest.mark.parametrize("lean", [0.0, 1.0])
def test_logits_are_summed_in_pieces(t, lean):
    """One word, so that lse is its logit, over 8192 inputs that all add up (lean 1) or cancel. The
    tensor core truncates its sum every 16 inputs, and the kernels sum at most 1024 inputs there: 64
    truncations of 2^-23 of the magnitudes at most, 16 more for the products of one step, and a few
    for adding the pieces. Summed in one piece it would be 512 truncations (measured 2.7e-5)."""
    h = 8192
    W = randn((1, h), 1.0, 3).cuda()
    X = ((1 - lean) * randn((t, h), 1.0, 4).float().cuda() + lean * W.float()).bfloat16()
    y = torch.zeros(t, dtype=torch.int64, device="cuda")
    loss, lse = B.qlora_vocab_loss_fwd(X, W, y)
    want = (X.double() @ W.double().T)[:, 0]
    assert_within(lse, want, (64 + 16 + 10) * 2 * U32 * (X.double().abs() @ W.double().abs().T)[:, 0], "lse")
    assert not loss.any()


def test_reference_gradient_against_differences():
    t, h, v = 5, 16, 40
    X, W, y = randn((t, h), 1.0, 1).double(), randn((v, h), 0.7, 2).double(), torch.tensor([3, -100, 39, 0, 3])
    dloss, dlse = torch.rand(t).double(), torch.randn(t).double()

    def f(x):
        z = x @ W.T
        lse = torch.logsumexp(z, 1)
        n = y != -100
        loss = torch.where(n, lse - z.gather(1, torch.where(n, y, 0)[:, None])[:, 0], 0)
        return (loss * dloss + lse * dlse).sum()
    dX = _reference(X.cuda(), W.cuda(), y.cuda(), dloss.cuda(), dlse.cuda())[4].cpu()
    d = randn((t, h), 1.0, 5).double()
    diff = (f(X + 1e-5 * d) - f(X - 1e-5 * d)) / 2e-5
    assert abs(diff - (dX * d).sum()) <= 1e-7 * (1 + abs(diff))


def test_confident_tokens_keep_their_small_gradient():
    """p at the target within 2^-10 of one: g there is p - 1, formed in fp32 and not from two bf16
    values, so it keeps its sign and size."""
    t, h, v = 64, 64, 512
    W = torch.zeros(v, h)
    W[:h] = torch.eye(h) * 8
    W[h:, 0] = -1
    y = torch.arange(t) % h
    X = torch.zeros(t, h)
    X[torch.arange(t), y] = 1.75
    X, W, y = X.bfloat16().cuda(), W.bfloat16().cuda(), y.cuda()
    dloss = torch.ones(t, device="cuda")
    ref = _reference(X, W, y, dloss)
    assert ((ref[0] > 0) & (ref[0] < 2.0 ** -10)).all()
    loss, lse, dX = B.qlora_vocab_loss_fwd_bwd(X, W, y, dloss)
    _check_forward(loss, lse, ref)
    for got in (dX, B.qlora_vocab_loss_bwd(X, W, y, lse, dloss)):
        _check_gradient(got, ref, h, v)
        at = got[torch.arange(t), y].double()
        # 8 (p - 1): bf16 twice, and p - 1 from exp(-loss) to a few 2^-24 of one
        want = ref[4][torch.arange(t), y]
        assert_within(at, want, 2.1 * U16 * want.abs() + 64 * U32 * (1 + lse.double().abs()), "8 (p - 1)")


@pytest.mark.parametrize("t", [9, 70, 300])
@pytest.mark.parametrize("scale", [1e-3, 30.0, 1000.0])
def test_flat_and_steep_logits(scale, t):
    """At 1000 some losses are far above 60: the one-call form computes such a run again."""
    h, v = 128, 1111
    X, W, y = _inputs(t, h, v, 77, sigma=1.0)
    X = (X.float() * scale).bfloat16()
    dloss = torch.full((t,), 1.0, device="cuda")
    ref = _reference(X, W, y, dloss)
    loss, lse, dX = B.qlora_vocab_loss_fwd_bwd(X, W, y, dloss)
    _check_forward(loss, lse, ref)
    _check_gradient(dX, ref, h, v)
    _check_gradient(B.qlora_vocab_loss_bwd(X, W, y, lse, dloss), ref, h, v)


@pytest.mark.parametrize("t", [30, 300])
def test_rows_that_are_not_finite_stay_alone(t):
    h, v = 64, 700
    X, W, y = _inputs(t, h, v, 5)
    y[:] = torch.arange(t) % v
    y[7] = y[9] = -100
    clean = B.qlora_vocab_loss_fwd_bwd(X, W, y, torch.ones(t, device="cuda"))
    X[4, 3], X[7, 1], X[9, 0] = float("nan"), float("inf"), float("nan")
    loss, lse, dX = B.qlora_vocab_loss_fwd_bwd(X, W, y, torch.ones(t, device="cuda"))
    rows = torch.ones(t, dtype=torch.bool, device="cuda")
    rows[[4, 7, 9]] = False
    for a, b in zip(clean, (loss, lse, dX)):
        assert torch.equal(a[rows], b[rows])
    assert torch.isnan(loss[4]) and torch.isnan(lse[4]) and torch.isnan(dX[4]).all()
    # not counted: no loss and no gradient, whatever the row holds
    assert loss[7] == 0 and loss[9] == 0 and not dX[7].any() and not dX[9].any()


@pytest.mark.parametrize("t", [20, 200])
def test_words_at_minus_infinity_count_for_nothing(t):
    """A word whose logit is -inf (here for every token) leaves the other words' softmax as it is."""
    h, v = 64, 600
    X, W, y = _inputs(t, h, v, 6)
    X[:, 0] = 1.0
    y[:] = torch.arange(t)
    loss, lse = B.qlora_vocab_loss_fwd(X, W[:512].contiguous(), y)
    W[512:], W[512:, 0] = 0, float("-inf")
    full = B.qlora_vocab_loss_fwd(X, W, y)
    assert_within(full[0], loss.double(), 4 * U32 * (1 + lse.double().abs()), "loss")
    W[:] = W[599]
    loss, lse = B.qlora_vocab_loss_fwd(X, W, y)
    assert (lse == float("-inf")).all()      # as a sum of no exponentials has it


@pytest.mark.parametrize("t", [40, 400])
def test_targets_outside_the_vocabulary_are_reported_and_not_counted(t):
    X, W, y = _inputs(t, 64, 100, 8)
    y[:] = 5
    y[3], y[8] = 100, -7
    assert B.last_status() == 0
    loss, _ = B.qlora_vocab_loss_fwd(X, W, y)
    assert B.last_status() == B.QLORA_DEV_TARGET and loss[3] == 0 and loss[8] == 0
    _, _, dX = B.qlora_vocab_loss_fwd_bwd(X, W, y, torch.ones(t, device="cuda"))
    assert B.last_status() == B.QLORA_DEV_TARGET and not dX[3].any() and not dX[8].any()
    loss, _ = B.qlora_vocab_loss_fwd(X, W, torch.full_like(y, 3), ignore_index=3)
    assert B.last_status() == 0 and not loss.any()


@pytest.mark.parametrize("t", [50, 700])
def test_the_same_bits_on_every_run_and_on_two_streams_at_once(t):
    X, W, y = _inputs(t, 256, 3001, 4)
    d = torch.ones(t, device="cuda")
    a = B.qlora_vocab_loss_fwd_bwd(X, W, y, d)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = [B.qlora_vocab_loss_fwd_bwd(X, W, y, d, stream=s) for s in (s1, s2, s1, s2)]
    torch.cuda.synchronize()
    for g in got:
        for u, w in zip(a, g):
            assert torch.equal(u, w)
