"""The operators against 64 bits at sizes where each kernel walks many rows, tiles or gate rows of its own:
CTAs that stay and prefetch, gate rows inside and across their runs, whole and split tiles of dX side by
side and several to a CTA pair. The comparisons and their bounds are those of the small sizes' tests."""

import pytest
import torch

from bit_quantized_lora_03_b200 import binding as B

import test_gpu_block_write_bounds as bounds
import test_gpu_norm_residual as norms
import test_gpu_vocab_loss as vocab
from block_util import U32, assert_within
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


# t, h, w_post, rows per gate (0: no gate), w_pre
NORMS = [
    (700, 4096, True, 100, True), (700, 4096, False, 1, True), (700, 4096, True, 0, False), (650, 4096, True, 700, True),
    (2500, 4096, True, 5, True), (2500, 4096, True, 700, True), (2500, 4104, True, 33, True), (330, 8192, True, 64, True),
    (5000, 264, True, 7, True), (6000, 256, True, 700, True), (9000, 512, False, 0, True), (4000, 1024, True, 1, True),
    (700, 16384, True, 9, True), (700, 8200, False, 350, True),
]


@pytest.mark.parametrize("t,h,post,rows,pre", NORMS)
def test_norms(t, h, post, rows, pre):
    norms.test_forward(t, h, True, post, rows, pre)
    norms.test_backward(t, h, True, post, rows, pre)


@pytest.mark.parametrize("t,h", [(2500, 4096), (6000, 256)])
def test_norm_alone(t, h):
    norms.test_forward(t, h, False, False, 0, True)
    norms.test_backward(t, h, False, False, 0, True)


# 90 tiles of dX, and 90 summed in several pieces; 256 tiles; more than one run of tokens
@pytest.mark.parametrize("t,h,v", [(2500, 2056, 1100), (2500, 2056, 20000), (4096, 4096, 1000), (4200, 264, 33000)])
def test_vocabulary_loss(t, h, v):
    vocab.test_forward_backward_and_both_at_once(t, h, v)


@pytest.mark.parametrize("t", [20, 300])
def test_a_logit_is_summed_in_pieces_of_512(t):
    """One word, so that lse is its logit. The first input's product is 2^24, where fp32 has steps of 2, and
    every 16 inputs behind it add 1.5, which a sum that is truncated every 16 inputs loses: 31 times, at most
    one step each, if no more than 512 inputs are summed in tensor memory, 63 times with 1024. The pieces'
    sums are added in fp32: 15 times half a step. Two steps for the statistics behind them."""
    h = 8192
    X, W = torch.zeros(t, h), torch.zeros(1, h)
    X[:, ::16], W[:, ::16] = 1.5, 1.0
    X[:, 0], W[:, 0] = 2.0 ** 12, 2.0 ** 12
    _, lse = B.qlora_vocab_loss_fwd(X.bfloat16().cuda(), W.bfloat16().cuda(), torch.zeros(t, dtype=torch.int64, device="cuda"))
    want = torch.full((t,), 2.0 ** 24 + 511 * 1.5, dtype=torch.float64)
    assert_within(lse, want, torch.full_like(want, 31 * 2 + 15 + 2 * 2), "lse")
    assert 63 * 1.5 > 31 * 2 + 15 + 2 * 2 and U32 * 2.0 ** 24 == 1.0


def test_outputs_and_workspaces_are_written_in_bounds():
    for t, h, rows in ((700, 4096, 100), (2500, 4104, 33), (6000, 256, 700)):
        bounds.test_norms(t, h, rows)
    bounds.test_vocabulary_loss(2500, 2056, 1100)
