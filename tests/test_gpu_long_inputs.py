"""Decode with inputs so long that the rank-r kernel stages a CTA's share of them in several pieces,
at ranks whose column pairs do not divide its threads evenly; and that kernel's index arithmetic."""

import os
import re

import numpy as np
import pytest
import torch

from bit_quantized_lora_03_b200 import binding as B
from bit_quantized_lora_03_b200 import build as build_mod
from bit_quantized_lora_03_b200 import inputs
from oracle import nf4_oracle as O

from block_util import U16, U32, assert_within
from gpu_util import assert_close_rms, f32, require_gpu


def _walk(threads, piece_pairs, r, share, idle_threads_work=False):
    """The highest index, relative to a piece's first pair, that a thread reads of a staged token, and the
    highest float that it stores of its sums for one token, over a share of `share` input pairs."""
    pairs = r // 2
    strides = threads // pairs
    piece = piece_pairs // (4 * strides) * (4 * strides)
    read = store = -1
    for tid in range(0, threads, 1):
        cp, kg = tid % pairs, tid // pairs
        if kg >= strides and not idle_threads_work:
            continue
        store = max(store, kg * r + 2 * cp + 1)
        for first in range(0, share, piece):
            end = min(first + piece, share)
            for pb in range(first + kg, end, 4 * strides):
                for u in range(4):
                    pr = pb + u * strides
                    if pr >= (share if idle_threads_work else end):
                        break
                    read = max(read, pr - first)
    return read, store


def test_threads_without_a_stride_would_read_behind_the_staged_piece():
    with open(os.path.join(build_mod.CSRC, "nf4_gemv.cuh")) as f:
        text = f.read().split("namespace gd {")[1]
    threads, piece = (int(re.search(rf"constexpr int {n} = (\d+);", text).group(1)) for n in ("kThreads", "kPiecePairs"))
    for r in range(16, 257, 16):
        for share in (1, 255, 256, 257, 416, 600):
            read, store = _walk(threads, piece, r, share)
            assert read < piece and store < 2 * threads, (r, share)
    # what such a thread would read if it worked: the word behind the last token's (the check sees it)
    assert [r for r in range(16, 257, 16) if _walk(threads, piece, r, 600, True)[0] >= piece] == [
        112, 176, 192, 208, 224, 240]


@pytest.mark.gpu
@pytest.mark.parametrize("t,r", [(16, 112), (5, 176), (1, 240), (9, 208), (16, 16)])
def test_inputs_of_several_pieces(t, r):
    require_gpu()
    li = inputs.random_linear(t, 32832, 64, r, 0.5, seed=r, with_grad=False)
    p = B.nf4_quantize(li.Wt.cuda())
    args = li.X.cuda(), p, li.L1.cuda(), li.L2.cuda(), li.s
    Y, sT = B.qlora_linear_fwd(*args)
    Y2, _, sT2 = B.qlora_linear_fwd_epilogue(*args)
    assert B.last_status() == 0
    W = O.nf4_dequantize(O.nf4_quantize(li.Wt.numpy()))
    want = li.s * (li.X.double() @ li.L1.double())
    # a sum of h exact products in fp32, and its rounding to bf16
    e = li.h * U32 * abs(li.s) * (li.X.double().abs() @ li.L1.double().abs())
    for y, st in ((Y, sT), (Y2, sT2)):
        assert_within(st, want, U16 * (want.abs() + e) + e, "sT")
        assert_close_rms(f32(y), O.qlora_linear_fwd(f32(li.X), np.asarray(W), f32(li.L1), f32(li.L2), li.s)[0], "Y")
