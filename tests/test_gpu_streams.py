"""Calls on another stream than their inputs' whose inputs are freed as soon as the call returns."""

import pytest
import torch

from bit_quantized_lora_03_b200 import binding as B

from block_util import randn
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu
T, H, O, R, V = 40, 256, 320, 16, 1000


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _packed():
    return B.nf4_quantize(randn((O, H), 0.02, 1, torch.float32).cuda())


def _c(shape, seed, dtype=torch.bfloat16):
    return randn(shape, 1.0, seed, dtype).cuda()


def _y():
    return (torch.arange(T) * 7 % V).cuda()


f32 = torch.float32
CALLS = {   # name: (inputs, call)
    "nf4_quantize": (lambda: [_c((O, H), 1, f32)], lambda s, w: B.nf4_quantize(w, stream=s)),
    "nf4_dequantize": (lambda: [_packed()], lambda s, p: B.nf4_dequantize(p, stream=s)),
    "linear_fwd": (lambda: [_c((T, H), 1), _packed(), _c((H, R), 2), _c((R, O), 3)],
                   lambda s, x, p, a, b: B.qlora_linear_fwd(x, p, a, b, 0.5, stream=s)),
    "linear_bwd": (lambda: [_c((T, O), 4), _c((T, H), 1), _packed(), _c((H, R), 2), _c((R, O), 3)],
                   lambda s, d, x, p, a, b: B.qlora_linear_bwd(d, x, p, a, b, 0.5, stream=s)),
    "dropout_apply": (lambda: [_c((T, H), 1)], lambda s, x: B.qlora_dropout_apply(x, 0.1, 5, stream=s)),
    "linear_fwd_dropout": (lambda: [_c((T, H), 1), _packed(), _c((H, R), 2), _c((R, O), 3)],
                           lambda s, x, p, a, b: B.qlora_linear_fwd_dropout(x, p, a, b, 0.5, 0.1, 3, stream=s)),
    "linear_bwd_dropout": (lambda: [_c((T, O), 4), _c((T, H), 1), _packed(), _c((H, R), 2), _c((R, O), 3)],
                           lambda s, d, x, p, a, b: B.qlora_linear_bwd_dropout(d, x, p, a, b, 0.5, 0.1, 3, stream=s)),
    "merge_adapters": (lambda: [_packed(), _c((H, R), 2), _c((R, O), 3)],
                       lambda s, p, a, b: B.merge_adapters(p, a, b, 0.5, stream=s)),
    "adamw_step": (lambda: [_c((64, 64), i, f32).abs() for i in range(4)],
                   lambda s, p, g, m, v: B.adamw_step(p, g, m, v, 1, stream=s)),
    "adamw_step_multi": (lambda: [_c((64, 64), i, f32).abs() for i in range(4)],
                         lambda s, p, g, m, v: B.adamw_step_multi([p], [g], [m], [v], 1, stream=s)),
    "linear_fwd_epilogue": (lambda: [_c((T, H), 1), _packed(), _c((H, R), 2), _c((R, O), 3), _c((O,), 4), _c((T, O), 5)],
                            lambda s, x, p, a, b, c, r: B.qlora_linear_fwd_epilogue(
                                x, p, a, b, 0.5, bias=c, act="silu", residual=r, want_Z=True, stream=s)),
    "epilogue_bwd": (lambda: [_c((T, O), 1), _c((T, O), 2)], lambda s, d, z: B.qlora_epilogue_bwd(d, z, "silu", stream=s)),
    "norm_residual_fwd": (lambda: [_c((T, H), 1), _c((T, H), 2), _c((H,), 3), _c((1, H), 4), _c((H,), 5)],
                          lambda s, x, y, o, g, i: B.qlora_norm_residual_fwd(x, y, w_post=o, gate=g, w_pre=i, stream=s)),
    "norm_residual_bwd": (lambda: [*(_c((T, H), i) for i in range(4)), _c((T,), 4, f32), _c((T,), 5, f32), _c((H,), 6),
                                   _c((1, H), 7), _c((H,), 8)],
                          lambda s, dx, dn, x, y, ro, ri, o, g, i: B.qlora_norm_residual_bwd(
                              dx, dn, x, y, ro, ri, w_post=o, gate=g, w_pre=i, stream=s)),
    "vocab_loss_fwd": (lambda: [_c((T, H), 1), _c((V, H), 2), _y()], lambda s, x, w, y: B.qlora_vocab_loss_fwd(x, w, y, stream=s)),
    "vocab_loss_bwd": (lambda: [_c((T, H), 1), _c((V, H), 2), _y(), _c((T,), 3, f32), _c((T,), 4, f32), _c((T,), 5, f32)],
                       lambda s, x, w, y, lse, d, e: B.qlora_vocab_loss_bwd(x, w, y, lse, d, dlse=e, stream=s)),
    "vocab_loss_fwd_bwd": (lambda: [_c((T, H), 1), _c((V, H), 2), _y(), _c((T,), 4, f32)],
                           lambda s, x, w, y, d: B.qlora_vocab_loss_fwd_bwd(x, w, y, d, stream=s)),
}


def _tensors(values):
    for v in values:
        yield from (v.codes, v.absmax_q8, v.absmax_s2) if isinstance(v, B.PackedNF4) else (v,)


@pytest.mark.parametrize("name", list(CALLS))
def test_inputs_freed_at_once_are_not_given_out_again(name):
    make, call = CALLS[name]
    side = torch.cuda.Stream()
    call(side, *make())     # (what the call keeps for later ones is there)
    torch.cuda.synchronize()
    values = make()
    kinds = [(t.shape, t.dtype, t.data_ptr()) for t in _tensors(values)]
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)      # a tenth of a second in front of the call
    out = call(side, *values)   # noqa: F841
    assert not side.query()
    del values
    again = [torch.empty(shape, dtype=dtype, device="cuda") for shape, dtype, _ in kinds for _ in range(2)]
    assert not side.query()     # the call has not begun
    got = {(t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()) for t in again}
    for shape, dtype, ptr in kinds:
        assert not any(a <= ptr < b for a, b in got), (name, tuple(shape), dtype)
    torch.cuda.synchronize()


@pytest.mark.parametrize("name", ["linear_fwd_epilogue", "epilogue_bwd", "norm_residual_bwd", "vocab_loss_fwd_bwd", "vocab_loss_bwd"])
def test_calls_on_a_second_stream_inside_a_capture(name):
    """The call joins the capture through its own stream; some of its inputs are made, and freed, in it."""
    make, call = CALLS[name]
    values, side = make(), torch.cuda.Stream()
    want = call(None, *values)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        copies = [v.clone() if torch.is_tensor(v) else v for v in values]
        side.wait_stream(torch.cuda.current_stream())
        out = call(side, *copies)
        torch.cuda.current_stream().wait_stream(side)
        del copies
        after = torch.zeros(1 << 20, device="cuda")     # noqa: F841
    for _ in range(2):
        for t in _tensors([o for o in (out if isinstance(out, tuple) else (out,)) if o is not None]):
            t.zero_()
        g.replay()
    torch.cuda.synchronize()
    pairs = zip(out, want) if isinstance(out, tuple) else ((out, want),)
    for a, b in pairs:
        assert a is None and b is None or torch.equal(a, b)
    del g, out, values
    torch.cuda.synchronize()
    assert B.last_status() == 0
