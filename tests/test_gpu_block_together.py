"""The operators used together, as a training step and a decode step use them: norm, linear with its
activation, linear back, norm with gate and residual scale, loss through the head; its whole backward
against autograd in 64 bits; the same captured into a graph and replayed on new inputs beside an eager
run; and calls on another device's tensors or another stream."""

import numpy as np
import pytest
import torch

from bit_quantized_lora_03_b200 import binding as B
from bit_quantized_lora_03_b200 import inputs
from oracle import nf4_oracle as O

from block_util import ACT, norm_fwd64, randn
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


H, F, V, R, S, SCALE, EPS = 256, 448, 1100, 16, 0.5, 0.7, 1e-5


class Block:
    """x -> norm -> up (bias, gelu) -> down -> x + scale.gate.norm(.) -> norm -> loss through the head."""

    def __init__(self, t, seq):
        self.t, self.seq = t, seq
        self.up, self.down = (inputs.random_linear(t, h, o, R, S, seed=i) for i, (h, o) in enumerate(((H, F), (F, H))))
        self.pu, self.pd = B.nf4_quantize(self.up.Wt.cuda()), B.nf4_quantize(self.down.Wt.cuda())
        c = lambda shape, s, i: randn(shape, s, i).cuda()  # noqa: E731
        self.w0, self.w1, self.w2 = (1 + c((H,), 0.1, 20 + i) for i in range(3))
        self.b, self.gate = c((F,), 0.3, 30), c((-(-t // seq), H), 0.5, 31)
        self.head = c((V, H), 2.0 / 16, 32)
        self.ad = [x.cuda() for x in (self.up.L1, self.up.L2, self.down.L1, self.down.L2)]

    def inputs(self, seed):
        y = torch.randint(0, V, (self.t,), generator=torch.Generator().manual_seed(seed))
        y[::5] = -100
        return randn((self.t, H), 1.0, seed).cuda(), y.cuda()

    def step(self, x, y, d):
        u1, u2, d1, d2 = self.ad
        _, n0, _, r0 = B.qlora_norm_residual_fwd(x, w_pre=self.w0, eps=EPS)
        a, z, su = B.qlora_linear_fwd_epilogue(n0, self.pu, u1, u2, S, bias=self.b, act="gelu", want_Z=True)
        m, _, sd = B.qlora_linear_fwd_epilogue(a, self.pd, d1, d2, S)
        xo, n, ro, ri = B.qlora_norm_residual_fwd(x, m, w_post=self.w1, gate=self.gate, w_pre=self.w2, scale=SCALE,
                                                  eps=EPS, rows_per_gate=self.seq)
        loss, lse, dn = B.qlora_vocab_loss_fwd_bwd(n, self.head, y, d)
        zero = torch.zeros_like(x)
        dxo, dm, dw1, dg, dw2 = B.qlora_norm_residual_bwd(zero, dn, xo, m, ro, ri, w_post=self.w1, gate=self.gate,
                                                          w_pre=self.w2, scale=SCALE, rows_per_gate=self.seq)
        ws = torch.empty(max(B.bwd_workspace_bytes(self.t, F, H, R), B.bwd_workspace_bytes(self.t, H, F, R)),
                         dtype=torch.uint8, device="cuda")
        da, dd1, dd2 = B.qlora_linear_bwd(dm, a, self.pd, d1, d2, S, sT=sd, ws=ws)
        dz, db = B.qlora_epilogue_bwd(da, z, "gelu")
        dn0, du1, du2 = B.qlora_linear_bwd(dz, n0, self.pu, u1, u2, S, sT=su, ws=ws)
        dx, _, _, _, dw0 = B.qlora_norm_residual_bwd(dxo, dn0, x, None, None, r0, w_pre=self.w0)
        return {"loss": loss, "dx": dx, "dw0": dw0, "dw1": dw1, "dw2": dw2, "dgate": dg, "db": db, "du1": du1,
                "du2": du2, "dd1": dd1, "dd2": dd2}

    def reference(self, x, y, d):
        deq = lambda li: torch.from_numpy(np.array(O.nf4_dequantize(O.nf4_quantize(li.Wt.numpy())))).double().cuda()  # noqa: E731
        W = [deq(li) for li in (self.up, self.down)]
        W = [w if w.shape == (li.o, li.h) else w.t() for w, li in zip(W, (self.up, self.down))]
        p = {k: v.double().requires_grad_(True) for k, v in dict(
            x=x, w0=self.w0, w1=self.w1, w2=self.w2, gate=self.gate, b=self.b, u1=self.ad[0], u2=self.ad[1],
            d1=self.ad[2], d2=self.ad[3]).items()}
        _, n0, _, _ = norm_fwd64(p["x"], None, None, None, p["w0"], 1.0, EPS, 0)
        a = ACT["gelu"](n0 @ W[0].T + S * (n0 @ p["u1"]) @ p["u2"] + p["b"])
        m = a @ W[1].T + S * (a @ p["d1"]) @ p["d2"]
        _, n, _, _ = norm_fwd64(p["x"], m, p["w1"], p["gate"], p["w2"], SCALE, EPS, self.seq)
        loss = torch.nn.functional.cross_entropy(n @ self.head.double().T, y, ignore_index=-100, reduction="none")
        (loss * d.double()).sum().backward()
        g = {k: v.grad for k, v in p.items()}
        return {"loss": loss.detach(), "dx": g["x"], "dw0": g["w0"], "dw1": g["w1"], "dw2": g["w2"], "dgate": g["gate"],
                "db": g["b"], "du1": g["u1"], "du2": g["u2"], "dd1": g["d1"], "dd2": g["d2"]}


@pytest.mark.parametrize("t,seq", [(7, 3), (16, 16), (150, 64), (700, 100)])
def test_a_step_and_its_gradients(t, seq):
    blk = Block(t, seq)
    x, y = blk.inputs(5)
    d = torch.full((t,), 1.0 / t, device="cuda")
    got, ref = blk.step(x, y, d), blk.reference(x, y, d)
    assert B.last_status() == 0
    # The tensors handed from one operator to the next are rounded to bf16, 2^-8 of a value at most, some
    # ten of them between the two ends, each entering with a factor of order one: a tenth of the norm is
    # far above their sum (10 x 2^-8 = 0.04) and far below what a wrong term or sign makes.
    for k, want in ref.items():
        far = (got[k].double() - want).norm() / want.norm()
        assert far <= 0.1, (k, far.item())


def test_captured_steps_replay_with_new_inputs_beside_eager_ones():
    """Two graphs of the same step and an eager run share no workspace: replayed one after the other and
    at once on two streams, each gives what its inputs give alone."""
    t = 150
    blk = Block(t, 50)
    d = torch.full((t,), 1.0 / t, device="cuda")
    sets = [blk.inputs(s) for s in (11, 12, 13)]
    alone = [blk.step(x, y, d) for x, y in sets]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graphs = []
    for _ in range(2):
        x, y = (v.clone() for v in sets[0])
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            blk.step(x, y, d)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = blk.step(x, y, d)
        graphs.append((g, x, y, out))
    for (g, x, y, out), s in zip(graphs, sets[1:]):
        x.copy_(s[0])
        y.copy_(s[1])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(3):
        for (g, _, _, _), st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        eager = blk.step(*sets[0], d)
    torch.cuda.synchronize()
    for got, want in ((eager, alone[0]), (graphs[0][3], alone[1]), (graphs[1][3], alone[2])):
        for k in want:
            assert torch.equal(got[k], want[k]), k
    assert B.last_status() == 0


def test_decode_step_in_a_graph():
    """One token through norm, linear, norm and loss (the decode kernels), captured and replayed."""
    blk = Block(1, 1)
    x, y = blk.inputs(3)
    y[:] = 17

    def decode():
        _, n0, _, _ = B.qlora_norm_residual_fwd(x, w_pre=blk.w0, eps=EPS)
        a, _, _ = B.qlora_linear_fwd_epilogue(n0, blk.pu, *blk.ad[:2], S, bias=blk.b, act="gelu")
        m, _, _ = B.qlora_linear_fwd_epilogue(a, blk.pd, *blk.ad[2:], S, residual=x)
        return m, *B.qlora_vocab_loss_fwd(m, blk.head, y)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        decode()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = decode()
    x.copy_(randn((1, H), 1.0, 77))
    g.replay()
    want = decode()
    torch.cuda.synchronize()
    # the decode sums' order may differ: a bf16 step of the linears, and what it makes of the loss
    for a, b in zip(out, want):
        assert torch.allclose(a.float(), b.float(), rtol=2.0 ** -6, atol=2.0 ** -6)


def test_stream_argument_orders_after_work_on_that_stream():
    st = torch.cuda.Stream()
    x = torch.zeros(2048, 4096, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(4096, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        for _ in range(20):
            x += 0.125      # exact in bf16 up to 2.5
    xo, n, _, _ = B.qlora_norm_residual_fwd(x, w_pre=w, stream=st)
    st.synchronize()
    assert (xo == 2.5).all() and torch.equal(n, torch.ones_like(n))


def test_refuses_tensors_of_two_devices():
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match="w_pre"):
        B.qlora_norm_residual_fwd(x, w_pre=torch.ones(64, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="targets"):
        B.qlora_vocab_loss_fwd(x, x, torch.zeros(4, dtype=torch.int64))
    with pytest.raises(ValueError, match="contiguous"):
        B.qlora_norm_residual_fwd(torch.zeros(64, 64, dtype=torch.bfloat16, device="cuda").t())
    with pytest.raises(RuntimeError, match="MISALIGNED"):
        B.qlora_norm_residual_fwd(torch.zeros(4 * 64 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(4, 64))
