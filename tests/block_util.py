"""64-bit forms of the operators around the linear, and the error bounds their tests use (not
collected as tests).

Rounding units: storing bf16 moves a value by at most 2^-8 of itself, storing or adding fp32 by
2^-24. A fp32 sum of n terms in any order is off by at most (n - 1) 2^-24 of the sum of the terms'
magnitudes (to first order)."""

import math

import torch

U16, U32 = 2.0 ** -8, 2.0 ** -24


def randn(shape, sigma, seed, dtype=torch.bfloat16):
    g = torch.Generator("cpu")
    g.manual_seed(seed)
    return (torch.randn(*shape, generator=g) * sigma).to(dtype)


def assert_within(got, want, bound, name):
    """|got - want| <= bound elementwise, NaN and infinities in the same places."""
    got, want, bound = got.detach().double().cpu(), want.double().cpu(), bound.double().cpu()
    assert got.shape == want.shape, (name, got.shape, want.shape)
    fine = torch.isfinite(want)
    assert torch.equal(fine, torch.isfinite(got)), f"{name}: non-finite values differ"
    off = ((got - want).abs() - bound)[fine]
    worst = off.max().item() if off.numel() else -1.0
    assert worst <= 0, f"{name}: over the bound by {worst:.3g} at {int((off > 0).sum())} of {off.numel()}"


ACT = {
    "none": lambda z: z,
    "relu": torch.relu,
    "gelu": lambda z: z * torch.special.ndtr(z),
    "gelu_tanh": lambda z: 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))),
    "silu": lambda z: z * torch.sigmoid(z),
}


def act_grad(z, act):
    """act'(z) by autograd in 64 bits (relu'(0) = 0)."""
    z = z.double().clone().requires_grad_(True)
    ACT[act](z).sum().backward()
    return z.grad


def norm_fwd64(x, y, w_post, gate, w_pre, scale, eps, rows):
    """(x', n, rstd_post, rstd_pre) in 64 bits; gate rows expanded here."""
    x = x.double()
    ro = ri = n = None
    if y is not None:
        u = y.double()
        if w_post is not None:
            ro = (u.square().mean(1) + eps).rsqrt()
            u = u * ro[:, None] * w_post.double()
        if gate is not None:
            u = u * gate.double()[torch.arange(x.shape[0], device=x.device) // rows]
        x = x + scale * u
    if w_pre is not None:
        ri = (x.square().mean(1) + eps).rsqrt()
        n = x * ri[:, None] * w_pre.double()
    return x, n, ro, ri
