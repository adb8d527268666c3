"""Plain 64-bit forms (torch on the CPU) of the rotary positions, the projections with low-rank adapters and the
gated feed-forward block, with bounds on what fp32 sums and one rounding may add."""
from __future__ import annotations

import math

import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}  # the largest relative error of a rounding


def bf16(gen, *shape, std=1.0):
    return (torch.randn(shape, generator=gen, dtype=torch.float64) * std).to(torch.bfloat16)


def i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def cumulative(lens):
    return [sum(lens[:i]) for i in range(len(lens) + 1)]


# ---- rotary positions ------------------------------------------------------------------------------
def frequencies(rot, theta, factor=1.0, orig_len=0, beta_fast=32.0, beta_slow=1.0):
    out = []
    for i in range(rot // 2):
        f = theta ** (-2 * i / rot)
        slow = 1.0
        if orig_len:
            pair = [rot * math.log(orig_len / (2 * math.pi * n)) / (2 * math.log(theta)) for n in (beta_fast, beta_slow)]
            lo, hi = max(math.floor(pair[0]), 0), min(math.ceil(pair[1]), rot - 1)
            slow = min(max((i - lo) / max(hi - lo, 0.001), 0.0), 1.0)
        out.append(f * (1 - slow) + slow * f / factor)
    return torch.tensor(out, dtype=torch.float64)


def rope(x, positions, freq, half, m=1.0):
    """x [n, heads, D] in 64 bits, the first 2 len(freq) elements of a head rotated.  Also |a| + |b| of each element's pair (0
    for the rest)."""
    n, rot = len(freq), 2 * len(freq)
    angle = positions.double()[:, None] * freq
    c, s = (m * torch.cos(angle))[:, None], (m * torch.sin(angle))[:, None]
    first = torch.arange(n) if half else 2 * torch.arange(n)
    second = first + n if half else first + 1
    y, size = x.clone(), torch.zeros_like(x)
    a, b = x[..., first], x[..., second]
    y[..., first], y[..., second] = a * c - b * s, b * c + a * s
    size[..., first] = size[..., second] = m * (a.abs() + b.abs())
    return y, size


# ---- projections -----------------------------------------------------------------------------------
def product(x, w):
    """x w^T, and a bound on the error of fp32 sums of bf16 products."""
    k = x.shape[1]
    return x @ w.T, (k + 8) * 2.0 ** -24 * (x.abs() @ w.abs().T)


def gated(x, g, u):
    """silu(x g^T) * (x u^T) and the bound before its rounding: the slope of silu is below 1.1, and expf, the division and the
    products are good to a few 2^-22."""
    (p, dp), (q, dq) = product(x, g), product(x, u)
    act = p * torch.sigmoid(p)
    y = act * q
    return y, 1.1 * dp * (q.abs() + dq) + act.abs() * dq + 2.0 ** -20 * y.abs() + 1e-37


def lora(x, w, a, b, scale, cu, which):
    """The shared projection plus each request's adapter, and the bound before rounding: fp32 sums on both sides, the low-rank
    activations to 2^-16."""
    y, d = product(x, w)
    for s, e in enumerate(which):
        first, last = max(cu[s], 0), min(cu[s + 1], x.shape[0])
        if not 0 <= e < a.shape[0] or first >= last:
            continue
        rows = slice(first, last)
        v, dv = product(x[rows], a[e])
        v, dv = v * scale[e], dv * abs(scale[e]) + 2.0 ** -16 * (v * scale[e]).abs()
        y[rows] += v @ b[e].T
        d[rows] += (dv + (b.shape[2] + 8) * 2.0 ** -24 * v.abs()) @ b[e].abs().T
    return y, d


def check(got, want, slack, what=""):
    """Every element within one rounding of its type and the bound."""
    got64 = got.detach().cpu().double()
    bound = HALF[got.dtype] * (want.abs() + slack) + slack
    bad = ~((got64 - want).abs() <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} elements outside the bound, worst excess " \
                          f"{float(((got64 - want).abs() - bound).max()):.3e}"
