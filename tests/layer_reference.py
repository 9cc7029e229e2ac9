"""Plain 64-bit implementations of the dense layer, its gradients, the orthogonalisation
and the Muon step, on the host, and the bounds that the kernels' arithmetic allows.

The tensor cores multiply 16-bit operands exactly and add 16 products at a time to an
fp32 sum whose low bits may be cut off: a step is off by less than 2^-22 of the largest
magnitude that meets there, which is at most the sum of the terms' magnitudes.
"""
from __future__ import annotations

import math

import torch

U = 2.0 ** -24
ROUND = {torch.bfloat16: 2.0 ** -8, torch.float32: U, torch.float16: 2.0 ** -11}
COEFS = (3.4445, -4.7750, 2.0315)
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")


def sum_error(magnitudes, terms):
    """Of a sum of `terms` products: steps of 16, and the joins of partial sums."""
    return (terms / 16 + 16) * 2.0 ** -22 * magnitudes


def stored(value, err, dtype):
    """`err` of the value before it is stored, and the rounding (to at least a subnormal step)."""
    return err + ROUND[dtype] * (value.abs() + err) + 1e-38


def act(z, kind):
    if kind == "relu":
        return z.clamp(min=0)
    if kind == "gelu":
        return z * torch.special.ndtr(z)
    if kind == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    if kind == "silu":
        return z * torch.sigmoid(z)
    return z


def act_slope(z, kind):
    if kind == "none":
        return torch.ones_like(z)
    if kind == "relu":
        return (z > 0).to(z.dtype)
    if kind == "gelu":
        return torch.special.ndtr(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if kind == "silu":
        q = torch.sigmoid(z)
        return q + z * q * (1 - q)
    t = torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z * z)


# The fp32 evaluations of value and slope: a dozen roundings of terms up to 2 (1 + |z|), the
# exponential's and erfc's few units in the last place, and arguments rounded before them (their
# factor |z| is at most 10 where the exponential is not yet 0 beside 2^-24).
def act_error(z):
    return 64 * U * (1 + z.abs())


SLOPE = 1.13    # the largest slope of any of them


def linear(x, w, bias=None, residual=None, kind="none"):
    """(y, z, bound of y, bound of z) before they are stored; x [P, T, K], w [P, N, K] float64."""
    z, mag = x @ w.mT, x.abs() @ w.abs().mT
    if bias is not None:
        z, mag = z + bias.unsqueeze(1), mag + bias.abs().unsqueeze(1)
    ez = sum_error(mag, x.shape[-1])
    y = act(z, kind)
    ey = ez * (SLOPE if kind != "none" else 1) + (act_error(z) if kind != "none" else 0)
    if residual is not None:
        y = y + residual
        ey = ey + 2 * U * (y.abs() + residual.abs())
    return y, z, ey, ez


def linear_grad(dy, z, x, w, kind="none", rounds=False):
    """(dx, dw, dbias) and their bounds before they are stored.  rounds: dz is rounded to bf16
    as the products' operand."""
    dz = dy * act_slope(z, kind) if kind != "none" else dy
    edz = dy.abs() * act_error(z) if kind != "none" else torch.zeros_like(dz)
    ep = edz + (ROUND[torch.bfloat16] * dz.abs() if rounds else 0)
    T, N = dz.shape[-2:]
    mdz = dz.abs() + ep
    dx, dw, db = dz @ w, dz.mT @ x, dz.sum(1)
    ex = ep @ w.abs() + sum_error(mdz @ w.abs(), N)
    ew = ep.mT @ x.abs() + sum_error(mdz.mT @ x.abs(), T)
    eb = edz.sum(1) + (T + 16) * U * dz.abs().sum(1)
    return (dx, dw, db), (ex, ew, eb)


def newton_schulz(x, steps=5, coefs=COEFS, eps=1e-7):
    """x [..., rows, cols] float64."""
    a, b, c = coefs
    x = x / x.flatten(-2).norm(dim=-1).clamp(min=eps)[..., None, None]
    if x.shape[-2] > x.shape[-1]:
        return newton_schulz_wide(x.mT, steps, coefs).mT
    return newton_schulz_wide(x, steps, coefs)


def newton_schulz_wide(x, steps, coefs):
    a, b, c = coefs
    for _ in range(steps):
        g = x @ x.mT
        x = a * x + (b * g + c * (g @ g)) @ x
    return x


def muon(mean, momentum, master, lr, mu, decay, nesterov, scale, steps=5, coef=1.0):
    """(master, momentum, O) of one matrix, float64."""
    g = mean * coef
    buf = mu * momentum + (1 - mu) * g
    u = mu * buf + (1 - mu) * g if nesterov else buf
    o = newton_schulz(u, steps)
    return (1 - lr * decay) * master - lr * scale * o, buf, o
