"""Logits with finite masks: rows some or all of whose values are a large negative constant,
and rows whose largest values are large, in every group size that the rules choose (warps, 128,
256 and 512 threads, clusters, rows longer than shared memory).  References in 64 bits on the GPU."""
import math

import pytest
import torch

import gradient_sync_zero_gb300 as dps
from model_reference import U, stored
from test_model_ops_gpu import BF, F32, bits
from test_model_ops_paths_gpu import within

pytestmark = pytest.mark.gpu

MASKS = [-1e9, -5e9, -1e10, -1e12, -1e20, -1e30, -1e35]
TOPS = [5e8, 5e9, 1e12]
PATTERNS = ["tail", "alternating", "most"]
SPECS = [(m, p) for m in MASKS for p in PATTERNS] + [(m, "whole") for m in MASKS] + \
        [(m, "top") for m in TOPS] + [(0.0, "plain")] * 2
GROUPS = [(1, 36, 700), (1, 2100, 2999), (2, 36, 5000), (1, 320, 20011), (1, 320, 50257), (1, 36, 50257),
          (1, 33, 450001)]


def _masked(P, T, V, dtype):
    """x, tokens, and per row the largest |ordinary logit| and whether the row is beyond them."""
    g = torch.Generator(device="cuda")
    g.manual_seed(V)
    x = 3 * torch.randn(P, T, V, generator=g, device="cuda")
    z, special = x.abs().amax(-1).double(), torch.zeros(P, T, dtype=torch.bool, device="cuda")
    at = torch.arange(V, device="cuda")
    tok = 2 * (V // 10)
    for r in range(P):
        for t in range(T):
            value, kind = SPECS[(r * T + t) % len(SPECS)]
            if kind == "tail":
                x[r, t, V // 3:] = value
            elif kind == "alternating":
                x[r, t, 1::2] = value
            elif kind == "most":
                x[r, t].masked_fill_((torch.rand(V, generator=g, device="cuda") < 0.95) & (at != tok), value)
            elif kind == "whole":
                x[r, t] = value
            elif kind == "top":
                x[r, t, [0, tok, V - 1]] = value
            special[r, t] = kind in ("whole", "top")
    tokens = torch.full((P, T), tok, device="cuda")
    return x.to(dtype), tokens, z, special


def _exact(x, tokens, alpha):
    """logp, lse and the softmax from differences, which lose nothing beside a large maximum."""
    top = x.double().amax(-1, keepdim=True)
    d = (x.double() - top) * alpha
    ls = torch.exp(d).sum(-1, keepdim=True).log()
    logp = (d - ls).gather(-1, tokens.unsqueeze(-1)).squeeze(-1)
    return logp, (top * alpha + ls).squeeze(-1), torch.exp(d - ls)


@pytest.mark.parametrize("alpha", [1.0, 0.5, 1.25])
@pytest.mark.parametrize("P,T,V", GROUPS, ids=str)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_finite_masks(P, T, V, dtype, alpha):
    """Bounds, Z a row's largest ordinary |scaled logit|: exponents are differences up to 2 Z
    that carry c's two roundings and their own (6 U Z) each, so do the token's, the references of
    merged sums 2 U Z, the last two operations 4 U Z + 2 U ln V; a thread adds V / 2G terms to each
    of its two sums.  Beside a maximum of up to 2^30 in base 2 the token's exponent and the logarithm
    are up to 32 and 63, and cancel: 200 U more where there is one."""
    x, tokens, z, special = _masked(P, T, V, dtype)
    logp, lse, p = _exact(x, tokens, alpha)
    group = 32 if V * x.element_size() <= 16384 else 128
    tol = U * (20 * alpha * z + V / (2 * group) + 64 + 4 * math.log(V)) + 200 * U * special
    a, b = torch.empty(P, T, device="cuda"), torch.empty(P, T, device="cuda")
    dps.dp_token_logprob(x, tokens, a, b, logit_scale=alpha)
    within(a, logp, tol)
    within(b, lse, tol + 3 * U * lse.abs())

    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda", dtype=torch.float64)   # noqa: E731
    moved = 0.3 * rnd(P, T)
    for c in (0.8, 1.2):                             # away from the clamp's corners
        moved = torch.where((torch.exp(moved) - c).abs() < 1e-2, moved + 4e-2, moved)
    old, rf, adv = (logp - moved).float(), (logp + 0.3 * rnd(P, T)).float(), rnd(P, T).float()
    w = 0.25 + 0.75 * torch.rand(P, T, generator=g, device="cuda")
    beta = 0.1
    q, A, d = torch.exp(logp - old.double()), adv.double(), rf.double() - logp
    held = q.clamp(0.8, 1.2) * A
    clipped = held < q * A
    pg, kl = -torch.minimum(q * A, held), torch.expm1(d) - d
    dlogp = w.double() * (torch.where(clipped, 0.0, -q * A) - beta * torch.expm1(d))
    terms = torch.stack((pg + beta * kl, pg, kl, clipped.double()), -1) * w.double().unsqueeze(-1)
    one = torch.zeros_like(p).scatter_(-1, tokens.unsqueeze(-1), 1.0)
    want = (dlogp * alpha).unsqueeze(-1) * (one - p)
    # the slope is off by at most (|slope| + 2 beta e^d + beta) w tol and a few U, and 0.1 (2 e^1.5 + 1) < 1
    err = (dlogp * alpha).abs().unsqueeze(-1) * (p * (2 * tol).unsqueeze(-1) + 4 * U)
    err += ((dlogp.abs() + 1.0) * (2 * tol + 16 * U) * alpha).unsqueeze(-1) * (p + one)
    stats = torch.empty(P, 4, device="cuda")
    dl = torch.full_like(x, float("nan"))
    kw = dict(ref_logp=rf, weight=w, cfg=dps.policy_cfg(0.2, 0.2, beta, alpha))
    dps.dp_policy_loss(x, tokens, old, adv, a, stats, dlogits=dl, **kw)
    within(a, logp, tol)
    within(dl, want, stored(want, err, dtype))
    row = w.double() * ((q * A.abs() + 3.0) * (2 * tol + 32 * U))
    within(stats, terms.sum(1), row.sum(1, keepdim=True) + U * terms.sum(1).abs())
    dps.dp_policy_loss(x, tokens, old, adv, a, stats, dlogits=x, **kw)      # in place
    assert torch.equal(bits(x), bits(dl))


@pytest.mark.parametrize("mask", MASKS)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_token_that_is_masked(mask, dtype):
    """Its log-probability is the mask's distance; it has no softmax, and nothing is NaN."""
    x = torch.randn(1, 3, 40000, device="cuda", generator=torch.Generator(device="cuda").manual_seed(2)).to(dtype)
    x[:, :, 1000:] = mask
    tokens = torch.full((1, 3), 30000, device="cuda")
    a, b = torch.empty(1, 3, device="cuda"), torch.empty(1, 3, device="cuda")
    dps.dp_token_logprob(x, tokens, a, b)
    logp, lse, _ = _exact(x, tokens, 1.0)
    tol = U * (20 * float(x[:, :, :1000].abs().max()) + 40000 / 256 + 64 + 4 * math.log(40000))
    within(a, logp, tol + 4 * U * logp.abs())
    within(b, lse, tol)
