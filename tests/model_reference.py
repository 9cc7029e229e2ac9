"""Plain 64-bit implementations of the operators at the ends of a training step,
on the host, and the error bounds the kernels' fp32 arithmetic allows.

U is fp32's unit roundoff.  Each bound adds the roundings of the operation
sequence to first order; stored() adds the rounding of the stored value.
"""
from __future__ import annotations

import numpy as np
import torch

U = 2.0 ** -24
ROUND = {torch.bfloat16: 2.0 ** -8, torch.float32: U}
M0, M1, W0, W1 = 0xD2511F53, 0xCD9E8D57, 0x9E3779B9, 0xBB67AE85


def philox4x32(counter, key, rounds=10):
    """counter: four uint64 arrays of 32-bit words; key: two ints."""
    m32, s32 = np.uint64(0xFFFFFFFF), np.uint64(32)
    c = [np.asarray(x, dtype=np.uint64) for x in counter]
    k0, k1 = int(key[0]), int(key[1])
    for _ in range(rounds):
        a, b = c[0] * np.uint64(M0), c[2] * np.uint64(M1)
        c = [(b >> s32) ^ c[1] ^ np.uint64(k0), b & m32, (a >> s32) ^ c[3] ^ np.uint64(k1), a & m32]
        k0, k1 = (k0 + W0) & 0xFFFFFFFF, (k1 + W1) & 0xFFFFFFFF
    return c


def keep_mask(P, n, p, seed, offset, rank0=0):
    """[P, n] bool."""
    out = np.empty((P, n), dtype=bool)
    b = np.arange(-(-n // 4), dtype=np.uint64)
    for r in range(P):
        one = np.ones_like(b)
        w = philox4x32([b & np.uint64(0xFFFFFFFF), b >> np.uint64(32), one * np.uint64(rank0 + r),
                        one * np.uint64(offset)], (seed & 0xFFFFFFFF, seed >> 32))
        out[r] = np.stack(w, -1).reshape(-1)[:n] >= np.uint64(round(p * 2 ** 32))
    return torch.from_numpy(out)


def dropout(x, p, seed, offset, rank0=0):
    """x [P, T, D] float64."""
    if round(p * 2 ** 32) == 0:
        return x
    keep = keep_mask(x.shape[0], x.shape[1] * x.shape[2], p, seed, offset, rank0).view_as(x)
    return torch.where(keep, x / (1 - p) if p < 1 else x, torch.zeros_like(x))


def lookup(table, tokens, scale, drop=None):
    """table [P, V, D] float64, tokens [P, T] -> [P, T, D]."""
    P, V, _ = table.shape
    real = (tokens >= 0) & (tokens < V)
    out = torch.stack([table[r][tokens[r].clamp(0, V - 1).long()] for r in range(P)]) * scale
    out = torch.where(real.unsqueeze(-1), out, torch.zeros_like(out))
    return out if drop is None else dropout(out, *drop)


def lookup_grad(dout, tokens, V, scale, drop=None):
    """(gradient, sum of the terms' magnitudes, tokens per row), float64."""
    d = dout if drop is None else dropout(dout, *drop)
    P, T, D = d.shape
    g, mag, n = (torch.zeros(P, V, k, dtype=torch.float64) for k in (D, D, 1))
    for r in range(P):
        for t in range(T):
            v = int(tokens[r, t])
            if 0 <= v < V:
                g[r, v] += scale * d[r, t]
                mag[r, v] += (scale * d[r, t]).abs()
                n[r, v] += 1
    return g, mag, n


def stored(ref, err, dtype):
    """Bound on |stored - ref| when the value is off by at most err before it is
    rounded to dtype."""
    return err + ROUND[dtype] * (ref.abs() + err) + 2.0 ** -133


def logprob(logits, tokens, alpha):
    """(logp, lse) float64 [P, T]."""
    z = logits * alpha
    lse = torch.logsumexp(z, -1)
    real = (tokens >= 0) & (tokens < z.shape[-1])
    at = tokens.clamp(0, z.shape[-1] - 1).long().unsqueeze(-1)
    zero = torch.zeros_like(lse)
    return torch.where(real, z.gather(-1, at).squeeze(-1) - lse, zero), torch.where(real, lse, zero)


def logprob_bound(logits, alpha):
    """Each exponent z - m carries the roundings of z, of the difference and of its
    scaling to base 2 (3 U max|z| each way at most), the exponential and the joins a few
    U more, the sum at most U per term of a thread's share (V / 256, no CTA has
    fewer threads) and of the tree; the logarithm and the last differences add U
    of their operands."""
    z = logits[torch.isfinite(logits)].abs().max().item() * alpha if logits.numel() else 0.0
    V = logits.shape[-1]
    return U * (10 * z + V / 256 + 48 + 4 * np.log(V + 1.0))


def logit_grad(logits, tokens, alpha, lse, dlogp):
    z = logits * alpha
    p = torch.exp(z - lse.unsqueeze(-1))
    one = torch.zeros_like(p)
    real = (tokens >= 0) & (tokens < z.shape[-1]) & (dlogp != 0)
    one.scatter_(-1, tokens.clamp(0, z.shape[-1] - 1).long().unsqueeze(-1), 1.0)
    g = (dlogp * alpha).unsqueeze(-1) * (one - p)
    return torch.where(real.unsqueeze(-1), g, torch.zeros_like(g)), p


def logit_grad_bound(p, logits, alpha, dlogp, lse_err):
    """p is off by its exponent's error (the roundings of z, of z - lse and of the
    scaling to base 2, and lse's own) and a few U; the product adds 3 U."""
    z = logits[torch.isfinite(logits)].abs().max().item() * alpha
    V = logits.shape[-1]
    rel = U * (6 * z + 4 * np.log(V + 1.0) + 32) + lse_err
    return (dlogp * alpha).abs().unsqueeze(-1) * (p * rel + 4 * U)


def policy(logits, tokens, old, ref, adv, weight, lo, hi, beta, alpha):
    """stats [P, 4], logp [P, T], dlogp [P, T], dlogits, p; float64."""
    V = logits.shape[-1]
    logp, lse = logprob(logits, tokens, alpha)
    w = torch.ones_like(logp) if weight is None else weight
    live = (tokens >= 0) & (tokens < V) & (w != 0)
    logp = torch.where(live, logp, torch.zeros_like(logp))
    q = torch.exp(logp - old)
    plain, held = q * adv, q.clamp(1 - lo, 1 + hi) * adv
    clipped = held < plain
    pg = -torch.minimum(plain, held)
    slope = torch.where(clipped, torch.zeros_like(q), -plain)
    kl = torch.zeros_like(q)
    if ref is not None:
        d = ref - logp
        kl = torch.expm1(d) - d
        if beta:
            slope = slope - beta * torch.expm1(d)
    terms = torch.stack((pg + beta * kl if beta else pg, pg, kl, clipped.double()), -1)
    stats = torch.where(live.unsqueeze(-1), terms * w.unsqueeze(-1), torch.zeros_like(terms)).sum(1)
    dlogp = torch.where(live, w * slope, torch.zeros_like(q))
    g, p = logit_grad(logits, tokens, alpha, lse, dlogp)
    return stats, logp, dlogp, g, p
