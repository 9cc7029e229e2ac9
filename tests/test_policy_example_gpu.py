"""The example that runs the step's operators together: its gradient replicas equal
autograd's in 64 bits, its training learns, and every operator's indexes hold under the
library built with index checks."""
import os
import subprocess
import sys

import pytest
import torch

import gradient_sync_zero_gb300 as dps
import model_reference as ref

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import policy_step  # noqa: E402

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_gradient_replicas_equal_autograd():
    """fp32 activations, so each gradient is off by its own bf16 rounding (2^-8) and
    fp32 sums of at most T + V terms."""
    P, T, V, D, p, draw = 3, 40, 61, 32, 0.2, 7
    s = policy_step.Step(P=P, T=T, V=V, D=D, p=p, act=torch.float32)
    g = torch.Generator().manual_seed(5)
    tokens = torch.randint(0, V, (P, T), generator=g)
    tokens[1, :3] = -1                                       # padding
    sampled = torch.randint(0, V, (P, T), generator=g)
    adv = torch.randn(P, T, generator=g)
    w = torch.rand(P, T, generator=g) / T
    w[2, :10] = 0.0
    weights = [s.weight(t).double().cpu().requires_grad_() for t in range(3)]

    def keep(off):
        return ref.keep_mask(P, T * D, p, s.seed, off).view(P, T, D) / (1 - p)

    real = (tokens >= 0).unsqueeze(-1)
    E, W, H = weights
    x = torch.stack([E[r][tokens[r].clamp(0)] for r in range(P)]) * D ** 0.5 * real * keep(2 * draw)
    h = x + (x @ W) * keep(2 * draw + 1)
    logits = h @ H.transpose(1, 2)
    logp = torch.log_softmax(logits, -1).gather(-1, sampled.unsqueeze(-1)).squeeze(-1)
    old = (logp.detach() - 0.05 * torch.randn(P, T, generator=g, dtype=torch.float64)).float()
    refl = (logp.detach() + 0.2 * torch.randn(P, T, generator=g, dtype=torch.float64)).float()
    q = torch.exp(logp - old)
    pg = -torch.minimum(q * adv, q.clamp(0.8, 1.2) * adv)
    d = refl - logp
    row = pg + 0.01 * (torch.expm1(d) - d)
    loss = torch.where(w != 0, w * row, torch.zeros_like(row)).sum(1)
    loss.sum().backward()

    s.forward(tokens.cuda(), draw)
    stats = s.backward(tokens.cuda(), sampled.cuda(), old.cuda(), adv.cuda(), refl.cuda(), w.cuda(), draw)
    assert (stats[:, 0].double().cpu() - loss.detach()).abs().max() < 1e-5 * loss.detach().abs().max() + 1e-6
    for t, name in ((policy_step.EMBED, "E"), (policy_step.BLOCK, "W"), (policy_step.HEAD, "H")):
        got, want = s.grad(t).double().cpu(), weights[t].grad
        scale = want.abs().max()
        assert ((got - want).abs() <= 2.0 ** -8 * want.abs() + 1e-5 * scale).all(), name
    unnamed = torch.ones(P, V, dtype=torch.bool)
    for r in range(P):
        unnamed[r, tokens[r][tokens[r] >= 0]] = False
    assert (s.grad(policy_step.EMBED).cpu()[unnamed] == 0).all()


def test_training_learns():
    history = policy_step.train(steps=120, T=512, V=23, D=32)
    first, last = sum(history[:5]) / 5, sum(history[-5:]) / 5
    assert first < 0.15 and last > 0.5, (first, last)


@pytest.mark.skipif(os.environ.get("DPSYNC_VARIANT") == "checked", reason="this test starts the checked run")
def test_operators_under_index_checks():
    from gradient_sync_zero_gb300 import build as dbuild
    dbuild.build(checked=True)
    env = dict(os.environ, DPSYNC_VARIANT="checked")
    r = subprocess.run([sys.executable, "-m", "pytest", "-m", "gpu", "-x", "-q", "-p", "no:cacheprovider",
                        "tests/test_model_ops_gpu.py", "-k", "gradient or step or lookup"],
                       cwd=ROOT, env=env, capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, r.stdout[-4000:] + r.stderr[-2000:]
    assert " passed" in r.stdout and " failed" not in r.stdout
