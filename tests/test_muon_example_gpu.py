"""The example that runs the dense layers, their gradients and the Muon step together: its gradient
replicas equal autograd's in 64 bits, and a step of it runs and keeps the replicas equal."""
import os
import sys

import pytest
import torch

import gradient_sync_zero_gb300 as dps

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import muon_step  # noqa: E402

pytestmark = pytest.mark.gpu


def test_gradient_replicas_equal_autograd():
    """bf16 activations x, z, a, h and gradients of them: every value on the longest way (x, a, h, logits'
    operand, dh, da, dz, dx, the slot) is rounded by at most 2^-8 and the roundings are independent, so
    norm against norm a gradient is off by about sqrt(9) 2^-8 / sqrt(3) and less than 9 * 2^-8."""
    P, T = 3, 150
    s = muon_step.Step(P=P, T=T, V=61, D=48, F=136)
    g = torch.Generator().manual_seed(3)
    tokens, targets = (torch.randint(0, 61, (P, T), generator=g) for _ in range(2))
    s.weight(1, muon_step.B1).copy_(0.1 * torch.randn(136, generator=g))
    w = {(k, t): s.weight(k, t).double().cpu().requires_grad_() for k, t in ((0, 0), (0, 1), (0, 2), (1, 0), (1, 1))}
    x = torch.stack([w[1, 0][r][tokens[r]] for r in range(P)])
    z = x @ w[0, 0].mT + w[1, 1].unsqueeze(1)
    h = x + (z * torch.special.ndtr(z)) @ w[0, 1].mT
    logp = torch.log_softmax(h @ w[0, 2].mT, -1).gather(-1, targets.unsqueeze(-1)).squeeze(-1)
    dlogp = torch.randn(P, T, generator=g) / T
    (logp * dlogp).sum().backward()
    got = s.forward(tokens.cuda(), targets.cuda())
    assert (got.double().cpu() - logp.detach()).norm() <= 4 * 2.0 ** -8 * logp.detach().norm()
    s.backward(tokens.cuda(), targets.cuda(), dlogp.cuda())
    for (k, t), v in w.items():
        err = (s.grad(k, t).double().cpu() - v.grad).norm() / v.grad.norm()
        assert err <= 9 * 2.0 ** -8, (k, t, float(err))


def test_steps_run_and_replicas_stay_equal():
    s = muon_step.Step(P=2, T=64, V=37, D=72, F=300)
    g = torch.Generator(device="cuda").manual_seed(4)
    for _ in range(3):
        tokens = torch.randint(0, 37, (2, 64), generator=g, device="cuda")
        before = [m.clone() for m in s.master]
        s.forward(tokens, tokens)
        s.backward(tokens, tokens, torch.full((2, 64), -1 / 64, device="cuda"))
        s.update()
        for k in range(2):
            L = s.plans[k].L
            assert torch.isfinite(s.master[k]).all() and not torch.equal(s.master[k], before[k])
            assert torch.equal(s.params[k][0, :L], s.params[k][1, :L])
            for t, shape in enumerate((s.matrices, s.others)[k]):
                a = s.plans[k].tensor_view(s.master[k], t, shape)
                assert torch.equal(s.weight(k, t)[0], a.to(torch.bfloat16))
    assert dps.dp_read_norm(s.plans[0], s.ws[0])[2] == 0 and dps.dp_product_timeouts() == 0
