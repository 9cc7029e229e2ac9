"""A training step whose dense layers run on the replicas and whose matrices Muon updates.

P virtual ranks hold a tiny next-token model: an embedding E, a block h = x + W2 gelu(W1 x + b1)
and a head H.  Two bucket plans, as two optimisers have: the matrices W1, W2 and H in
one, what AdamW trains (E and b1) in the other.

    x = E[tokens]                                   dp_embedding_forward
    a = gelu(x W1^T + b1)                            dp_linear_forward, its argument kept
    h = x + a W2^T                                   dp_linear_forward with the residual
    logits = h H^T                                   dp_linear_forward
    loss = -mean log p(target)                       dp_token_logprob and its gradient
    dH, dh;  dW2, da;  dW1, db1, dx                  dp_linear_backward, into their slots
    dE                                               dp_embedding_backward, into its slot
    W1, W2, H <- Muon on the mean over the ranks     dp_reduce_scatter_mean, dp_muon_step
    E, b1 <- AdamW                                   dp_fused_zero_step

Run: python examples/muon_step.py
"""
from __future__ import annotations

import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gradient_sync_zero_gb300 as dps  # noqa: E402

W1, W2, HEAD = 0, 1, 2
EMBED, B1 = 0, 1


class Step:
    def __init__(self, P=4, T=256, V=96, D=64, F=160, seed=1):
        self.P, self.T, self.V, self.D, self.F = P, T, V, D, F
        self.matrices = ((F, D), (D, F), (V, D))
        self.others = ((V, D), (F,))
        self.plans = [dps.Plan([math.prod(s) for s in shapes], bucket_bytes=16 << 10, P=P)
                      for shapes in (self.matrices, self.others)]
        self.ws = [p.new_workspace() for p in self.plans]
        self.params = [p.new_replicas() for p in self.plans]
        self.grads = [p.new_replicas() for p in self.plans]
        self.master = [p.new_state() for p in self.plans]
        self.m = [p.new_state() for p in self.plans]          # Muon's momentum, AdamW's m
        self.mean, self.v = self.plans[0].new_state(), self.plans[1].new_state()
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.gen = g
        for k, shapes in enumerate((self.matrices, self.others)):
            for t, shape in enumerate(shapes):
                w = torch.randn(*shape, generator=g, device="cuda") / math.sqrt(shape[-1])
                if len(shape) == 1:
                    w.zero_()
                self.plans[k].tensor_view(self.master[k], t, shape).copy_(w)
                self.weight(k, t).copy_(w.to(torch.bfloat16))          # every rank's replica
        self.muon = dps.Muon(self.plans[0], dict(enumerate(self.matrices)))
        self.muon_ws = self.muon.new_workspace()
        bf = dict(dtype=torch.bfloat16, device="cuda")
        self.x, self.h, self.dh, self.dx = (torch.empty(P, T, D, **bf) for _ in range(4))
        self.z, self.a, self.da = (torch.empty(P, T, F, **bf) for _ in range(3))
        self.logits = torch.empty(P, T, V, device="cuda")
        self.logp, self.lse = (torch.empty(P, T, device="cuda") for _ in range(2))
        self.embed_ws = dps.new_embedding_workspace(P, T, V, D)
        ins = ((self.x, W1), (self.a, W2), (self.h, HEAD))
        self.fwd_ws = [dps.new_linear_workspace(x, self.weight(0, t)) for x, t in ins]
        self.bwd_ws = [dps.new_linear_workspace(x, self.weight(0, t), backward=True) for x, t in ins]
        self.t = 0

    def _view(self, bufs, k, t):
        return self.plans[k].tensor_view(bufs[k], t, (self.matrices, self.others)[k][t])

    def weight(self, k, t):
        """Tensor t of plan k of every rank, a view of the parameter replicas."""
        return self._view(self.params, k, t)

    def grad(self, k, t):
        """Its slot of the gradient replicas."""
        return self._view(self.grads, k, t)

    def forward(self, tokens, targets):
        """Log-probabilities [P, T] of the targets."""
        dps.dp_embedding_forward(self.weight(1, EMBED), tokens, self.x)
        dps.dp_linear_forward(self.x, self.weight(0, W1), self.a, bias=self.weight(1, B1), z=self.z,
                              act=dps.DP_ACT_GELU, ws=self.fwd_ws[W1])
        dps.dp_linear_forward(self.a, self.weight(0, W2), self.h, residual=self.x, ws=self.fwd_ws[W2])
        dps.dp_linear_forward(self.h, self.weight(0, HEAD), self.logits, ws=self.fwd_ws[HEAD])
        dps.dp_token_logprob(self.logits, targets, self.logp, self.lse)
        return self.logp

    def backward(self, tokens, targets, dlogp):
        """Every gradient slot of the last forward."""
        dps.dp_token_logprob_backward(self.logits, targets, self.lse, dlogp, self.logits)
        dps.dp_linear_backward(self.logits, self.h, self.weight(0, HEAD), dx=self.dh,
                               dw=self.grad(0, HEAD), ws=self.bwd_ws[HEAD])
        dps.dp_linear_backward(self.dh, self.a, self.weight(0, W2), dx=self.da, dw=self.grad(0, W2),
                               ws=self.bwd_ws[W2])
        dps.dp_linear_backward(self.da, self.x, self.weight(0, W1), dx=self.dx, dw=self.grad(0, W1),
                               dbias=self.grad(1, B1), z=self.z, act=dps.DP_ACT_GELU,
                               ws=self.bwd_ws[W1])
        self.dx += self.dh                       # the residual's gradient
        dps.dp_embedding_backward(self.dx, tokens, self.grad(1, EMBED), self.embed_ws)

    def update(self, lr=0.02):
        self.t += 1
        dps.dp_reduce_scatter_mean(self.plans[0], self.ws[0], self.grads[0], self.mean)
        dps.dp_muon_step(self.muon, self.ws[0], self.muon_ws, self.mean, self.master[0], self.m[0],
                         self.params[0], dps.muon_cfg(lr=lr, weight_decay=0.0))
        dps.dp_fused_zero_step(self.plans[1], self.ws[1], self.grads[1], self.params[1],
                               self.master[1], self.m[1], self.v,
                               dps.adamw_cfg(lr=lr, weight_decay=0.0, step=self.t))


def train(steps=50, **kw):
    """Mean loss of each step, predicting (5 t + 3) mod V from t."""
    s = Step(**kw)
    dlogp = torch.full((s.P, s.T), -1.0 / s.T, device="cuda")
    losses = []
    for _ in range(steps):
        tokens = torch.randint(0, s.V, (s.P, s.T), generator=s.gen, device="cuda")
        targets = (5 * tokens + 3) % s.V
        losses.append(-s.forward(tokens, targets).mean())
        s.backward(tokens, targets, dlogp)
        s.update()
    for plan, ws in zip(s.plans, s.ws):
        dps.dp_read_norm(plan, ws)               # raises what a kernel of the plan reported
    assert dps.dp_product_timeouts() == 0        # of the layers, which have no plan
    return torch.stack(losses).tolist()


if __name__ == "__main__":
    for i, loss in enumerate(train(steps=101)):
        if i % 20 == 0:
            print(f"step {i:4d}  loss {loss:.3f}")
