"""A policy-gradient step of data-parallel training, from tokens to updated replicas.

P virtual ranks hold the same tiny language model in the parameter replicas of a
bucket plan: an embedding E, one residual block h = x + dropout(x W) and a head H.
Every step each rank samples one token per position, is rewarded where it hits the
position's goal, and takes a few clipped steps on its sample:

    x = dropout(sqrt(D) E[tokens])                  dp_embedding_forward
    h = x + dropout(x W)                            dp_dropout
    logits = h H^T                                  a matrix product per rank
    loss, dlogits                                   dp_policy_loss (dlogits over logits)
    dH = dlogits^T h, dh = dlogits H                matrix products, dH into its slot
    dW = x^T dropout'(dh), dx = dh + dropout'(dh) W^T   dp_dropout
    dE = the sorted sums of dropout'(dx)            dp_embedding_backward, into its slot
    E, W, H <- AdamW on the mean over the ranks     dp_fused_zero_step

The gradients land in the gradient replicas themselves; nothing is gathered or
copied before the synchronisation.  Run: python examples/policy_step.py
"""
from __future__ import annotations

import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gradient_sync_zero_gb300 as dps  # noqa: E402

EMBED, BLOCK, HEAD = 0, 1, 2


class Step:
    def __init__(self, P=4, T=256, V=61, D=64, p=0.1, seed=1, act=torch.bfloat16):
        self.P, self.T, self.V, self.D, self.p, self.seed, self.act = P, T, V, D, p, seed, act
        self.plan = dps.Plan([V * D, D * D, V * D], bucket_bytes=16 << 10, P=P)
        self.ws = self.plan.new_workspace()
        self.params, self.grads = self.plan.new_replicas(), self.plan.new_replicas()
        self.master, self.m, self.v = (self.plan.new_state() for _ in range(3))
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.gen = g
        for t, shape in enumerate(((V, D), (D, D), (V, D))):
            w = torch.randn(*shape, generator=g, device="cuda") / math.sqrt(D)
            self.plan.tensor_view(self.master, t, shape).copy_(w)
            self.weight(t).copy_(w.to(torch.bfloat16))          # every rank's replica
        self.embed_ws = dps.new_embedding_workspace(P, T, V, D)
        self.x, self.block, self.h, self.dx = (torch.empty(P, T, D, dtype=act, device="cuda")
                                               for _ in range(4))
        self.logits = torch.empty(P, T, V, dtype=act, device="cuda")
        self.logp = torch.empty(P, T, device="cuda")
        self.stats = torch.empty(P, 4, device="cuda")
        self.cfg = dps.policy_cfg(clip_low=0.2, clip_high=0.2, kl_beta=0.01)
        self.t = 0

    def _view(self, buf, t):
        return self.plan.tensor_view(buf, t, (self.D, self.D) if t == BLOCK else (self.V, self.D))

    def weight(self, t):
        """Weight t of every rank, a view of the parameter replicas."""
        return self._view(self.params, t)

    def grad(self, t):
        """Its slot of the gradient replicas."""
        return self._view(self.grads, t)

    def _drops(self, draw):
        """The two dropouts of one forward: offsets 2 * draw and 2 * draw + 1."""
        return (dps.dropout_cfg(self.p, self.seed, 2 * draw),
                dps.dropout_cfg(self.p, self.seed, 2 * draw + 1))

    def forward(self, tokens, draw):
        d_embed, d_block = self._drops(draw)
        dps.dp_embedding_forward(self.weight(EMBED), tokens, self.x, scale=math.sqrt(self.D),
                                 dropout=d_embed)
        torch.matmul(self.x, self.weight(BLOCK).to(self.act), out=self.block)
        dps.dp_dropout(self.block, self.h, d_block, residual=self.x)
        torch.matmul(self.h, self.weight(HEAD).to(self.act).transpose(1, 2), out=self.logits)
        return self.logits

    def backward(self, tokens, sampled, old_logp, advantage, ref_logp, weight, draw):
        """Loss statistics [P, 4] of the last forward, and every gradient slot."""
        d_embed, d_block = self._drops(draw)
        dps.dp_policy_loss(self.logits, sampled, old_logp, advantage, self.logp, self.stats,
                           dlogits=self.logits, ref_logp=ref_logp, weight=weight, cfg=self.cfg)
        dlogits = self.logits
        self.grad(HEAD).copy_(torch.matmul(dlogits.transpose(1, 2), self.h))
        torch.matmul(dlogits, self.weight(HEAD).to(self.act), out=self.dx)
        dps.dp_dropout(self.dx, self.block, d_block)
        self.grad(BLOCK).copy_(torch.matmul(self.x.transpose(1, 2), self.block))
        self.dx += torch.matmul(self.block, self.weight(BLOCK).to(self.act).transpose(1, 2))
        dps.dp_embedding_backward(self.dx, tokens, self.grad(EMBED), self.embed_ws,
                                  scale=math.sqrt(self.D), dropout=d_embed)
        return self.stats

    def update(self, lr=3e-3):
        self.t += 1
        cfg = dps.adamw_cfg(lr=lr, weight_decay=0.0, max_norm=1.0, step=self.t)
        dps.dp_fused_zero_step(self.plan, self.ws, self.grads, self.params, self.master, self.m,
                               self.v, cfg)


def train(steps=60, inner=2, **kw):
    """Mean reward of each step."""
    s = Step(**kw)
    P, T, V = s.P, s.T, s.V
    weight = torch.full((P, T), 1.0 / T, device="cuda")
    ref_logp = None
    rewards = []
    for step in range(steps):
        tokens = torch.randint(0, V, (P, T), generator=s.gen, device="cuda")
        goal = (5 * tokens + 3) % V
        draw = step * (inner + 1)
        probs = torch.softmax(s.forward(tokens, draw).float(), -1)
        sampled = torch.multinomial(probs.flatten(0, 1), 1, generator=s.gen).view(P, T)
        old_logp = torch.empty(P, T, device="cuda")
        dps.dp_token_logprob(s.logits, sampled, old_logp)
        ref_logp = old_logp              # the policy before this step's updates
        reward = (sampled == goal).float()
        rewards.append(reward.mean())
        advantage = (reward - reward.mean()) * V ** 0.5
        for k in range(inner):
            s.forward(tokens, draw + k)
            s.backward(tokens, sampled, old_logp, advantage, ref_logp, weight, draw + k)
            s.update()
    return torch.stack(rewards).tolist()


if __name__ == "__main__":
    history = train(steps=200)
    for i in range(0, len(history), 20):
        print(f"step {i:4d}  mean reward {history[i]:.3f}")
    print(f"step {len(history) - 1:4d}  mean reward {history[-1]:.3f}")
