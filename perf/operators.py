"""The operators at the two ends of a training step, as cases to measure.

Embedding lookup and its gradient, dropout, token log-probabilities and their
gradient, and the clipped policy loss, each over P data-parallel replicas whose
parameters and gradients lie in the replica buffers of a bucket plan.

``run`` computes a case either in its plain form (elementary torch operations in
32 bits) or, with ``own`` set, through the package's operators.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}
ZIPF = 2.7          # token v is drawn with probability ~ 1 / (v + ZIPF): a few tokens are very frequent
LEARN = 0.02        # standard deviation of embedding weights


# ----------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------
def listed():
    return [
        # one new token looked up while sampling a completion (latency)
        dict(name="lookup one token", op="lookup", P=1, T=1, V=32000, D=2048, dtype="bf16",
             scale=1.0, p=0.0, pad=0.0),
        # GPT-2 small, 8 replicas x 8 sequences of 1024, with its embedding dropout
        dict(name="lookup gpt2 dropout", op="lookup", P=8, T=8192, V=50257, D=768, dtype="bf16",
             scale=1.0, p=0.1, pad=0.02),
        # odd sizes, fp32 activations, a scaled embedding (sqrt(D)) and padding
        dict(name="embedding grad odd", op="lookup_grad", P=4, T=777, V=1009, D=131, dtype="f32",
             scale=math.sqrt(131.0), p=0.1, pad=0.1),
        # the 1.1B model's embedding gradient: 8 replicas x 8 sequences of 2048
        dict(name="embedding grad llama", op="lookup_grad", P=8, T=16384, V=32000, D=2048,
             dtype="bf16", scale=1.0, p=0.0, pad=0.0),
        # residual dropout of one GPT-2 small block over 8 replicas
        dict(name="dropout gpt2 residual", op="dropout", P=8, T=8192, D=768, dtype="bf16", p=0.1,
             residual=True),
        # the backward of a dropout over odd sizes in fp32
        dict(name="dropout grad odd", op="dropout", P=3, T=333, D=257, dtype="f32", p=0.25,
             residual=False),
        # the log-probabilities of a few sampled tokens (latency; rows longer than the batch is wide)
        dict(name="logprob 4 rows", op="logprob", P=1, T=4, V=50257, dtype="bf16", alpha=1.25),
        # the reference model's log-probabilities of a batch: 8 replicas x 2048 tokens
        dict(name="logprob llama", op="logprob", P=8, T=2048, V=32000, dtype="bf16", alpha=1.0),
        # cross-entropy's gradient over an odd vocabulary (rows that no vector load is aligned to)
        dict(name="logprob grad gpt2", op="logprob_grad", P=8, T=1024, V=50257, dtype="bf16",
             alpha=1.0, masked=0.1),
        # the same in fp32, a short sequence
        dict(name="logprob grad f32", op="logprob_grad", P=2, T=17, V=32000, dtype="f32",
             alpha=1.0, masked=0.0),
        # a toy policy step: small vocabulary, fp32, no prompt
        dict(name="policy small f32", op="policy", P=4, T=33, V=1000, dtype="f32", alpha=1.0,
             masked=0.0, beta=0.05, lo=0.2, hi=0.2),
        # a policy step of the 2.5B model's head: 8 replicas x 2048 tokens, a quarter of them prompt
        dict(name="policy 50304", op="policy", P=8, T=2048, V=50304, dtype="bf16", alpha=1.0,
             masked=0.25, beta=0.04, lo=0.2, hi=0.28),
    ]


_MOST = 2.6e9           # bytes of work of the largest drawn case
_MOST_DROPPED = 6.0e7   # values of the largest drawn case with dropout


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    while True:
        op = rng.choice(["lookup", "lookup_grad", "dropout", "logprob", "logprob_grad", "policy"])
        c = dict(op=op, P=rng.choice([1, 2, 3, 4, 8]), T=_log_int(rng, 1, 16384),
                 dtype=rng.choice(["bf16", "bf16", "f32"]))
        if op in ("lookup", "lookup_grad"):
            c.update(V=rng.choice([50257, 32000, 50304, _log_int(rng, 97, 131072)]),
                     D=rng.choice([768, 2048, 2560, _log_int(rng, 16, 4096)]),
                     scale=rng.choice([1.0, 8.5]), p=rng.choice([0.0, 0.0, 0.1, 0.35]),
                     pad=rng.choice([0.0, 0.05, 0.4]))
        elif op == "dropout":
            c.update(D=rng.choice([768, 2048, 2560, _log_int(rng, 1, 8192)]),
                     p=rng.choice([0.05, 0.1, 0.25, 0.5]), residual=rng.random() < 0.5)
        else:
            c.update(V=rng.choice([50257, 32000, 50304, _log_int(rng, 97, 131072)]),
                     alpha=rng.choice([1.0, 1.0, 0.7, 1.25]))
            if op != "logprob":
                c.update(masked=rng.choice([0.0, 0.25, 0.5, 0.9]))
            if op == "policy":
                c.update(beta=rng.choice([0.0, 0.04, 0.1]), lo=0.2, hi=rng.choice([0.2, 0.28]))
        if work(c)["bytes"] > _MOST:
            continue
        # random words cost the plain form far more than the values they mask
        if not c.get("p") or c["P"] * c["T"] * c["D"] <= _MOST_DROPPED:
            return c


def _kept_rows(case):
    """Rows of one rank whose weight is not zero: in every 64 rows the first
    `masked` share belongs to the prompt."""
    T, prompt = case["T"], round(64 * case["masked"])
    return T - (T // 64) * prompt - min(T % 64, prompt)


def _pads(case):
    return int(case["T"] * case["pad"])


def _distinct(case):
    """Expected number of different rows that one rank's tokens look up."""
    V, n = case["V"], case["T"] - _pads(case)
    v = np.arange(V, dtype=np.float64)
    pv = np.log((v + 1 + ZIPF) / (v + ZIPF)) / math.log((V + ZIPF) / ZIPF)
    return float(np.sum(-np.expm1(n * np.log1p(-pv))))


def work(case):
    op, P, T, es = case["op"], case["P"], case["T"], SIZE[case["dtype"]]
    if op == "lookup":
        row = case["D"] * es
        return {"bytes": P * (_distinct(case) * row + T * row + 8 * T), "flops": P * T * case["D"]}
    if op == "lookup_grad":
        row, n = case["D"] * es, T - _pads(case)
        return {"bytes": P * (n * row + case["V"] * row + 8 * T), "flops": 2 * P * n * case["D"]}
    if op == "dropout":
        n = P * T * case["D"]
        return {"bytes": (3 if case["residual"] else 2) * es * n, "flops": 2 * n}
    n, V = P * T, case["V"]
    if op == "logprob":
        return {"bytes": n * (V * es + 8 + 8), "flops": 4 * n * V}
    k = P * _kept_rows(case)
    if op == "logprob_grad":
        return {"bytes": k * V * es + n * (V * es + 8 + 8), "flops": 4 * k * V}
    return {"bytes": k * V * es + n * (V * es + 8 + 20), "flops": 8 * k * V}


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------
def _tokens(case, g):
    """[P, T] int64, Zipf-like; the last `pad` share of each rank's tokens is -1."""
    V = case["V"]
    u = torch.rand(case["P"], case["T"], generator=g, device="cuda", dtype=torch.float64)
    t = (ZIPF * ((V + ZIPF) / ZIPF) ** u - ZIPF).floor().clamp_(0, V - 1).to(torch.int64)
    n = _pads(case) if "pad" in case else 0
    if n:
        t[:, case["T"] - n:] = -1
    return t


def _slot(case):
    """Offset and replica stride (elements) of the embedding inside replicas that
    hold other tensors too, as a bucket plan lays them out."""
    n = -(-case["V"] * case["D"] // 8) * 8
    off = 1024
    return off, -(-(off + n + 512) // 128) * 128


def _replica_view(buf, case):
    off, _ = _slot(case)
    V, D = case["V"], case["D"]
    return buf[:, off:off + V * D].unflatten(1, (V, D))


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, P, T, dt = case["op"], case["P"], case["T"], DTYPES[case["dtype"]]

    def normal(*shape, dtype=dt, std=1.0):
        return torch.randn(*shape, generator=g, device="cuda", dtype=dtype).mul_(std)

    s = dict(case=dict(case), seed=int(seed) * 2654435761 % (1 << 62) + 1, offset=int(seed) % 977)
    if op in ("lookup", "lookup_grad"):
        _, stride = _slot(case)
        s["tokens"] = _tokens(case, g)
        if op == "lookup":
            s["params"] = normal(P, stride, std=LEARN)
            s["out"] = torch.empty(P, T, case["D"], dtype=dt, device="cuda")
        else:
            s["dx"] = normal(P, T, case["D"], std=1e-2)
            s["grads"] = torch.zeros(P, stride, dtype=dt, device="cuda")
        return s
    if op == "dropout":
        s["x"] = normal(P, T, case["D"])
        s["out"] = torch.empty_like(s["x"])
        s["residual"] = normal(P, T, case["D"]) if case["residual"] else None
        return s
    V = case["V"]
    logits = normal(P, T, V, std=2.0)
    tokens = torch.randint(0, V, (P, T), generator=g, device="cuda")
    # a sampled token is a likely one
    lift = normal(P, T, 1, dtype=torch.float32, std=3.0).add_(9.0)
    at = tokens.unsqueeze(-1)
    logits.scatter_(-1, at, (logits.gather(-1, at).float() + lift).to(dt))
    s.update(logits=logits, tokens=tokens)
    if op == "logprob":
        s["logp"] = torch.empty(P, T, dtype=torch.float32, device="cuda")
        s["lse"] = torch.empty(P, T, dtype=torch.float32, device="cuda")
        return s
    keep = (torch.arange(T, device="cuda") % 64) >= round(64 * case["masked"])
    weight = keep.float().div_(max(1, _kept_rows(case))).expand(P, T).contiguous()
    s["dlogits"] = torch.empty_like(logits)
    if op == "logprob_grad":
        # the forward's result, one rank at a time
        s["lse"] = torch.stack([_logprob(x, t, case["alpha"])[1] for x, t in zip(logits, tokens)])
        s["dlogp"] = -weight
        return s
    logp = torch.stack([_logprob(x, t, case["alpha"])[0] for x, t in zip(logits, tokens)])
    # a policy that moved a little since it sampled, and a little more from its reference; no
    # ratio lies within rounding of a clip bound, where the gradient jumps
    moved = normal(P, T, dtype=torch.float32, std=0.15)
    for bound in (math.log(1.0 - case["lo"]), math.log(1.0 + case["hi"])):
        near = (moved - bound).abs() < 1e-3
        moved = torch.where(near, moved + 4e-3, moved)
    s["old"] = logp - moved
    s["ref"] = logp + normal(P, T, dtype=torch.float32, std=0.3)
    # one advantage for each 64 tokens
    adv = normal(P, -(-T // 64), dtype=torch.float32)
    s["adv"] = adv.repeat_interleave(64, 1)[:, :T].contiguous()
    s["weight"] = weight
    s["logp"] = torch.empty(P, T, dtype=torch.float32, device="cuda")
    s["stats"] = torch.empty(P, 4, dtype=torch.float32, device="cuda")
    return s


# ----------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------
def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    import gradient_sync_zero_gb300 as dps
    c = s["case"]
    op = c["op"]
    drop = dps.dropout_cfg(c["p"], s["seed"], s["offset"]) if c.get("p") else None
    if op == "lookup":
        dps.dp_embedding_forward(_replica_view(s["params"], c), s["tokens"], s["out"],
                                 scale=c["scale"], dropout=drop)
        return s["out"]
    if op == "lookup_grad":
        grad = _replica_view(s["grads"], c)
        if "ws" not in s:
            s["ws"] = dps.new_embedding_workspace(c["P"], c["T"], c["V"], c["D"])
        dps.dp_embedding_backward(s["dx"], s["tokens"], grad, s["ws"], scale=c["scale"],
                                  dropout=drop)
        return grad
    if op == "dropout":
        dps.dp_dropout(s["x"], s["out"], drop, residual=s["residual"])
        return s["out"]
    if op == "logprob":
        dps.dp_token_logprob(s["logits"], s["tokens"], s["logp"], s["lse"],
                             logit_scale=c["alpha"])
        return s["logp"], s["lse"]
    if op == "logprob_grad":
        dps.dp_token_logprob_backward(s["logits"], s["tokens"], s["lse"], s["dlogp"],
                                      s["dlogits"], logit_scale=c["alpha"])
        return s["dlogits"]
    cfg = dps.policy_cfg(clip_low=c["lo"], clip_high=c["hi"], kl_beta=c["beta"],
                         logit_scale=c["alpha"])
    dps.dp_policy_loss(s["logits"], s["tokens"], s["old"], s["adv"], s["logp"], s["stats"],
                       dlogits=s["dlogits"], ref_logp=s["ref"], weight=s["weight"], cfg=cfg)
    return s["stats"], s["logp"], s["dlogits"]


def _mul_hi_lo(a, m):
    """High and low 32 bits of the product of 32-bit words held in int64."""
    x = a * m                                  # wraps modulo 2**64
    return (x >> 32) & 0xFFFFFFFF, x & 0xFFFFFFFF


def _keep(P, n, p, seed, offset):
    """[P, n] bool: Philox4x32-10 (Salmon et al., "Parallel random numbers: as easy
    as 1, 2, 3", 2011), element i from word i % 4 of counter (i // 4, rank, offset)."""
    b = torch.arange(-(-n // 4), device="cuda", dtype=torch.int64).expand(P, -1)
    r = torch.arange(P, device="cuda", dtype=torch.int64).unsqueeze(1).expand_as(b)
    c0, c1, c2, c3 = b & 0xFFFFFFFF, b >> 32, r, torch.full_like(b, offset)
    k0, k1 = seed & 0xFFFFFFFF, seed >> 32
    for _ in range(10):
        h0, l0 = _mul_hi_lo(c0, 0xD2511F53)
        h1, l1 = _mul_hi_lo(c2, 0xCD9E8D57)
        c0, c1, c2, c3 = h1 ^ c1 ^ k0, l1, h0 ^ c3 ^ k1, l0
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    words = torch.stack((c0, c1, c2, c3), dim=-1).flatten(1)[:, :n]
    return words >= round(p * 2 ** 32)


def _drop(x, s, case):
    """x [P, T, D] fp32 after dropout."""
    if not case.get("p"):
        return x
    keep = _keep(x.shape[0], x.shape[1] * x.shape[2], case["p"], s["seed"], s["offset"])
    return torch.where(keep.view_as(x), x * (1.0 / (1.0 - case["p"])), 0.0)


def _logprob(x, tokens, alpha):
    z = x.float() * alpha
    m = z.amax(-1, keepdim=True)
    log_sum = torch.exp(z - m).sum(-1).log()
    m = m.squeeze(-1)
    return z.gather(-1, tokens.unsqueeze(-1)).squeeze(-1) - m - log_sum, m + log_sum


def _logit_grad(x, tokens, lse, dlogp, alpha):
    g = torch.exp(x.float() * alpha - lse.unsqueeze(-1)).mul_(-dlogp.unsqueeze(-1) * alpha)
    at = tokens.unsqueeze(-1)
    g.scatter_(-1, at, g.gather(-1, at) + dlogp.unsqueeze(-1) * alpha)
    return torch.where(dlogp.unsqueeze(-1) == 0, 0.0, g)


def _run_plain(s):
    c = s["case"]
    op, dt = c["op"], DTYPES[c["dtype"]]
    if op in ("lookup", "lookup_grad"):
        P, V, D = c["P"], c["V"], c["D"]
        real = (s["tokens"] >= 0) & (s["tokens"] < V)
        tok = torch.where(real, s["tokens"], 0)
        rank = torch.arange(P, device="cuda").unsqueeze(1)
        if op == "lookup":
            x = _replica_view(s["params"], c)[rank, tok].float() * c["scale"]
            return _drop(torch.where(real.unsqueeze(-1), x, 0.0), s, c).to(dt)
        dx = _drop(s["dx"].float(), s, c) * c["scale"]
        dx = torch.where(real.unsqueeze(-1), dx, 0.0)
        dw = torch.zeros(P * V, D, device="cuda", dtype=torch.float32)
        dw.index_add_(0, (rank * V + tok).flatten(), dx.flatten(0, 1))
        return dw.to(dt).view(P, V, D)
    if op == "dropout":
        y = _drop(s["x"].float(), s, c)
        return (y + s["residual"].float() if c["residual"] else y).to(dt)
    if op == "logprob":
        return _logprob(s["logits"], s["tokens"], c["alpha"])
    if op == "logprob_grad":
        return _logit_grad(s["logits"], s["tokens"], s["lse"], s["dlogp"], c["alpha"]).to(dt)
    logp, lse = _logprob(s["logits"], s["tokens"], c["alpha"])
    w = s["weight"]
    logp = torch.where(w == 0, 0.0, logp)
    ratio = torch.exp(logp - s["old"])
    plain, clipped = ratio * s["adv"], ratio.clamp(1.0 - c["lo"], 1.0 + c["hi"]) * s["adv"]
    d = s["ref"] - logp
    pg, kl = -torch.minimum(plain, clipped), torch.expm1(d) - d
    dlogp = torch.where(clipped < plain, 0.0, -plain) - c["beta"] * torch.expm1(d)
    terms = torch.stack((pg + c["beta"] * kl, pg, kl, (clipped < plain).float()), dim=-1)
    live = (w != 0).unsqueeze(-1)
    stats = torch.where(live, terms * w.unsqueeze(-1), 0.0).sum(1)
    dlogp = torch.where(w == 0, 0.0, dlogp * w)
    return stats, logp, _logit_grad(s["logits"], s["tokens"], lse, dlogp, c["alpha"]).to(dt)


# ----------------------------------------------------------------------------
# the definition in 64 bits
# ----------------------------------------------------------------------------
def _exact_keep(P, n, p, seed, offset):
    """[P, n] on the host, with unsigned words."""
    lim, m32 = np.uint64(round(p * 2 ** 32)), np.uint64(0xFFFFFFFF)
    out = np.empty((P, n), dtype=bool)
    for r in range(P):
        x = np.zeros((4, -(-n // 4)), dtype=np.uint64)
        x[0] = np.arange(x.shape[1], dtype=np.uint64)
        x[2], x[3] = np.uint64(r), np.uint64(offset)
        key = [seed & 0xFFFFFFFF, seed >> 32]
        for _ in range(10):
            a, b = x[0] * np.uint64(0xD2511F53), x[2] * np.uint64(0xCD9E8D57)
            x = np.stack(((b >> np.uint64(32)) ^ x[1] ^ np.uint64(key[0]), b & m32,
                          (a >> np.uint64(32)) ^ x[3] ^ np.uint64(key[1]), a & m32))
            key = [(key[0] + 0x9E3779B9) % 2 ** 32, (key[1] + 0xBB67AE85) % 2 ** 32]
        out[r] = x.T.reshape(-1)[:n] >= lim
    return out


def exact(case, seed):
    c, op, P, T = case, case["op"], case["P"], case["T"]
    s = prepare(case, seed)
    f64 = torch.float64
    factor = None
    if c.get("p"):
        D = c["D"]
        keep = torch.from_numpy(_exact_keep(P, T * D, c["p"], s["seed"], s["offset"])).cuda()
        factor = keep.view(P, T, D)          # bool; scaled where it is used
    gone = 1.0 - c.get("p", 0.0)
    if op == "dropout":
        y = s["x"].to(f64).div_(gone)
        y[~factor] = 0.0
        return y if s["residual"] is None else y.add_(s["residual"].to(f64))
    if op == "lookup":
        y = torch.zeros(P, T, c["D"], dtype=f64, device="cuda")
        for r in range(P):
            rows = ((s["tokens"][r] >= 0) & (s["tokens"][r] < c["V"])).nonzero().squeeze(1)
            w = _replica_view(s["params"], c)[r].index_select(0, s["tokens"][r][rows])
            y[r, rows] = w.to(f64) * c["scale"] / gone
        if factor is not None:
            y.mul_(factor)
        return y
    if op == "lookup_grad":
        dw = torch.zeros(P, c["V"], c["D"], dtype=f64, device="cuda")
        for r in range(P):
            rows = ((s["tokens"][r] >= 0) & (s["tokens"][r] < c["V"])).nonzero().squeeze(1)
            d = s["dx"][r][rows].to(f64)
            if factor is not None:
                d = d * factor[r][rows]
            dw[r].index_put_((s["tokens"][r][rows],), d, accumulate=True)
        return dw.mul_(c["scale"] / gone)

    def log_softmax(r):
        z = s["logits"][r].to(f64).mul_(c["alpha"])
        lse = torch.logsumexp(z, -1)
        return z, lse, z[torch.arange(T, device="cuda"), s["tokens"][r]] - lse

    if op == "logprob":
        got = [log_softmax(r)[1:] for r in range(P)]
        return torch.stack([g[1] for g in got]), torch.stack([g[0] for g in got])

    def logit_grad(r, z, lse, dlogp):
        g = z.sub_(lse.unsqueeze(1)).exp_().neg_()
        g[torch.arange(T, device="cuda"), s["tokens"][r]] += 1.0
        return g.mul_((dlogp * c["alpha"]).unsqueeze(1))

    grads = torch.empty(P, T, c["V"], dtype=f64, device="cuda")
    if op == "logprob_grad":
        for r in range(P):
            z = s["logits"][r].to(f64).mul_(c["alpha"])
            grads[r] = logit_grad(r, z, s["lse"][r].to(f64), s["dlogp"][r].to(f64))
        return grads
    stats, logps = torch.zeros(P, 4, dtype=f64, device="cuda"), []
    for r in range(P):
        z, lse, logp = log_softmax(r)
        w, adv = s["weight"][r].to(f64), s["adv"][r].to(f64)
        logp = logp * (w != 0)
        q = (logp - s["old"][r].to(f64)).exp()
        over = ((q > 1.0 + c["hi"]) & (adv > 0)) | ((q < 1.0 - c["lo"]) & (adv < 0))
        held = torch.where(adv > 0, q.clamp(max=1.0 + c["hi"]), q.clamp(min=1.0 - c["lo"]))
        d = s["ref"][r].to(f64) - logp
        kl = torch.expm1(d) - d
        stats[r, 1], stats[r, 2] = -(w * held * adv).sum(), (w * kl).sum()
        stats[r, 3] = (w * over).sum()
        stats[r, 0] = stats[r, 1] + c["beta"] * stats[r, 2]
        slope = torch.where(over, torch.zeros_like(q), -q * adv) - c["beta"] * torch.expm1(d)
        grads[r] = logit_grad(r, z, lse, w * slope)
        logps.append(logp)
    return stats, torch.stack(logps), grads
