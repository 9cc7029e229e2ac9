"""The dense layer of a training step and the update of its weights, as cases to measure.

The linear layer (matrix product with bias, activation and residual) and its
gradients over P data-parallel replicas, the orthogonalisation of matrices by
Newton-Schulz products, and the Muon step of a bucket plan's matrices.

``run`` computes a case either in its plain form (elementary torch operations in
32 bits) or, with ``own`` set, through the package's operators.
"""
from __future__ import annotations

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}
WEIGHT = 0.02                       # standard deviation of weights and biases
COEFS = (3.4445, -4.7750, 2.0315)   # the quintic's, steep at 0
EPS = 1e-7
CAP = 25 << 20                      # bytes of a bucket
# matrices of one layer of the 1.1B model: q, k, v, o, gate, up, down
LLAMA = "2048x2048 256x2048 256x2048 2048x2048 5632x2048 5632x2048 2048x5632"


# ----------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------
def listed():
    return [
        # one new token through a feed-forward matrix while sampling a completion (latency)
        dict(name="linear one token", op="linear", P=1, T=1, K=2048, N=5632, dtype="bf16",
             act="none", bias=False, residual=False, keep=False),
        # a few dozen tokens (a batch of sequences at one position) through the down projection
        dict(name="linear 48 tokens", op="linear", P=1, T=48, K=5632, N=2048, dtype="bf16",
             act="none", bias=False, residual=True, keep=False),
        # odd sizes that no vector load is aligned to, fp32 output
        dict(name="linear odd", op="linear", P=3, T=333, K=257, N=131, dtype="f32",
             act="gelu", bias=True, residual=True, keep=True),
        # the 2.5B model's first feed-forward matrix, 8 replicas x 1024 tokens
        dict(name="linear 2.5B fc", op="linear", P=8, T=1024, K=2560, N=10240, dtype="bf16",
             act="gelu_tanh", bias=True, residual=False, keep=True),
        # gradients over odd sizes, fp32 incoming gradient
        dict(name="linear grad odd", op="linear_grad", P=4, T=777, K=131, N=193, dtype="f32",
             act="gelu", bias=True),
        # GPT-2 small's attention input projection, 8 replicas x 4 sequences of 1024
        dict(name="linear grad gpt2 qkv", op="linear_grad", P=8, T=4096, K=768, N=2304,
             dtype="bf16", act="none", bias=True),
        # the 1.1B model's gate, 8 replicas x 1 sequence of 2048
        dict(name="linear grad llama gate", op="linear_grad", P=8, T=2048, K=2048, N=5632,
             dtype="bf16", act="silu", bias=False),
        # the updates of a toy model's matrices (latency)
        dict(name="orthogonalize toy", op="orthogonalize", P=3, rows=48, cols=131, dtype="f32",
             steps=5),
        # one large matrix: the 2.5B model's attention input projection
        dict(name="orthogonalize qkv", op="orthogonalize", P=1, rows=7680, cols=2560,
             dtype="bf16", steps=5),
        # feed-forward matrices of four layers of the 1.1B model
        dict(name="orthogonalize ffn", op="orthogonalize", P=4, rows=2048, cols=5632,
             dtype="bf16", steps=5),
        # the step of a toy policy's embedding, block and head, 4 replicas
        dict(name="muon toy", op="muon", P=4, shapes="61x64 64x64 61x64", lr=2e-4, decay=0.1,
             momentum=0.95, nesterov=True, steps=5),
        # two layers of the 1.1B model, 8 replicas
        dict(name="muon llama", op="muon", P=8, shapes=LLAMA + " " + LLAMA, lr=2e-4, decay=0.1,
             momentum=0.95, nesterov=True, steps=5),
    ]


_MOST = {"linear": 4.4e11, "linear_grad": 7.6e11, "orthogonalize": 1.4e12, "muon": 2.4e12}


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    while True:
        op = rng.choice(["linear", "linear", "linear_grad", "orthogonalize", "muon"])
        P = rng.choice([1, 2, 3, 4, 8])
        width = lambda: rng.choice([768, 2048, 2560, 5632, _log_int(rng, 16, 10240)])  # noqa: E731
        if op in ("linear", "linear_grad"):
            c = dict(op=op, P=P, T=_log_int(rng, 1, 16384), K=width(), N=width(),
                     dtype=rng.choice(["bf16", "bf16", "f32"]),
                     act=rng.choice(["none", "none", "relu", "gelu", "gelu_tanh", "silu"]),
                     bias=rng.random() < 0.5)
            if op == "linear":
                c.update(residual=rng.random() < 0.4, keep=c["act"] != "none" and rng.random() < 0.5)
        elif op == "orthogonalize":
            c = dict(op=op, P=P, rows=width(), cols=width(), dtype=rng.choice(["bf16", "f32"]),
                     steps=rng.choice([3, 5, 5, 6]))
        else:
            side = lambda: rng.choice([256, 768, 2048, _log_int(rng, 16, 4096)])  # noqa: E731
            kinds = ["%dx%d" % (side(), side()) for _ in range(rng.randint(1, 3))]
            c = dict(op=op, P=P, shapes=" ".join(rng.choice(kinds) for _ in range(rng.randint(1, 8))),
                     lr=rng.choice([1e-4, 2e-4]), decay=rng.choice([0.0, 0.1]),
                     momentum=rng.choice([0.9, 0.95]), nesterov=rng.random() < 0.7,
                     steps=rng.choice([3, 5, 5, 6]))
        w = work(c)
        if w["flops"] <= _MOST[op] and w["bytes"] <= 3e9:
            return c


def _shapes(case):
    return [tuple(int(x) for x in s.split("x")) for s in case["shapes"].split()]


def _products(rows, cols, steps):
    """Operations of the iteration on one matrix: X X^T and A^2 are symmetric, so half
    of each is enough, and (bA + cA^2) X."""
    m, n = min(rows, cols), max(rows, cols)
    return steps * (m * m * n + m ** 3 + 2 * m * m * n)


def work(case):
    op, P = case["op"], case["P"]
    if op == "muon":
        n = sum(r * c for r, c in _shapes(case))
        # mean in, momentum and master in and out, a bf16 replica for each rank out
        return {"bytes": n * (4 + 8 + 8 + 2 * P),
                "flops": sum(_products(r, c, case["steps"]) for r, c in _shapes(case))}
    if op == "orthogonalize":
        n = P * case["rows"] * case["cols"]
        return {"bytes": n * (SIZE[case["dtype"]] + 2),
                "flops": P * _products(case["rows"], case["cols"], case["steps"])}
    T, K, N, es = case["T"], case["K"], case["N"], SIZE[case["dtype"]]
    if op == "linear":
        outs = 1 + (1 if case["residual"] else 0) + (1 if case["keep"] else 0)
        return {"bytes": P * (2 * (T * K + N * K) + outs * es * T * N + (2 * N if case["bias"] else 0)),
                "flops": 2 * P * T * N * K}
    ins = 2 if case["act"] != "none" else 1
    return {"bytes": P * (2 * (2 * T * K + 2 * N * K) + ins * es * T * N + (2 * N if case["bias"] else 0)),
            "flops": 4 * P * T * N * K}


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------
def _slots(sizes, P):
    """Offsets of tensors in the flat space of a bucket plan, its length and the replicas'
    stride: last tensor first, 8-element slots, buckets of at most CAP bytes of bf16 that
    are padded to 16 P elements."""
    off, start, fill, open_ = [0] * len(sizes), 0, 0, False
    pad = lambda n: -(-n // (16 * P)) * 16 * P  # noqa: E731
    for t in reversed(range(len(sizes))):
        need = -(-sizes[t] // 8) * 8
        if open_ and fill and fill + need > CAP // 2:
            start, fill = start + pad(fill), 0
        open_ = True
        off[t] = start + fill
        fill += need
    total = start + pad(fill)
    return off, total, -(-total // 128) * 128 + 128


def _replica_view(buf, off, *shape):
    """A tensor of every rank inside the replicas: [P, *shape], rows strided by the replicas' stride."""
    return buf[:, off:off + math.prod(shape)].unflatten(1, shape)


def _gradient(g, rows, cols, std):
    """Noise, and a few directions that carry as much again."""
    k = min(8, rows, cols)
    u = torch.randn(rows, k, generator=g, device="cuda")
    v = torch.randn(k, cols, generator=g, device="cuda")
    x = torch.randn(rows, cols, generator=g, device="cuda")
    return x.addmm_(u, v, alpha=1.0 / math.sqrt(k)).mul_(std)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, P = case["op"], case["P"]

    def normal(*shape, dtype=torch.bfloat16, std=1.0):
        return torch.randn(*shape, generator=g, device="cuda", dtype=dtype).mul_(std)

    s = dict(case=dict(case))
    if op == "orthogonalize":
        r, c = case["rows"], case["cols"]
        s["x"] = torch.stack([_gradient(g, r, c, 5e-4) for _ in range(P)]).to(DTYPES[case["dtype"]])
        s["out"] = torch.empty(P, r, c, dtype=torch.bfloat16, device="cuda")
        return s
    if op == "muon":
        shapes = _shapes(case)
        off, L, stride = _slots([r * c for r, c in shapes], P)
        s["mean"], s["momentum"], s["master"] = (torch.zeros(L, device="cuda") for _ in range(3))
        for o, (r, c) in zip(off, shapes):
            # a running mean of gradients is smaller than one of them
            s["mean"][o:o + r * c] = _gradient(g, r, c, 5e-4).view(-1)
            s["momentum"][o:o + r * c] = _gradient(g, r, c, 2e-4).view(-1)
            s["master"][o:o + r * c] = normal(r * c, dtype=torch.float32, std=WEIGHT)
        s["params"] = torch.zeros(P, stride, dtype=torch.bfloat16, device="cuda")
        s["params"][:, :L] = s["master"].to(torch.bfloat16)
        return s
    T, K, N, dt = case["T"], case["K"], case["N"], DTYPES[case["dtype"]]
    # the layer's slots in replicas that hold other tensors too
    s["at"], _, stride = _slots([N * K, N, 1000], P)
    s["x"] = normal(P, T, K)
    s["params"] = normal(P, stride, std=WEIGHT)
    if op == "linear":
        s["y"] = torch.empty(P, T, N, dtype=dt, device="cuda")
        s["z"] = torch.empty_like(s["y"]) if case["keep"] else None
        s["residual"] = normal(P, T, N, dtype=dt) if case["residual"] else None
        return s
    s["dy"] = normal(P, T, N, dtype=dt, std=1e-2)
    # what the forward kept
    s["z"] = None
    if case["act"] != "none":
        s["z"] = normal(P, T, N, dtype=dt, std=WEIGHT * math.sqrt(K))
    s["dx"] = torch.empty_like(s["x"])
    s["grads"] = torch.zeros(P, stride, dtype=torch.bfloat16, device="cuda")
    return s


# ----------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------
def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    import gradient_sync_zero_gb300 as dps
    c = s["case"]
    op, P = c["op"], c["P"]
    if op == "orthogonalize":
        if "ws" not in s:
            s["ws"] = dps.new_orthogonalize_workspace(P, c["rows"], c["cols"])
        cfg = dps.newton_schulz_cfg(*COEFS, eps=EPS, steps=c["steps"])
        dps.dp_orthogonalize(s["x"], s["out"], s["ws"], cfg)
        return s["out"]
    if op == "muon":
        if "muon" not in s:
            shapes = _shapes(c)
            plan = dps.Plan([a * b for a, b in shapes], CAP, P)
            s["plan_ws"] = plan.new_workspace()
            s["muon"] = dps.Muon(plan, dict(enumerate(shapes)))
            s["ws"] = s["muon"].new_workspace()
        cfg = dps.muon_cfg(lr=c["lr"], momentum=c["momentum"], weight_decay=c["decay"],
                           nesterov=c["nesterov"], scale=dps.DP_MUON_MATCH_RMS,
                           newton_schulz=dps.newton_schulz_cfg(*COEFS, eps=EPS, steps=c["steps"]))
        dps.dp_muon_step(s["muon"], s["plan_ws"], s["ws"], s["mean"], s["master"], s["momentum"],
                         s["params"], cfg)
        return s["master"], s["momentum"], s["params"]
    T, K, N = c["T"], c["K"], c["N"]
    act = {"none": dps.DP_ACT_NONE, "relu": dps.DP_ACT_RELU, "gelu": dps.DP_ACT_GELU,
           "gelu_tanh": dps.DP_ACT_GELU_TANH, "silu": dps.DP_ACT_SILU}[c["act"]]
    w = _replica_view(s["params"], s["at"][0], N, K)
    if "ws" not in s:
        s["ws"] = dps.new_linear_workspace(s["x"], w, backward=op == "linear_grad")
    if op == "linear":
        bias = _replica_view(s["params"], s["at"][1], N) if c["bias"] else None
        dps.dp_linear_forward(s["x"], w, s["y"], bias=bias, residual=s["residual"], z=s["z"],
                              act=act, ws=s["ws"])
        return (s["y"], s["z"]) if c["keep"] else s["y"]
    dw = _replica_view(s["grads"], s["at"][0], N, K)
    db = _replica_view(s["grads"], s["at"][1], N) if c["bias"] else None
    dps.dp_linear_backward(s["dy"], s["x"], w, dx=s["dx"], dw=dw, dbias=db, z=s["z"], act=act,
                           ws=s["ws"])
    return (s["dx"], dw, db) if c["bias"] else (s["dx"], dw)


def _act(z, kind):
    if kind == "relu":
        return torch.where(z > 0, z, 0.0)
    if kind == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if kind == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    if kind == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


def _act_slope(z, kind):
    if kind == "relu":
        return (z > 0).float()
    if kind == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + \
            z * torch.exp(-0.5 * z * z) * (1.0 / math.sqrt(2.0 * math.pi))
    if kind == "gelu_tanh":
        k = math.sqrt(2.0 / math.pi)
        t = torch.tanh(k * (z + 0.044715 * z * z * z))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * k * (1.0 + 3 * 0.044715 * z * z)
    q = 1.0 / (1.0 + torch.exp(-z))
    return q * (1.0 + z * (1.0 - q))


def _newton_schulz(x, steps):
    """x [..., rows, cols] in fp32."""
    tall = x.shape[-2] > x.shape[-1]
    if tall:
        x = x.mT
    x = x / x.square().sum((-2, -1), keepdim=True).sqrt().clamp(min=EPS)
    a, b, c = COEFS
    for _ in range(steps):
        gram = x @ x.mT
        x = a * x + (b * gram + c * (gram @ gram)) @ x
    return x.mT if tall else x


def _run_plain(s):
    c = s["case"]
    op = c["op"]
    if op == "orthogonalize":
        return _newton_schulz(s["x"].float(), c["steps"]).to(torch.bfloat16)
    if op == "muon":
        mu, shapes = c["momentum"], _shapes(c)
        off, _, _ = _slots([a * b for a, b in shapes], c["P"])
        for o, (rows, cols) in zip(off, shapes):
            at = slice(o, o + rows * cols)
            g, buf, w = (s[k][at].view(rows, cols) for k in ("mean", "momentum", "master"))
            buf.copy_(mu * buf + (1.0 - mu) * g)
            u = mu * buf + (1.0 - mu) * g if c["nesterov"] else buf
            lr = c["lr"] * 0.2 * math.sqrt(max(rows, cols))
            w.copy_((1.0 - c["lr"] * c["decay"]) * w - lr * _newton_schulz(u, c["steps"]))
            s["params"][:, at] = w.view(-1).to(torch.bfloat16)
        return s["master"], s["momentum"], s["params"]
    N, K, dt = c["N"], c["K"], DTYPES[c["dtype"]]
    x, w = s["x"].float(), _replica_view(s["params"], s["at"][0], N, K).float()
    if op == "linear":
        z = x @ w.mT
        if c["bias"]:
            z = z + _replica_view(s["params"], s["at"][1], N).float().unsqueeze(1)
        y = _act(z, c["act"])
        if c["residual"]:
            y = y + s["residual"].float()
        return (y.to(dt), z.to(dt)) if c["keep"] else y.to(dt)
    dz = s["dy"].float()
    if c["act"] != "none":
        dz = dz * _act_slope(s["z"].float(), c["act"])
    bf = torch.bfloat16
    dx, dw = (dz @ w).to(bf), (dz.mT @ x).to(bf)
    return (dx, dw, dz.sum(1).to(bf)) if c["bias"] else (dx, dw)


# ----------------------------------------------------------------------------
# the definition in 64 bits
# ----------------------------------------------------------------------------
def _exact_orthogonal(x, steps):
    """One matrix in 64 bits, by its smaller side's Gram matrix on the left or right."""
    x = x / max(float(torch.linalg.vector_norm(x)), EPS)
    a, b, c = COEFS
    for _ in range(steps):
        if x.shape[0] <= x.shape[1]:
            q = torch.mm(x, x.t())
            p = torch.addmm(q, q, q, beta=b, alpha=c)
            p.diagonal().add_(a)
            x = torch.mm(p, x)
        else:
            q = torch.mm(x.t(), x)
            p = torch.addmm(q, q, q, beta=b, alpha=c)
            p.diagonal().add_(a)
            x = torch.mm(x, p)
    return x


def _exact_act(z, kind):
    """(value, slope)."""
    if kind == "none":
        return z, torch.ones_like(z)
    if kind == "relu":
        return z.clamp(min=0.0), (z > 0).to(z.dtype)
    if kind == "gelu":
        half = torch.special.ndtr(z)
        return z * half, half + z * torch.exp(z.square() / -2) / math.sqrt(2 * math.pi)
    if kind == "silu":
        q = torch.sigmoid(z)
        return z * q, torch.addcmul(q, q, z * (1 - q))
    # 0.5 (1 + tanh u) is the logistic function of 2 u
    k = 2 * math.sqrt(2 / math.pi)
    q = torch.sigmoid(k * (z + 0.044715 * z.pow(3)))
    return z * q, q + z * q * (1 - q) * k * (1 + 0.134145 * z.square())


def exact(case, seed):
    c, op, P, f64 = case, case["op"], case["P"], torch.float64
    s = prepare(case, seed)
    if op == "orthogonalize":
        return torch.stack([_exact_orthogonal(x.to(f64), c["steps"]) for x in s["x"]])
    if op == "muon":
        shapes, mu = _shapes(c), c["momentum"]
        off, L, _ = _slots([r * k for r, k in shapes], P)
        master, momentum = s["master"].to(f64), s["momentum"].to(f64)
        for o, (r, k) in zip(off, shapes):
            g = s["mean"][o:o + r * k].to(f64)
            buf = momentum[o:o + r * k]
            buf += (1 - mu) * (g - buf)
            u = g + mu * (buf - g) if c["nesterov"] else buf
            step = 0.2 * c["lr"] * max(r, k) ** 0.5
            w = master[o:o + r * k]
            w -= c["lr"] * c["decay"] * w
            w -= step * _exact_orthogonal(u.view(r, k), c["steps"]).reshape(-1)
        params = torch.zeros(s["params"].shape, dtype=f64, device="cuda")
        params[:, :L] = master
        return master, momentum, params
    T, K, N = c["T"], c["K"], c["N"]
    w0, b0 = s["at"][:2]
    outs = []
    for r in range(P):
        x = s["x"][r].to(f64)
        w = s["params"][r, w0:w0 + N * K].view(N, K).to(f64)
        if op == "linear":
            z = torch.mm(x, w.t())
            if c["bias"]:
                z += s["params"][r, b0:b0 + N].to(f64)
            y = _exact_act(z, c["act"])[0]
            if c["residual"]:
                y = y + s["residual"][r].to(f64)
            outs.append((y, z) if c["keep"] else (y,))
        else:
            dz = s["dy"][r].to(f64)
            if c["act"] != "none":
                dz = dz * _exact_act(s["z"][r].to(f64), c["act"])[1]
            got = (torch.mm(dz, w), torch.mm(dz.t(), x))
            outs.append(got + (dz.sum(0),) if c["bias"] else got)
    got = tuple(torch.stack(o) for o in zip(*outs))
    return got[0] if len(got) == 1 else got
