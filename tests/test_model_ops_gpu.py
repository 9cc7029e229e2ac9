"""The operators at the ends of a training step on the GPU, against plain 64-bit
implementations on the host, with bounds derived from the kernels' arithmetic
(model_reference.py)."""
import numpy as np
import pytest
import torch

import gradient_sync_zero_gb300 as dps
import model_reference as ref
from model_reference import U, stored

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def rnd(g, *shape, dtype=F32, std=1.0):
    return (torch.randn(*shape, generator=g) * std).to(dtype)


def close(got, want, bound):
    got = got.detach().double().cpu()
    bad = ~((got - want).abs() <= bound)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:3].tolist(),
                           got[bad][:3].tolist(), want[bad][:3].tolist())


def bits(t):
    t = t.detach().contiguous()
    return t.view(torch.int16 if t.dtype == BF else torch.int32).cpu()


def strided(t, row_pad, rank_pad=0, lead=0):
    """A CUDA copy of [P, T, D] `t` with rows D + row_pad apart, rank_pad elements more
    between ranks, its first element `lead` elements into its buffer.  Everything
    around it is NaN."""
    P, T, D = t.shape
    row, rank = D + row_pad, T * (D + row_pad) + rank_pad
    buf = torch.full((lead + P * rank + 64,), float("nan"), dtype=t.dtype, device="cuda")
    v = buf.as_strided((P, T, D), (rank, row, 1), lead)
    v.copy_(t)
    return v, buf


# ---------------------------------------------------------------- dropout
DROP_SHAPES = [(1, 1, 1), (2, 1, 3), (3, 7, 5), (4, 33, 64), (2, 5, 257), (1, 3, 4096), (2, 100, 48),
               (1, 1, 100003)]


@pytest.mark.parametrize("shape", DROP_SHAPES, ids=str)
@pytest.mark.parametrize("tx,to,res", [(BF, BF, BF), (F32, F32, None), (BF, F32, F32), (F32, BF, None),
                                       (F32, F32, BF)])
def test_dropout(shape, tx, to, res):
    g = gen(1)
    x = rnd(g, *shape, dtype=tx)
    rs = None if res is None else rnd(g, *shape, dtype=res)
    p, seed, off = 0.3, 0x1234567890ABCDEF, 11
    want = ref.dropout(x.double(), p, seed, off)
    err = 3 * U * want.abs()
    if rs is not None:
        want = want + rs.double()
        err = err + U * want.abs()
    out = torch.empty(shape, dtype=to, device="cuda")
    dps.dp_dropout(x.cuda(), out, dps.dropout_cfg(p, seed, off), residual=None if rs is None else rs.cuda())
    close(out, want, stored(want, err, to))


@pytest.mark.parametrize("p", [0.0, 1e-10, 1.0, 1 - 1e-12])
@pytest.mark.parametrize("D", [24, 13])
def test_dropout_of_nothing_and_everything(p, D):
    x = rnd(gen(2), 2, 6, D).cuda()
    x[0, 2, 1], x[1, 3, 4] = float("nan"), float("inf")
    out, r = torch.empty_like(x), torch.ones_like(x)
    dps.dp_dropout(x, out, dps.dropout_cfg(p, 5), residual=r)
    if p < 0.5:
        assert torch.equal(bits(out), bits(x + 1))
    else:
        assert torch.equal(out, r)
    if p == 0.0:
        dps.dp_dropout(x, out, None)
        assert torch.equal(bits(out), bits(x))


def test_dropped_infinities_and_nan_are_zero():
    P, T, D, p, seed = 2, 9, 40, 0.5, 99
    keep = ref.keep_mask(P, T * D, p, seed, 0).view(P, T, D)
    x = torch.where(keep, torch.ones(P, T, D), torch.tensor(float("nan")))
    x[:, ::2] = torch.where(keep[:, ::2], x[:, ::2], torch.tensor(float("inf")))
    out = torch.empty(P, T, D, device="cuda")
    dps.dp_dropout(x.cuda(), out, dps.dropout_cfg(p, seed))
    assert torch.equal(out.cpu(), torch.where(keep, 2.0, 0.0))


def test_dropout_ranks_offsets_and_seeds():
    """Rank r of a call with rank0 = k is rank r + k of one with rank0 = 0; masks of
    ranks, offsets and seeds differ; the kept share is 1 - p within five standard
    deviations."""
    n, p = 1 << 18, 0.25
    x = torch.ones(4, 1, n, device="cuda")
    a, b, c, d = (torch.empty_like(x) for _ in range(4))
    dps.dp_dropout(x, a, dps.dropout_cfg(p, 7, 3))
    dps.dp_dropout(x[:2], b[:2], dps.dropout_cfg(p, 7, 3, rank0=2))
    assert torch.equal(a[2:], b[:2])
    dps.dp_dropout(x, c, dps.dropout_cfg(p, 7, 4))
    dps.dp_dropout(x, d, dps.dropout_cfg(p, 7 + (1 << 32), 3))
    sd = 5 * (p * (1 - p) / n) ** 0.5
    for t in (a, c, d):
        assert ((t != 0).float().mean(-1) - (1 - p)).abs().max() < sd
    same = p * p + (1 - p) * (1 - p)
    for u, v in ((a[0], a[1]), (a, c), (a, d)):
        assert abs(float(((u != 0) == (v != 0)).float().mean()) - same) < 5 * (same * (1 - same) / n) ** 0.5


@pytest.mark.parametrize("row_pad,rank_pad,lead", [(0, 0, 0), (8, 16, 8), (3, 5, 1), (0, 7, 0), (5, 0, 0)])
@pytest.mark.parametrize("D", [32, 21])
def test_dropout_strides(row_pad, rank_pad, lead, D):
    """Strided x, residual and out, in place on the residual too; nothing around the
    output is written.  Element counters do not depend on strides."""
    x = rnd(gen(4), 3, 10, D, dtype=BF)
    r = rnd(gen(5), 3, 10, D, dtype=BF)
    cfg = dps.dropout_cfg(0.4, 21, 2)
    want = torch.empty(3, 10, D, dtype=BF, device="cuda")
    dps.dp_dropout(x.cuda(), want, cfg, residual=r.cuda())
    xs, _ = strided(x, row_pad, rank_pad, lead)
    rs, rbuf = strided(r, row_pad, rank_pad, lead)
    os_, obuf = strided(torch.zeros_like(x), row_pad, rank_pad, lead)
    dps.dp_dropout(xs, os_, cfg, residual=rs)
    assert torch.equal(os_, want)
    os_.fill_(float("nan"))
    assert torch.isnan(obuf).all()
    dps.dp_dropout(xs, rs, cfg, residual=rs)          # in place on the residual
    assert torch.equal(rs, want)
    rs.fill_(float("nan"))
    assert torch.isnan(rbuf).all()


def test_dropout_in_place_column_slices_and_interleaved_ranks():
    x = rnd(gen(6), 2, 8, 16).cuda()
    cfg = dps.dropout_cfg(0.5, 1)
    want = torch.empty_like(x)
    dps.dp_dropout(x, want, cfg)
    y = x.clone()
    dps.dp_dropout(y, y, cfg)
    assert torch.equal(y, want)
    both = torch.cat((x, torch.zeros_like(x)), -1)    # x left, out right, in one buffer
    dps.dp_dropout(both[..., :16], both[..., 16:], cfg)
    assert torch.equal(both[..., 16:], want) and torch.equal(both[..., :16], x)
    woven = torch.zeros(8, 2, 16, device="cuda")      # [T][P][D]
    dps.dp_dropout(x, woven.transpose(0, 1), cfg)
    assert torch.equal(woven.transpose(0, 1), want)
    flat = torch.empty(8, 16, device="cuda")          # [T, D]: one rank
    dps.dp_dropout(x[0], flat, cfg)
    assert torch.equal(flat, want[0])


def test_dropout_backward_is_the_adjoint_of_its_forward():
    x, dy = rnd(gen(7), 2, 50, 33).cuda(), rnd(gen(8), 2, 50, 33).cuda()
    cfg = dps.dropout_cfg(0.35, 77, 9)
    y, dx = torch.empty_like(x), torch.empty_like(x)
    dps.dp_dropout(x, y, cfg)
    dps.dp_dropout(dy, dx, cfg)
    a, b = (y.double() * dy.double()).sum(), (x.double() * dx.double()).sum()
    assert abs(a - b) <= 4 * U * float((x.double() * dx.double()).abs().sum())
    # the gradient by differences: dropout is linear, so a step of one is exact
    e = torch.zeros_like(x)
    e[1, 20, 7] = 1.0
    ye = torch.empty_like(x)
    dps.dp_dropout(e, ye, cfg)
    assert abs(float((ye * dy).sum()) - float(dx[1, 20, 7])) <= 4 * U * abs(float(dx[1, 20, 7]))


def test_captured_graph_draws_a_new_mask_at_each_replay():
    x = torch.ones(2, 4, 100, device="cuda")
    out = torch.empty_like(x)
    state = torch.tensor([5, 1], dtype=torch.int64, device="cuda")
    cfg = dps.dropout_cfg(0.5, 0, 0, seed_dev=state)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        dps.dp_dropout(x, out, cfg)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dps.dp_dropout(x, out, cfg)
    for seed, off in ((5, 1), (5, 2), (1 << 40, 0xFFFFFFFF)):
        state.copy_(torch.tensor([seed, off]))
        graph.replay()
        want = torch.empty_like(x)
        dps.dp_dropout(x, want, dps.dropout_cfg(0.5, seed, off))
        assert torch.equal(out, want)


# ---------------------------------------------------------------- lookup
LOOKUPS = [(1, 1, 1, 1), (2, 3, 5, 8), (3, 17, 11, 131), (2, 64, 100, 256), (1, 5, 7, 2049), (4, 9, 1000, 48),
           (2, 300, 40, 32)]


@pytest.mark.parametrize("P,T,V,D", LOOKUPS, ids=str)
@pytest.mark.parametrize("tw,to", [(BF, BF), (F32, F32), (BF, F32), (F32, BF)])
@pytest.mark.parametrize("p", [0.0, 0.2])
def test_lookup(P, T, V, D, tw, to, p):
    g = gen(10)
    table = rnd(g, P, V, D, dtype=tw)
    tokens = torch.randint(-1, V + 1, (P, T), generator=g)
    drop = (p, 123456789123, 4)
    want = ref.lookup(table.double(), tokens, 3.25, drop)
    for ty in (torch.int32, torch.int64):
        out = torch.full((P, T, D), float("nan"), dtype=to, device="cuda")
        dps.dp_embedding_forward(table.cuda(), tokens.to(ty).cuda(), out, scale=3.25,
                                 dropout=dps.dropout_cfg(*drop))
        close(out, want, stored(want, 4 * U * want.abs(), to))


def test_lookup_equals_lookup_then_dropout():
    """In fp32 the fused dropout draws the mask of dp_dropout on [P, T, D]."""
    table = rnd(gen(11), 2, 50, 24).cuda()
    tokens = torch.randint(0, 50, (2, 37), generator=gen(12)).cuda()
    cfg = dps.dropout_cfg(0.3, 8, 1, rank0=6)
    a, b, c = (torch.empty(2, 37, 24, device="cuda") for _ in range(3))
    dps.dp_embedding_forward(table, tokens, a, scale=0.5, dropout=cfg)
    dps.dp_embedding_forward(table, tokens, b, scale=0.5)
    dps.dp_dropout(b, c, cfg)
    assert torch.equal(a, c)


@pytest.mark.parametrize("D", [16, 15])
def test_lookup_in_a_plan_slot_with_strided_output(D):
    """The table is its slot of the parameter replicas; rows that no token names hold
    NaN; ranks may share one table (rank stride 0)."""
    V = 31
    plan = dps.Plan([77, V * D, 500], 1 << 20, 3)
    params = plan.new_replicas()
    params.fill_(float("nan"))
    view = plan.tensor_view(params, 1, (V, D))
    tokens = torch.randint(0, V, (3, 19), generator=gen(13))
    for r in range(3):
        for v in set(tokens[r].tolist()):
            view[r, v] = rnd(gen(100 * r + v), D, dtype=BF).cuda()
    want = torch.stack([view[r].cpu()[tokens[r]] for r in range(3)])
    out, buf = strided(torch.zeros(3, 19, D, dtype=BF), 3, 1, 5)
    dps.dp_embedding_forward(view, tokens.cuda(), out)
    assert torch.equal(bits(out), bits(want.cuda()))
    out.fill_(float("nan"))
    assert torch.isnan(buf).all()
    one = rnd(gen(14), V, D, dtype=BF).cuda()
    dps.dp_embedding_forward(one.expand(3, V, D), tokens.cuda(), out)
    assert torch.equal(out.cpu(), torch.stack([one.cpu()[t] for t in tokens]))


def test_lookup_past_2_to_31_elements():
    """The second rank's table and the last rows lie past 2^31 elements."""
    V, D = 70000, 32768                                # 2.29e9 elements a rank
    buf = torch.zeros(2 * V * D, dtype=BF, device="cuda")
    table = buf.view(2, V, D)
    for r in range(2):
        for v in (0, 65535, V - 1):
            table[r, v] = 1 + r + v % 64
    tokens = torch.tensor([[V - 1, 0, 65535, -1]] * 2, device="cuda")
    out = torch.empty(2, 4, D, dtype=BF, device="cuda")
    dps.dp_embedding_forward(table, tokens, out)
    want = torch.tensor([[1 + (V - 1) % 64, 1, 1 + 65535 % 64, 0], [2 + (V - 1) % 64, 2, 2 + 65535 % 64, 0]])
    assert torch.equal(out[:, :, 0].float().cpu(), want.float())
    assert torch.equal(out[:, :, -1].float().cpu(), want.float())
    # and its gradient
    ws = dps.new_embedding_workspace(2, 4, V, D)
    dps.dp_embedding_backward(out, tokens, table, ws)
    assert torch.equal(table[:, [V - 1, 0, 65535], 5].float().cpu(), want[:, :3].float())
    assert float(table[1, V - 2].abs().max()) == 0 and float(table[0, 65534].abs().max()) == 0


def test_empty_lookup():
    table = torch.zeros(2, 4, 8, device="cuda")
    dps.dp_embedding_forward(table, torch.zeros(2, 0, dtype=torch.int64, device="cuda"),
                             torch.zeros(2, 0, 8, device="cuda"))


# ---------------------------------------------------------------- its gradient
def _grad_case(P, T, V, D, tx, tg, kind, seed=0, p=0.0, scale=1.5, accumulate=False, ty=torch.int64):
    g = gen(seed)
    dout = rnd(g, P, T, D, dtype=tx)
    if kind == "uniform":
        tokens = torch.randint(0, V, (P, T), generator=g)
    elif kind == "skewed":                     # most tokens are one of two
        tokens = torch.randint(0, V, (P, T), generator=g)
        hot = torch.rand(P, T, generator=g)
        tokens = torch.where(hot < 0.6, torch.tensor(V - 1), torch.where(hot < 0.8, torch.tensor(V // 2), tokens))
    elif kind == "one":
        tokens = torch.full((P, T), V // 3)
    elif kind == "padded":
        tokens = torch.randint(0, V, (P, T), generator=g)
        tokens[:, T // 2:] = -100
        tokens[0] = V                          # a rank with nothing at all
    dead = (tokens < 0) | (tokens >= V)
    dout[dead] = float("nan")                  # never read
    drop = (p, 0xDEADBEEF12345, 3)
    want, mag, n = ref.lookup_grad(torch.nan_to_num(dout.double()), tokens, V, scale, drop)
    plan = dps.Plan([40, V * D, 9], 1 << 30, P)
    buf = torch.full((P, plan.stride), 7.0, dtype=tg, device="cuda")
    view = plan.tensor_view(buf, 1, (V, D))
    err = (n + 4) * U * mag
    if accumulate:
        old = rnd(g, P, V, D, dtype=tg)
        view.copy_(old)
        want = torch.where(n > 0, want + old.double(), old.double())
        err = err + U * want.abs()
    else:
        view.fill_(float("nan"))
    ws = dps.new_embedding_workspace(P, T, V, D)
    ws.fill_(0xA5)
    args = (dout.cuda(), tokens.to(ty).cuda(), view, ws)
    kw = dict(scale=scale, dropout=dps.dropout_cfg(*drop), accumulate=accumulate)
    dps.dp_embedding_backward(*args, **kw)
    bound = torch.where(n > 0, stored(want, err, tg), torch.zeros(())) if accumulate else stored(want, err, tg)
    close(view, want, bound)
    first = bits(view)
    if accumulate:
        view.copy_(old)
    dps.dp_embedding_backward(*args, **kw)     # the same bits again, on a used workspace
    assert torch.equal(first, bits(view))
    o = plan.tensor(1)[1]
    assert (buf[:, :o] == 7).all() and (buf[:, o + V * D:] == 7).all()


GRADS = [(1, 1, 1, 1), (2, 1, 5, 8), (3, 50, 7, 33), (2, 200, 1000, 16), (4, 129, 64, 131), (1, 777, 3, 264),
         (2, 31, 40, 2050), (2, 1025, 300, 40)]


@pytest.mark.parametrize("P,T,V,D", GRADS, ids=str)
@pytest.mark.parametrize("kind", ["uniform", "skewed", "one", "padded"])
def test_lookup_gradient(P, T, V, D, kind):
    _grad_case(P, T, V, D, BF, BF, kind, seed=T)


@pytest.mark.parametrize("tx,tg", [(F32, F32), (BF, F32), (F32, BF)])
@pytest.mark.parametrize("D", [24, 19])
@pytest.mark.parametrize("accumulate", [False, True])
def test_lookup_gradient_types_dropout_and_accumulation(tx, tg, D, accumulate):
    _grad_case(2, 150, 20, D, tx, tg, "skewed", seed=D, p=0.3, accumulate=accumulate, ty=torch.int32)


@pytest.mark.parametrize("accumulate", [False, True])
def test_lookup_gradient_without_tokens(accumulate):
    grad = torch.full((2, 6, 8), 3.0, device="cuda", dtype=BF)
    ws = dps.new_embedding_workspace(2, 0, 6, 8)
    dps.dp_embedding_backward(torch.zeros(2, 0, 8, device="cuda"),
                              torch.zeros(2, 0, dtype=torch.int64, device="cuda"), grad, ws,
                              accumulate=accumulate)
    assert (grad == (3.0 if accumulate else 0.0)).all()


def _grad_by_torch(dout, tokens, V, scale=1.0):
    """Per rank, in 64 bits on the GPU (larger cases than the host loop's)."""
    P, T, D = dout.shape
    g = torch.zeros(P, V, D, dtype=torch.float64, device="cuda")
    mag, n = torch.zeros_like(g), torch.zeros(P, V, 1, dtype=torch.float64, device="cuda")
    for r in range(P):
        ok = ((tokens[r] >= 0) & (tokens[r] < V)).nonzero().squeeze(1)
        d = dout[r][ok].double() * scale
        g[r].index_add_(0, tokens[r][ok], d)
        mag[r].index_add_(0, tokens[r][ok], d.abs())
        n[r].index_add_(0, tokens[r][ok], torch.ones(len(ok), 1, dtype=torch.float64, device="cuda"))
    return g, mag, n


@pytest.mark.parametrize("P,T,V,D,hot", [(2, 20000, 50257, 64, 0.3), (1, 70001, 500, 40, 0.9), (3, 4097, 131072, 24, 0.0),
                                         (8, 3000, 2000, 768, 0.5), (1, 300000, 3, 8, 0.5)])
def test_lookup_gradient_large(P, T, V, D, hot):
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    dout = torch.randn(P, T, D, generator=g, device="cuda").to(BF)
    tokens = torch.randint(0, V, (P, T), generator=g, device="cuda")
    tokens = torch.where(torch.rand(P, T, generator=g, device="cuda") < hot, torch.full_like(tokens, V // 2), tokens)
    want, mag, n = _grad_by_torch(dout, tokens, V)
    grad = torch.full((P, V, D), float("nan"), device="cuda")
    ws = dps.new_embedding_workspace(P, T, V, D)
    dps.dp_embedding_backward(dout, tokens, grad, ws)
    bad = ~((grad.double() - want).abs() <= stored(want, (n + 4) * U * mag, F32))
    assert not bad.any(), int(bad.sum())
    again = torch.empty_like(grad)
    dps.dp_embedding_backward(dout, tokens, again, ws)
    assert torch.equal(grad, again)


def test_lookup_gradient_is_the_adjoint_and_the_difference():
    """Both kernels on the GPU: <lookup(E), dout> = <E, grad(dout)>; and, the lookup being
    linear, one entry of the gradient is the change of <lookup, dout> for a step of one."""
    P, T, V, D = 2, 60, 13, 24
    table, dout = rnd(gen(20), P, V, D).cuda(), rnd(gen(21), P, T, D).cuda()
    tokens = torch.randint(-1, V, (P, T), generator=gen(22)).cuda()
    cfg = dps.dropout_cfg(0.25, 5, 6)
    out, grad = torch.empty(P, T, D, device="cuda"), torch.empty(P, V, D, device="cuda")
    dps.dp_embedding_forward(table, tokens, out, scale=1.25, dropout=cfg)
    dps.dp_embedding_backward(dout, tokens, grad, dps.new_embedding_workspace(P, T, V, D), scale=1.25, dropout=cfg)
    a, b = (out.double() * dout.double()), (table.double() * grad.double())
    assert abs(a.sum() - b.sum()) <= (T + 8) * U * float(a.abs().sum())
    v = int(tokens[tokens >= 0][0])
    step = torch.zeros_like(table)
    step[0, v, 3] = 1.0
    moved = torch.empty_like(out)
    dps.dp_embedding_forward(step, tokens, moved, scale=1.25, dropout=cfg)
    terms = moved.double() * dout.double()
    assert abs(float(terms.sum()) - float(grad[0, v, 3])) <= (T + 8) * U * float(terms.abs().sum())


# ---------------------------------------------------------------- log-probabilities
LOGITS = [(1, 1, 1), (2, 3, 2), (1, 2, 7), (3, 5, 129), (2, 7, 1000), (1, 3, 50257), (2, 2, 32000), (1, 40, 4099),
          (1, 1, 131073), (1, 2, 300001), (1, 300, 97)]


def _logits(P, T, V, dtype, seed=0, std=3.0):
    g = gen(seed + V)
    x = rnd(g, P, T, V, dtype=dtype, std=std)
    tokens = torch.randint(0, V, (P, T), generator=g)
    at = tokens.unsqueeze(-1)
    x.scatter_(-1, at, (x.gather(-1, at).float() + 6).to(dtype))
    return x, tokens


@pytest.mark.parametrize("P,T,V", LOGITS, ids=str)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_logprob_and_its_gradient(P, T, V, dtype):
    x, tokens = _logits(P, T, V, dtype)
    alpha = float(np.float32(0.8))
    if P * T > 2:
        tokens[-1, -1] = -100
        x[-1, -1] = float("nan")                       # not read
    clean = torch.nan_to_num(x.double())
    logp, lse = ref.logprob(clean, tokens, alpha)
    tol = ref.logprob_bound(clean, alpha)
    xd, td = x.cuda(), tokens.cuda()
    glp, gls = (torch.full((P, T), float("nan"), device="cuda") for _ in range(2))
    dps.dp_token_logprob(xd, td, glp, gls, logit_scale=alpha)
    close(glp, logp, tol)
    close(gls, lse, tol)
    only = torch.empty_like(glp)
    dps.dp_token_logprob(xd, td.int(), only, logit_scale=alpha)
    assert torch.equal(only, glp)
    # the gradient, from the kernel's own lse
    dlogp = rnd(gen(V), P, T)
    if P * T > 3:
        dlogp[0, 0] = 0.0
        xd[0, 0] = float("nan")                        # not read either
    g, p = ref.logit_grad(clean, tokens, alpha, gls.double().cpu(), dlogp.double())
    bound = stored(g, ref.logit_grad_bound(p, clean, alpha, dlogp.double(), 0.0), dtype)
    dl = torch.full_like(xd, float("nan"))
    dps.dp_token_logprob_backward(xd, td, gls, dlogp.cuda(), dl, logit_scale=alpha)
    close(dl, g, bound)
    dps.dp_token_logprob_backward(xd, td, gls, dlogp.cuda(), xd, logit_scale=alpha)   # in place
    assert torch.equal(bits(xd), bits(dl))


@pytest.mark.parametrize("row_pad,rank_pad,lead", [(1, 0, 0), (3, 5, 1), (8, 8, 8), (64, 3, 7)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_logits_strides(row_pad, rank_pad, lead, dtype):
    """Rows at every alignment, logits and dlogits aligned differently; the same bits as
    contiguous rows are not promised, the bound is."""
    P, T, V = 2, 9, 1234
    x, tokens = _logits(P, T, V, dtype, seed=5)
    logp, lse = ref.logprob(x.double(), tokens, 1.0)
    xs, _ = strided(x, row_pad, rank_pad, lead)
    a, b = (torch.empty(P, T, device="cuda") for _ in range(2))
    dps.dp_token_logprob(xs, tokens.cuda(), a, b)
    tol = ref.logprob_bound(x.double(), 1.0)
    close(a, logp, tol)
    close(b, lse, tol)
    dlogp = rnd(gen(1), P, T)
    g, p = ref.logit_grad(x.double(), tokens, 1.0, b.double().cpu(), dlogp.double())
    bound = stored(g, ref.logit_grad_bound(p, x.double(), 1.0, dlogp.double(), 0.0), dtype)
    for args in ((row_pad, rank_pad, lead), (2, 1, 3), (0, 0, 0)):
        ds, buf = strided(torch.zeros_like(x), *args)
        dps.dp_token_logprob_backward(xs, tokens.cuda(), b, dlogp.cuda(), ds)
        close(ds, g, bound)
        ds.fill_(float("nan"))
        assert torch.isnan(buf).all()
        old = logp.float()
        cfg = dps.policy_cfg()
        w = dlogp.abs()
        lp, st = torch.empty(P, T, device="cuda"), torch.empty(P, 4, device="cuda")
        dps.dp_policy_loss(xs, tokens.cuda(), old.cuda(), dlogp.cuda(), lp, st, dlogits=ds, weight=w.cuda(), cfg=cfg)
        want = ref.policy(x.double(), tokens, old.double(), None, dlogp.double(), w.double(), 0.2, 0.2, 0.0, 1.0)
        close(ds, want[3], stored(want[3], _policy_bound(want, x.double(), 1.0, tol), dtype))
        ds.fill_(float("nan"))
        assert torch.isnan(buf).all()


@pytest.mark.parametrize("V", [9, 1031, 60000, 300001])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_logits_of_minus_infinity_and_extremes(V, dtype):
    """-inf and the type's lowest value have no probability (a masked vocabulary); a
    row with one finite logit has log-probability 0 there; a row of nothing but -inf gives
    lse = -inf, logp = NaN; huge logits do not overflow."""
    low = torch.finfo(dtype).min
    x, tokens = _logits(1, 6, V, dtype)
    x[0, 0, ::2] = float("-inf")
    tokens[0, 0] = 1
    x[0, 1] = float("-inf")
    x[0, 1, V - 1], tokens[0, 1] = 5.0, V - 1
    x[0, 2] = float("-inf")
    x[0, 3, :V - 2] = low
    tokens[0, 3] = V - 2
    x[0, 4] = 60000.0
    x[0, 4, 3], tokens[0, 4] = 60160.0, 3
    tokens[0, 5] = 2
    x[0, 5, 2] = float("-inf")                          # the token itself has none
    logp, lse = ref.logprob(x.double(), tokens, 1.0)
    a, b = (torch.empty(1, 6, device="cuda") for _ in range(2))
    dps.dp_token_logprob(x.cuda(), tokens.cuda(), a, b)
    a, b = a.double().cpu(), b.double().cpu()
    tol = ref.logprob_bound(torch.where(x.double().abs() > 1e5, 0.0, x.double()), 1.0)
    rows = [0, 1, 3, 4]
    assert ((a - logp)[0, rows].abs() <= tol).all() and ((b - lse)[0, rows].abs() <= tol).all()
    assert torch.isnan(a[0, 2]) and b[0, 2] == float("-inf")
    assert a[0, 5] == float("-inf") and abs(b[0, 5] - lse[0, 5]) <= tol
    dlogp = torch.ones(1, 6)
    dlogp[0, 2] = 0.0
    dl = torch.empty(1, 6, V, dtype=dtype, device="cuda")
    dps.dp_token_logprob_backward(x.cuda(), tokens.cuda(), b.float().cuda(), dlogp.cuda(), dl)
    g, p = ref.logit_grad(x.double(), tokens, 1.0, b, dlogp.double())
    g[0, 2] = 0
    fin = torch.where(x.double().abs() > 1e5, 0.0, x.double())
    close(dl, g, stored(g, torch.nan_to_num(ref.logit_grad_bound(p, fin, 1.0, dlogp.double(), 0.0)), dtype))


# ---------------------------------------------------------------- the policy loss
def _policy_bound(want, logits, alpha, tol):
    """dlogits: the slope's ratio is off by the log-probability's error (and the
    exponential's few U), p by its own; slopes are at most q |A| + beta |e^d - 1|."""
    _, _, dlogp, g, p = want
    d = dlogp.abs()
    # d(slope) <= (|slope| + w beta) * 2 tol, and w beta is below the caller's bound on w here
    return ref.logit_grad_bound(p, logits, alpha, dlogp, tol) + ((d + 1.0) * (2 * tol + 16 * U) * alpha).unsqueeze(-1) * (p + (g != 0))


POLICY = [(1, 1, 1), (2, 5, 7), (4, 33, 1000), (1, 3, 50257), (2, 4, 32000), (1, 2, 131073), (1, 1, 300001),
          (3, 130, 64)]


def _policy_inputs(P, T, V, dtype, masked, lo=0.2, hi=0.28, alpha=1.0):
    x, tokens = _logits(P, T, V, dtype, seed=9)
    g = gen(P * T)
    logp, _ = ref.logprob(x.double(), tokens, alpha)
    moved = 0.3 * torch.randn(P, T, generator=g, dtype=torch.float64)
    for b in (np.log(1 - lo), np.log(1 + hi)):         # away from the clamp's corners
        moved = torch.where((moved - b).abs() < 1e-2, moved + 3e-2, moved)
    old = (logp - moved).float()
    rf = (logp + 0.3 * torch.randn(P, T, generator=g, dtype=torch.float64)).float()
    adv = torch.randn(P, T, generator=g)
    w = torch.rand(P, T, generator=g)
    if masked:
        w[torch.rand(P, T, generator=g) < 0.4] = 0.0
        w[0] = 0.0                                     # a rank whose mask leaves nothing
        x[w == 0] = float("nan")
        if T > 1:
            tokens[-1, 0] = -1
            x[-1, 0] = float("inf")
    return x, tokens, old, rf, adv, w


@pytest.mark.parametrize("P,T,V", POLICY, ids=str)
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("masked", [False, True])
def test_policy_loss(P, T, V, dtype, masked):
    beta, lo, hi, alpha = 0.1, 0.2, 0.28, float(np.float32(1.1))
    x, tokens, old, rf, adv, w = _policy_inputs(P, T, V, dtype, masked, lo, hi, alpha)
    clean = torch.nan_to_num(x.double(), posinf=0.0)
    want = ref.policy(clean, tokens, old.double(), rf.double(), adv.double(), w.double(), lo, hi, beta, alpha)
    tol = ref.logprob_bound(clean, alpha)
    cfg = dps.policy_cfg(lo, hi, beta, alpha)
    logp, stats = torch.full((P, T), float("nan"), device="cuda"), torch.full((P, 4), float("nan"), device="cuda")
    xd = x.cuda()
    dl = torch.full_like(xd, float("nan"))
    args = (tokens.cuda(), old.cuda(), adv.cuda(), logp, stats)
    kw = dict(ref_logp=rf.cuda(), weight=w.cuda(), cfg=cfg)
    dps.dp_policy_loss(xd, *args, dlogits=dl, **kw)
    close(logp, want[1], tol)
    # a row's terms move by at most (q |A| + beta |e^d - 1|) times the log-probability's
    # error, and carry a few U of their own; q <= e^1.5, |A| and |d| below 5 here
    q = torch.exp((want[1] - old.double()))
    row = w.double() * ((q * adv.double().abs() + 3.0) * (2 * tol + 32 * U))
    row = torch.where((want[2] != 0) | (w > 0), row, torch.zeros_like(row)).sum(1, keepdim=True)
    close(stats, want[0], row + U * want[0].abs())
    close(dl, want[3], stored(want[3], _policy_bound(want, clean, alpha, tol), dtype))
    # forward only, and in place
    l2, s2 = torch.empty_like(logp), torch.empty_like(stats)
    dps.dp_policy_loss(xd, args[0], args[1], args[2], l2, s2, **kw)
    assert torch.equal(l2, logp) and torch.equal(s2, stats)
    dps.dp_policy_loss(xd, args[0], args[1], args[2], l2, s2, dlogits=xd, **kw)
    assert torch.equal(bits(xd), bits(dl)) and torch.equal(l2, logp) and torch.equal(s2, stats)


def test_policy_loss_without_reference_or_weight():
    P, T, V = 2, 21, 333
    x, tokens, old, rf, adv, _ = _policy_inputs(P, T, V, F32, False)
    logp, stats, dl = torch.empty(P, T, device="cuda"), torch.empty(P, 4, device="cuda"), torch.empty(P, T, V, device="cuda")
    for r in (None, rf):                               # with one, beta = 0: the KL term is only reported
        want = ref.policy(x.double(), tokens, old.double(), None if r is None else r.double(), adv.double(), None,
                          0.2, 0.2, 0.0, 1.0)
        dps.dp_policy_loss(x.cuda(), tokens.cuda(), old.cuda(), adv.cuda(), logp, stats, dlogits=dl,
                           ref_logp=None if r is None else r.cuda())
        tol = ref.logprob_bound(x.double(), 1.0)
        q = torch.exp(want[1] - old.double())
        row = ((q * adv.double().abs() + 3.0) * (2 * tol + 32 * U)).sum(1, keepdim=True)
        close(stats, want[0], row + U * want[0].abs())
        close(dl, want[3], stored(want[3], _policy_bound(want, x.double(), 1.0, tol), F32))
        assert r is not None or (stats[:, 2] == 0).all()


def test_policy_loss_of_no_rows():
    stats = torch.full((3, 4), 9.0, device="cuda")
    e = torch.zeros(3, 0, device="cuda")
    dps.dp_policy_loss(torch.zeros(3, 0, 5, device="cuda"), torch.zeros(3, 0, dtype=torch.int64, device="cuda"), e, e,
                       e, stats)
    assert (stats == 0).all()


def test_policy_gradient_by_differences():
    """Kernel against kernel: a step along random directions of the fp32 logits changes the
    loss by <dlogits, step> (central, step 1e-2: truncation ~1e-5 relative, cancellation
    ~ 2 U |loss| sqrt(rows) / 1e-2 below 1e-4)."""
    P, T, V = 1, 12, 40
    x, tokens, old, rf, adv, w = _policy_inputs(P, T, V, F32, False)
    w = w / w.sum()
    kw = dict(ref_logp=rf.cuda(), weight=w.cuda(), cfg=dps.policy_cfg(0.2, 0.28, 0.1))
    logp, stats, dl = torch.empty(P, T, device="cuda"), torch.empty(P, 4, device="cuda"), torch.empty(P, T, V, device="cuda")
    t = (tokens.cuda(), old.cuda(), adv.cuda())
    dps.dp_policy_loss(x.cuda(), *t, logp, stats, dlogits=dl, **kw)
    h = 1e-3
    for seed in range(4):
        d = rnd(gen(50 + seed), P, T, V)
        d = d / d.norm()
        loss = []
        for s in (h, -h):
            lp, st = torch.empty_like(logp), torch.empty_like(stats)
            dps.dp_policy_loss((x + s * d).cuda(), *t, lp, st, **kw)
            loss.append(float(st[0, 0].double()))
        num, got = (loss[0] - loss[1]) / (2 * h), float((dl.cpu().double() * d.double()).sum())
        assert abs(num - got) <= 2e-3 * float(dl.norm()) + 1e-4, (num, got)


def test_cross_entropy_is_logprob_with_a_mean():
    """dlogp = -1/n gives torch's cross-entropy gradient (computed in 64 bits)."""
    P, T, V = 2, 8, 501
    x, tokens = _logits(P, T, V, F32)
    xd = x.double().requires_grad_()
    torch.nn.functional.cross_entropy(xd.flatten(0, 1), tokens.flatten()).backward()
    lp, lse, dl = torch.empty(P, T, device="cuda"), torch.empty(P, T, device="cuda"), torch.empty(P, T, V, device="cuda")
    dps.dp_token_logprob(x.cuda(), tokens.cuda(), lp, lse)
    dlogp = torch.full((P, T), -1.0 / (P * T))
    dps.dp_token_logprob_backward(x.cuda(), tokens.cuda(), lse, dlogp.cuda(), dl)
    p = torch.softmax(x.double(), -1)
    bound = ref.logit_grad_bound(p, x.double(), 1.0, dlogp.double(), ref.logprob_bound(x.double(), 1.0))
    close(dl, xd.grad, stored(xd.grad, bound, F32))


# ---------------------------------------------------------------- streams and graphs
def test_whole_step_on_another_stream_and_captured():
    """Lookup, policy loss and embedding gradient enqueued on a side stream give the bits
    of the default stream, and so does their captured graph on new inputs."""
    P, T, V, D = 2, 40, 700, 64
    table = rnd(gen(30), P, V, D, dtype=BF).cuda()
    tokens = torch.randint(0, V, (P, T), generator=gen(31)).cuda()
    old, adv = rnd(gen(32), P, T, std=0.1).cuda() - 6, rnd(gen(33), P, T).cuda()
    state = torch.tensor([3, 4], device="cuda")
    cfg = dps.dropout_cfg(0.1, 0, 0, seed_dev=state)
    ws = dps.new_embedding_workspace(P, T, V, D)

    def make():
        return (torch.empty(P, T, D, dtype=BF, device="cuda"), torch.empty(P, T, V, dtype=BF, device="cuda"),
                torch.empty(P, T, device="cuda"), torch.empty(P, 4, device="cuda"),
                torch.empty(P, V, D, dtype=BF, device="cuda"))

    def step(x, dl, lp, st, grad, stream=None):
        dps.dp_embedding_forward(table, tokens, x, scale=2.0, dropout=cfg, stream=stream)
        torch.matmul(x, table.transpose(1, 2), out=dl)
        dps.dp_policy_loss(dl, tokens, old, adv, lp, st, dlogits=dl, stream=stream)
        torch.matmul(dl, table, out=x)
        dps.dp_embedding_backward(x, tokens, grad, ws, scale=2.0, dropout=cfg, stream=stream)

    want = make()
    step(*want)
    torch.cuda.synchronize()
    side, got = torch.cuda.Stream(), make()
    with torch.cuda.stream(side):
        step(*got)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    got = make()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(*got)
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    state.copy_(torch.tensor([3, 5]))
    tokens.copy_(torch.randint(0, V, (P, T), generator=gen(34)))
    graph.replay()
    got = [t.clone() for t in got]
    step(*want)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
