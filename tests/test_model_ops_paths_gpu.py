"""The operators at the ends of a training step at sizes that reach every variant their
rules choose between: rows by warps, by 128, 256 and 512 threads, by clusters, rows longer
than shared memory, empty embedding rows written beside the sort and beside the sums.
References in 64 bits on the GPU."""
import pytest
import torch

import gradient_sync_zero_gb300 as dps
import model_reference as ref
from model_reference import U, stored
from test_model_ops_gpu import BF, F32, _grad_by_torch, _policy_bound, bits

pytestmark = pytest.mark.gpu


def within(got, want, bound):
    bad = ~((got.double() - want).abs() <= bound)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:3].tolist())


# (P, T, V): rows of 2 to 16 KB in numbers (warps), 32 to 64 KB (256 threads), over 64 KB (512), few
# rows and long ones (clusters), past eight CTAs' shared memory
ROWS = [(2, 1100, 2501), (4, 520, 1030), (2, 1030, 8000), (1, 330, 9001), (2, 160, 20011), (1, 320, 50257),
        (1, 2, 500001), (1, 1, 1000003), (3, 1, 40000)]


@pytest.mark.parametrize("P,T,V", ROWS, ids=str)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_token_rows(P, T, V, dtype):
    g = torch.Generator(device="cuda")
    g.manual_seed(V)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")   # noqa: E731
    x = (3 * rnd(P, T, V)).to(dtype)
    tokens = torch.randint(0, V, (P, T), generator=g, device="cuda")
    at = tokens.unsqueeze(-1)
    x.scatter_(-1, at, (x.gather(-1, at).float() + 6).to(dtype))
    w = torch.rand(P, T, generator=g, device="cuda")
    w[:, 1::3] = 0.0
    x[w == 0] = float("nan")
    clean = torch.nan_to_num(x.double())
    logp, lse = ref.logprob(clean, tokens, 1.0)
    tol = ref.logprob_bound(clean, 1.0)
    live = w != 0
    glp, gls = torch.empty(P, T, device="cuda"), torch.empty(P, T, device="cuda")
    dps.dp_token_logprob(x, torch.where(live, tokens, -100), glp, gls)
    zero = torch.zeros_like(logp)
    within(glp, torch.where(live, logp, zero), tol)
    within(gls, torch.where(live, lse, zero), tol)

    dlogp = torch.where(live, rnd(P, T), torch.zeros(P, T, device="cuda"))
    want, p = ref.logit_grad(clean, tokens, 1.0, gls.double(), dlogp.double())
    dl = torch.full_like(x, float("nan"))
    dps.dp_token_logprob_backward(x, tokens, gls, dlogp, dl)
    within(dl, want, stored(want, ref.logit_grad_bound(p, clean, 1.0, dlogp.double(), 0.0), dtype))
    del want, p

    moved = 0.3 * rnd(P, T).double()
    for b in (0.8, 1.2):                          # away from the clamp's corners
        moved = torch.where((torch.exp(moved) - b).abs() < 1e-2, moved + 4e-2, moved)
    old, rf, adv = (logp - moved).float(), (logp + 0.3 * rnd(P, T)).float(), rnd(P, T)
    kw = dict(ref_logp=rf, weight=w, cfg=dps.policy_cfg(0.2, 0.2, 0.1))
    stats = torch.empty(P, 4, device="cuda")
    dps.dp_policy_loss(x, tokens, old, adv, glp, stats, dlogits=dl, **kw)
    want = ref.policy(clean, tokens, old.double(), rf.double(), adv.double(), w.double(), 0.2, 0.2, 0.1, 1.0)
    within(glp, want[1], tol)
    within(dl, want[3], stored(want[3], _policy_bound(want, clean, 1.0, tol), dtype))
    q = torch.exp(want[1] - old.double())
    row = torch.where(live, w.double() * ((q * adv.double().abs() + 3.0) * (2 * tol + 32 * U)), zero)
    within(stats, want[0], row.sum(1, keepdim=True) + U * want[0].abs())
    first = bits(dl)
    dps.dp_policy_loss(x, tokens, old, adv, glp, stats, dlogits=x, **kw)      # in place
    assert torch.equal(bits(x), first)


@pytest.mark.parametrize("V", [700, 5000, 70001])
@pytest.mark.parametrize("T", [6, 2100])
def test_far_rows(V, T):
    """Rows whose scaled maximum would overflow: of the lowest value alone (uniform), of
    huge values, and with a +inf (NaN), in place; among ordinary rows, in every group size."""
    if T > 6 and V > 5000:
        V = 9000
    g = torch.Generator(device="cuda")
    g.manual_seed(V)
    x = torch.randn(1, T, V, generator=g, device="cuda")
    low = torch.finfo(torch.float32).min
    x[0, 1] = low
    x[0, 2] = 1e38
    x[0, 2, V // 2] = 1.5e38
    x[0, 3, 5] = float("inf")
    tokens = torch.full((1, T), V // 2, device="cuda")
    lp, le = torch.empty(1, T, device="cuda"), torch.empty(1, T, device="cuda")
    dps.dp_token_logprob(x, tokens, lp, le, logit_scale=2.0)
    logv = torch.log(torch.tensor(float(V), dtype=torch.float64))
    assert abs(float(lp[0, 1]) + float(logv)) < 1e-5 * float(logv) and float(lp[0, 2]) == 0.0
    assert torch.isnan(lp[0, 3])
    ok = [0] + list(range(4, T))
    want, _ = ref.logprob(x[:, ok].double(), tokens[:, ok], 2.0)
    within(lp[:, ok], want, ref.logprob_bound(x[:, ok].double(), 2.0))
    old, adv = torch.where(torch.isfinite(lp), lp, 0.0), torch.ones(1, T, device="cuda")
    stats = torch.empty(1, 4, device="cuda")
    dps.dp_policy_loss(x, tokens, old, adv, lp, stats, dlogits=x, cfg=dps.policy_cfg(logit_scale=2.0))
    # q = 1: dlogits = -2 (1[v = token] - p); p is 1 / V, or 1 at the largest
    row = torch.full((V,), 2.0 / V, dtype=torch.float64, device="cuda")
    row[V // 2] -= 2.0
    assert ((x[0, 1].double() - row).abs() <= 1e-5 * row.abs()).all()
    assert (x[0, 2] == 0).all() and torch.isnan(x[0, 3]).any()


# empty rows: all beside the sort, split between the launches, short rows, rows off 16-byte
# boundaries, several chunks (all beside the sums)
SLOTS = [(2, 500, 300, 256), (2, 500, 60000, 256), (2, 500, 60000, 251), (2, 300, 400000, 16), (1, 3000, 90000, 136),
         (2, 17000, 30000, 24), (64, 40, 500, 72), (1, 16384, 97, 100), (1, 16385, 97, 100)]


@pytest.mark.parametrize("P,T,V,D", SLOTS, ids=str)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_embedding_gradient_slots(P, T, V, D, dtype):
    g = torch.Generator(device="cuda")
    g.manual_seed(D)
    dout = torch.randn(P, T, D, generator=g, device="cuda").to(dtype)
    tokens = torch.randint(0, V, (P, T), generator=g, device="cuda", dtype=torch.int32)
    tokens[:, ::5] = V - 1                            # the slot's last row
    tokens[:, 1::7] = 0
    tokens[-1, T // 2:] = -1
    want, mag, n = _grad_by_torch(dout, tokens, V)
    plan = dps.Plan([11, V * D, 7], 1 << 34, P)
    buf = torch.full((P, plan.stride), 5.0, dtype=dtype, device="cuda")
    view = plan.tensor_view(buf, 1, (V, D))
    view.fill_(float("nan"))
    ws = dps.new_embedding_workspace(P, T, V, D)
    ws.fill_(0xFF)
    dps.dp_embedding_backward(dout, tokens, view, ws)
    within(view, want, stored(want, (n + 4) * U * mag, dtype))
    o = plan.tensor(1)[1]
    assert (buf[:, :o] == 5).all() and (buf[:, o + V * D:] == 5).all()
    once = view.clone()
    dps.dp_embedding_backward(dout, tokens, view, ws)
    assert torch.equal(once, view)


def test_vectors_that_overlap_are_refused():
    x = torch.zeros(1, 4, 8, device="cuda")
    t = torch.zeros(1, 4, dtype=torch.int64, device="cuda")
    a, b = torch.zeros(1, 4, device="cuda"), torch.zeros(1, 4, device="cuda")
    stats = torch.zeros(1, 4, device="cuda")
    with pytest.raises(dps.DPError, match="overlap"):
        dps.dp_token_logprob(x, t, a, a)
    for old, adv, w, rf in ((a, b, None, None), (b, a, None, None), (b, b, a, None), (b, b, None, a)):
        with pytest.raises(dps.DPError, match="overlap"):
            dps.dp_policy_loss(x, t, old, adv, a, stats, ref_logp=rf, weight=w)
    with pytest.raises(dps.DPError, match="overlap"):
        dps.dp_policy_loss(x, t, b, b, a, a.view(1, 4))
