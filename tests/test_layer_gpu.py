"""The dense layer, its gradients, the orthogonalisation and the Muon step on the GPU, against
plain 64-bit implementations on the host, with bounds derived from the kernels' arithmetic
(layer_reference.py)."""
import os
import subprocess
import sys

import pytest
import torch

import gradient_sync_zero_gb300 as dps
import layer_reference as ref
from layer_reference import ROUND, U, stored

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
ACT = dict(zip(ref.ACTS, range(5)))
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(autouse=True)
def no_timeouts():
    yield
    assert dps.dp_product_timeouts(reset=True) == 0


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def rnd(g, *shape, dtype=BF, std=1.0):
    return (torch.randn(*shape, generator=g) * std).to(dtype)


def close(got, want, bound):
    got = got.detach().double().cpu()
    bad = ~((got - want).abs() <= bound)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:3].tolist(), got[bad][:3].tolist(), want[bad][:3].tolist(),
                           bound.expand_as(want)[bad][:3].tolist())


def strided(t, row_pad, rank_pad=0, lead=0):
    """A CUDA copy of [P, T, D] `t` with rows D + row_pad apart, rank_pad elements more between
    ranks, its first element `lead` elements into its buffer.  Everything around it is NaN."""
    P, T, D = t.shape
    row, rank = D + row_pad, T * (D + row_pad) + rank_pad
    buf = torch.full((lead + P * rank + 64,), float("nan"), dtype=t.dtype, device="cuda")
    v = buf.as_strided((P, T, D), (rank, row, 1), lead)
    v.copy_(t)
    return v, buf


def untouched(buf, view):
    """What lies around a view is still NaN."""
    b = buf.clone()
    b.as_strided(view.shape, view.stride(), view.storage_offset()).fill_(float("nan"))
    return bool(torch.isnan(b).all())


def forward(x, w, dt=BF, zt=BF, bias=None, residual=None, kind="none", keep=True, **kw):
    P, T, N = x.shape[0], x.shape[1], w.shape[1]
    y = torch.full((P, T, N), float("nan"), dtype=dt, device="cuda")
    z = torch.full((P, T, N), float("nan"), dtype=zt, device="cuda") if keep else None
    dps.dp_linear_forward(x, w, y, bias=bias, residual=residual, z=z, act=ACT[kind], ws=dps.new_linear_workspace(x, w))
    return y, z


# P, T, in_dim, out_dim: one token to several tiles, K below, at and off the copies' 64, odd sizes,
# tiles that end inside, tokens as columns (up to 128 rows) and as rows, K cut in parts
SHAPES = [(1, 1, 1, 1), (2, 1, 64, 256), (1, 3, 200, 40), (3, 48, 333, 129), (1, 64, 4096, 256), (2, 65, 96, 300),
          (1, 128, 1024, 64), (2, 129, 72, 33), (1, 257, 63, 255), (3, 333, 257, 131), (2, 512, 640, 520),
          (1, 1100, 130, 7), (1, 5, 2048, 5632), (64, 2, 24, 17), (1, 2304, 65, 2200)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward_plain(shape):
    P, T, K, N = shape
    g = gen(1)
    x, w = rnd(g, P, T, K), rnd(g, P, N, K, std=0.05)
    y, z = forward(x.cuda(), w.cuda(), dt=F32, zt=BF)
    want, _, err, _ = ref.linear(x.double(), w.double())
    close(y, want, stored(want, err, F32))
    close(z, want, stored(want, err, BF))


@pytest.mark.parametrize("kind", ref.ACTS)
@pytest.mark.parametrize("shape", [(2, 17, 72, 40), (2, 300, 96, 77), (1, 520, 64, 512)], ids=str)
@pytest.mark.parametrize("dt,zt,rt", [(BF, BF, BF), (F32, BF, F32), (BF, F32, F32)])
def test_forward_bias_activation_residual(shape, kind, dt, zt, rt):
    P, T, K, N = shape
    g = gen(2)
    x, w, b = rnd(g, P, T, K), rnd(g, P, N, K, std=0.3), rnd(g, P, N)
    r = rnd(g, P, T, N, dtype=rt)
    y, z = forward(x.cuda(), w.cuda(), dt, zt, b.cuda(), r.cuda(), kind)
    wy, wz, ey, ez = ref.linear(x.double(), w.double(), b.double(), r.double(), kind)
    close(y, wy, stored(wy, ey, dt))
    close(z, wz, stored(wz, ez, zt))
    only, _ = forward(x.cuda(), w.cuda(), dt, zt, b.cuda(), None, kind, keep=False)
    wy, _, ey, _ = ref.linear(x.double(), w.double(), b.double(), None, kind)
    close(only, wy, stored(wy, ey, dt))


# rows on 16-byte boundaries or off them, in x, in w, in the outputs; gaps between ranks
@pytest.mark.parametrize("pads", [(8, 8, 8, 0), (1, 0, 0, 0), (0, 3, 0, 0), (5, 1, 7, 1), (0, 0, 3, 2), (16, 24, 1, 5)],
                         ids=str)
@pytest.mark.parametrize("T", [20, 300])
def test_forward_strides(pads, T):
    px, pw, py, lead = pads
    P, K, N = 3, 104, 88
    g = gen(3)
    x, w, r = rnd(g, P, T, K), rnd(g, P, N, K, std=0.1), rnd(g, P, T, N)
    xs, _ = strided(x, px, px * 8, lead)
    ws_, _ = strided(w, pw, pw * 16, lead)
    ys, ybuf = strided(r, py, 40, lead)                     # y is the residual itself
    zs, zbuf = strided(torch.zeros(P, T, N), py, 8, lead)
    dps.dp_linear_forward(xs, ws_, ys, residual=ys, z=zs, act=dps.DP_ACT_SILU, ws=dps.new_linear_workspace(xs, ws_))
    wy, wz, ey, ez = ref.linear(x.double(), w.double(), None, r.double(), "silu")
    close(ys, wy, stored(wy, ey, BF))
    close(zs, wz, stored(wz, ez, F32))
    assert untouched(ybuf, ys) and untouched(zbuf, zs)


def test_weights_shared_between_ranks():
    """rank_stride 0 for w and the bias: one weight for all ranks."""
    g = gen(4)
    x, w, b = rnd(g, 3, 200, 64), rnd(g, 1, 96, 64, std=0.2), rnd(g, 1, 96)
    y, _ = forward(x.cuda(), w.cuda().expand(3, 96, 64), F32, bias=b.cuda().expand(3, 96))
    want, _, err, _ = ref.linear(x.double(), w.double().expand(3, 96, 64), b.double().expand(3, 96))
    close(y, want, stored(want, err, F32))


@pytest.mark.parametrize("T", [3, 300])
def test_ranks_inside_rows_and_rows_shown_twice(T):
    """[T, P, K] seen as [P, T, K], and one row expanded to T."""
    g = gen(20)
    x, w = rnd(g, T, 3, 64), rnd(g, 3, 40, 64, std=0.2)
    y = torch.full((T, 3, 40), float("nan"), device="cuda").transpose(0, 1)
    xs, wc = x.cuda().transpose(0, 1), w.cuda()
    dps.dp_linear_forward(xs, wc, y, ws=dps.new_linear_workspace(xs, wc))
    want, _, err, _ = ref.linear(x.double().transpose(0, 1), w.double())
    close(y, want, stored(want, err, F32))
    one = rnd(g, 3, 1, 64)
    y, _ = forward(one.cuda().expand(3, T, 64), wc, F32)
    want, _, err, _ = ref.linear(one.double().expand(3, T, 64), w.double())
    close(y, want, stored(want, err, F32))
    dy, dw = rnd(g, 3, 1, 40), torch.empty(3, 40, 64, device="cuda")
    dps.dp_linear_backward(dy.cuda().expand(3, T, 40), xs, wc, dw=dw, ws=dps.new_linear_workspace(xs, wc, True))
    (_, want, _), (_, err, _) = ref.linear_grad(dy.double().expand(3, T, 40), None, x.double().transpose(0, 1), w.double())
    close(dw, want, stored(want, err, F32))


def test_long_sums_in_fp32():
    """K past the lengths where a tile takes two and four accumulators."""
    g = gen(5)
    for T, K, N in ((140, 6000, 40), (3000, 4200, 1600), (2600, 9000, 1500)):
        x, w = rnd(g, 1, T, K), rnd(g, 1, N, K)
        y, _ = forward(x.cuda(), w.cuda(), F32, keep=False)
        want = x.double().cuda() @ w.double().cuda().mT
        # norm against norm: sums cut off at 2^-23 of themselves per 16 products, in parts of 4096
        assert (y - want).norm() <= 4096 / 16 * 2.0 ** -24 * want.norm()


def test_values_out_of_range_stay_in_their_rows():
    g = gen(6)
    for T in (40, 400):
        x, w = rnd(g, 2, T, 72), rnd(g, 2, 50, 72)
        x[0, 3, 5], x[1, T - 1, 71], x[1, 7, 0] = float("nan"), float("inf"), float("-inf")
        y, z = forward(x.cuda(), w.cuda(), F32, F32)
        rows = torch.zeros(2, T, dtype=torch.bool)
        rows[0, 3] = rows[1, T - 1] = rows[1, 7] = True
        assert not torch.isfinite(y.cpu()[rows]).any() and torch.isfinite(y.cpu()[~rows]).all()


@pytest.mark.parametrize("kind", ref.ACTS)
def test_activations_of_extreme_arguments(kind):
    """Through an identity weight: z is x exactly."""
    vals = torch.tensor([0.0, -0.0, 1e-38, -1e-30, 0.5, -0.5, 3.0, -3.0, 9.0, -9.0, 14.0, -14.0, 100.0, -100.0, 1e4, -1e4,
                         1e18, -1e18, 3e38, -3e38]).to(BF)
    n = vals.numel()
    x, w = torch.diag(vals).unsqueeze(0), torch.eye(n, dtype=BF).unsqueeze(0)
    x, w = x.cuda(), w.cuda()
    y, z = forward(x, w, F32, F32, kind=kind)
    assert torch.equal(torch.diagonal(z[0]).cpu(), vals.float())
    want = ref.act(vals.double(), kind)
    got = torch.diagonal(y[0]).double().cpu()
    assert ((got - want).abs() <= 32 * U * want.abs() + 64 * U * (vals.double().abs() < 20) + 1e-37).all(), (got, want)
    dy = torch.ones_like(y)
    db = torch.empty(1, n, device="cuda")
    dps.dp_linear_backward(dy, x, w, dbias=db, z=torch.diagonal(z[0]).view(1, 1, n).expand(1, n, n).contiguous(), act=ACT[kind],
                           ws=dps.new_linear_workspace(x, w, True))
    slope = ref.act_slope(vals.double().clamp(-100, 100), kind)
    assert ((db[0].double().cpu() / n - slope).abs() <= ref.act_error(vals.double().clamp(-20, 20))).all()


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_backward_plain(shape):
    """No activation and bf16 dy: nothing is rounded before the products."""
    P, T, K, N = shape
    g = gen(7)
    x, w, dy = rnd(g, P, T, K), rnd(g, P, N, K, std=0.05), rnd(g, P, T, N)
    xc, wc = x.cuda(), w.cuda()
    nan = lambda *s: torch.full(s, float("nan"), device="cuda")   # noqa: E731
    dx, dw, db = nan(P, T, K), nan(P, N, K), nan(P, N)
    dps.dp_linear_backward(dy.cuda(), xc, wc, dx=dx, dw=dw, dbias=db, ws=dps.new_linear_workspace(xc, wc, True))
    for got, want, err in zip((dx, dw, db), *ref.linear_grad(dy.double(), None, x.double(), w.double())):
        close(got, want, stored(want, err, F32))


@pytest.mark.parametrize("kind", ref.ACTS)
@pytest.mark.parametrize("dyt,zt,gt", [(BF, BF, BF), (F32, F32, F32), (F32, BF, BF)])
def test_backward_activation(kind, dyt, zt, gt):
    P, T, K, N = 2, 300, 77, 136
    g = gen(8)
    x, w = rnd(g, P, T, K), rnd(g, P, N, K, std=0.2)
    dy, z = rnd(g, P, T, N, dtype=dyt), rnd(g, P, T, N, dtype=zt, std=1.5)
    xc, wc = x.cuda(), w.cuda()
    dx, dw, db = (torch.empty(*s, dtype=gt, device="cuda") for s in ((P, T, K), (P, N, K), (P, N)))
    dps.dp_linear_backward(dy.cuda(), xc, wc, dx=dx, dw=dw, dbias=db, z=z.cuda(), act=ACT[kind],
                           ws=dps.new_linear_workspace(xc, wc, True))
    rounds = kind != "none" or dyt == F32
    wants, errs = ref.linear_grad(dy.double(), z.double(), x.double(), w.double(), kind, rounds)
    for got, want, err in zip((dx, dw, db), wants, errs):
        close(got, want, stored(want, err, gt))
        # the roundings of dz are independent of each other: no drift, norm against norm
        assert (got.double().cpu() - want).norm() <= 2 * ROUND[BF] * want.norm()


def test_backward_accumulates_into_replica_slots():
    P, T, K, N = 3, 150, 64, 72
    plan = dps.Plan([1000, N * K, N, 77], 1 << 20, P)
    params, grads = plan.new_replicas(), plan.new_replicas()
    g = gen(9)
    params.copy_(rnd(g, P, plan.stride, std=0.1))
    old = rnd(g, P, plan.stride)
    grads.copy_(old)
    w, dw, db = plan.tensor_view(params, 1, (N, K)), plan.tensor_view(grads, 1, (N, K)), plan.tensor_view(grads, 2, (N,))
    x, dy = rnd(g, P, T, K), rnd(g, P, T, N)
    xc = x.cuda()
    before = (plan.tensor_view(old, 1, (N, K)), plan.tensor_view(old, 2, (N,)))
    dx = torch.empty_like(xc)
    dps.dp_linear_backward(dy.cuda(), xc, w, dx=dx, dw=dw, dbias=db, accumulate=True,
                           ws=dps.new_linear_workspace(xc, w, True))
    wants, errs = ref.linear_grad(dy.double(), None, x.double(), w.double().cpu())
    close(dx, wants[0], stored(wants[0], errs[0], BF))
    for got, want, err, b in zip((dw, db), wants[1:], errs[1:], before):
        want, err = want + b.double(), err + 2 * U * (want.abs() + b.double().abs())
        close(got, want, stored(want, err, BF))
    rest = grads.cpu()
    for t, s in ((1, (N, K)), (2, (N,))):
        plan.tensor_view(rest, t, s).copy_(plan.tensor_view(old, t, s))
    assert torch.equal(rest.view(torch.int16), old.view(torch.int16))


@pytest.mark.parametrize("accumulate", [False, True])
def test_no_tokens(accumulate):
    x = torch.empty(2, 0, 24, dtype=BF, device="cuda")
    w = torch.randn(2, 40, 24, device="cuda").to(BF)
    y = torch.empty(2, 0, 40, device="cuda")
    dps.dp_linear_forward(x, w, y)
    dw, db = torch.ones(2, 40, 24, device="cuda"), torch.ones(2, 40, device="cuda")
    dps.dp_linear_backward(y, x, w, dx=x.clone(), dw=dw, dbias=db, accumulate=accumulate,
                           ws=dps.new_linear_workspace(x, w, True))
    assert (dw == int(accumulate)).all() and (db == int(accumulate)).all()


def test_single_outputs_and_same_bits():
    """Each output alone equals its part of the whole call, twice."""
    g = gen(10)
    P, T, K, N = 2, 700, 96, 160
    x, w, dy, z = (t.cuda() for t in (rnd(g, P, T, K), rnd(g, P, N, K), rnd(g, P, T, N), rnd(g, P, T, N)))
    ws = dps.new_linear_workspace(x, w, True)
    new = lambda: [torch.empty(*s, dtype=BF, device="cuda") for s in ((P, T, K), (P, N, K), (P, N))]   # noqa: E731
    whole = new()
    dps.dp_linear_backward(dy, x, w, *whole, z=z, act=dps.DP_ACT_GELU, ws=ws)
    for _ in range(2):
        parts = new()
        for i in range(3):
            ws.fill_(255)
            args = [None] * 3
            args[i] = parts[i]
            dps.dp_linear_backward(dy, x, w, *args, z=z, act=dps.DP_ACT_GELU, ws=ws)
        for a, b in zip(whole, parts):
            assert torch.equal(a, b)


# ---------------------------------------------------------------- orthogonalisation
def emulated(x, steps, coefs=ref.COEFS):
    """The tensor-core path's roundings in 64 bits: fp16 operands, the iterate as a pair."""
    a, b, c = coefs
    h = lambda t: t.half().double()   # noqa: E731
    tall = x.shape[0] > x.shape[1]
    x = x.mT if tall else x
    m, n = x.shape
    S = 1.0
    while S < 32768 and 2 * S * S < m * n:
        S *= 2
    x = x / x.norm() * S
    for _ in range(steps):
        hi = h(x)
        gram = h(hi @ hi.mT / S ** 2)
        q = h(b * gram + c * (gram @ gram))
        x = a * (hi + h(x - hi)) + q @ hi
    return (x.mT if tall else x) / S


def spectrum(g, rows, cols, kind):
    x = torch.randn(rows, cols, generator=g, dtype=torch.float64)
    if kind == "decay":      # singular values 1, 1/2, 1/3 ...
        u, s, v = torch.linalg.svd(x, full_matrices=False)
        x = u @ torch.diag(1.0 / torch.arange(1, len(s) + 1, dtype=torch.float64)) @ v
    if kind == "rank 1":
        x = torch.outer(x[:, 0], x[0])
    return x


SMALL = [(1, 1), (1, 7), (9, 1), (3, 5), (16, 16), (48, 131), (131, 48), (64, 64), (61, 64), (2, 900), (64, 320), (100, 90)]


@pytest.mark.parametrize("shape", SMALL, ids=str)
@pytest.mark.parametrize("dt", [BF, F32])
def test_orthogonalize_small(shape, dt):
    """In fp32 throughout: a step's sums of at most n terms are off by n U of their terms'
    magnitudes and the steepest step takes errors up 3.5-fold, so five steps leave
    at most 5 * 3.5^5 * (n + 8) U of the norm, far below the rounding to bf16."""
    rows, cols = shape
    g = gen(11)
    x = torch.stack([spectrum(g, rows, cols, k) for k in ("noise", "decay", "rank 1")]).to(dt)
    want = ref.newton_schulz(x.double())
    out = torch.full((3, rows, cols), float("nan"), dtype=BF, device="cuda")
    dps.dp_orthogonalize(x.cuda(), out, dps.new_orthogonalize_workspace(3, rows, cols))
    err = 5 * 3.5 ** 5 * (max(shape) + 8) * U * want.flatten(1).norm(dim=1)[:, None, None]
    close(out, want, stored(want, err, BF))


LARGE = [(130, 130), (256, 256), (257, 300), (300, 257), (90, 700), (700, 90), (600, 520), (2, 20000), (20000, 3), (1000, 72),
         (64, 900), (1200, 50), (33, 40001), (64, 3001), (5000, 40)]


@pytest.mark.parametrize("shape", LARGE, ids=str)
@pytest.mark.parametrize("dt", [BF, F32])
def test_orthogonalize_one_step(shape, dt):
    """One step, whose error has a bound: G, Q and X each rounded to fp16 (2^-11 of an entry, or
    half a subnormal step), sums by sum_error."""
    rows, cols = shape
    g = gen(12)
    x = torch.stack([spectrum(g, rows, cols, k) for k in ("noise", "decay")]).to(dt)
    want = ref.newton_schulz(x.double(), 1)
    out = torch.full((2, rows, cols), float("nan"), dtype=BF, device="cuda")
    dps.dp_orthogonalize(x.cuda(), out, dps.new_orthogonalize_workspace(2, rows, cols), dps.newton_schulz_cfg(steps=1))
    a, b, c = ref.COEFS
    h, tiny = ROUND[torch.float16], 2.0 ** -25
    y = x.double() / x.double().flatten(1).norm(dim=1)[:, None, None]
    y = y.mT if rows > cols else y
    m, n = y.shape[1:]
    S = 1.0
    while S < 32768 and 2 * S * S < m * n:
        S *= 2
    ya = y.abs() * (1 + h) + tiny / S
    gram, mag = y @ y.mT, ya @ ya.mT
    eg = (2.1 * h) * mag + n * 2.1 * tiny / S * ya.max() + sum_error(mag, n)
    eg = eg + h * (gram.abs() + eg) + tiny
    ga = gram.abs() + eg
    eq = abs(b) * eg + c * (2 * eg @ ga + sum_error(ga @ ga, m)) + 4 * U * ga
    q = b * gram + c * gram @ gram
    eq = eq + h * (q.abs() + eq) + tiny
    qa = q.abs() + eq
    err = eq @ ya + qa @ (h * ya + tiny / S) + sum_error(qa @ ya, m) + 8 * U * (a * ya) + 2.0 ** -21 * ya
    err = err.mT if rows > cols else err
    close(out, want, stored(want, err, BF))


sum_error = ref.sum_error


@pytest.mark.parametrize("kind", ["noise", "decay", "rank 1"])
@pytest.mark.parametrize("shape", LARGE, ids=str)
def test_orthogonalize_five_steps(shape, kind):
    """Norm against norm, what the header says: 2e-3 and the rounding to bf16 (2^-8 at most, 1.7e-3 on
    the whole); and the same roundings done in 64 bits.  The sums differ by 2^-22 there, so operands near
    a rounding's border fall to either side (by 2^-10) and later roundings are drawn anew: the two
    are apart by sqrt(2) * 2e-3 from the operands and 1.7e-3 from the store, together 3.3e-3."""
    rows, cols = shape
    x = spectrum(gen(13), rows, cols, kind).to(F32)
    want = ref.newton_schulz(x.double())
    out = torch.full((1, rows, cols), float("nan"), dtype=BF, device="cuda")
    dps.dp_orthogonalize(x[None].cuda(), out, dps.new_orthogonalize_workspace(1, rows, cols))
    got = out[0].double().cpu()
    assert (got - want).norm() <= 2.7e-3 * want.norm()
    same = emulated(x.double(), 5)
    assert (got - same).norm() <= 3.3e-3 * same.norm()


@pytest.mark.parametrize("rows,cols", [(40, 60), (300, 200)])
def test_orthogonalize_layouts_scales_and_zeros(rows, cols):
    """Values whose squares leave fp32, zero and broken matrices beside good ones, off-boundary
    rows, in place."""
    g = gen(14)
    base = torch.randn(6, rows, cols, generator=g)
    x = base.clone()
    x[1] *= 1e30
    x[2] *= 1e-18          # the norm is above eps only if the squares did not vanish
    x[3] = 0.0
    x[4, 5, 6] = float("nan")
    x[5, 1, 1] = float("inf")
    x = x.to(BF)
    want = ref.newton_schulz(x[:3].double(), eps=1e-25)
    cfg = dps.newton_schulz_cfg(eps=1e-25)
    ws = dps.new_orthogonalize_workspace(6, rows, cols)
    xs, buf = strided(x, 3, 5, 1)
    out, obuf = strided(torch.zeros_like(x), 5, 3, 1)
    dps.dp_orthogonalize(xs, out, ws, cfg)
    for i in range(3):
        assert (out[i].double().cpu() - want[i]).norm() <= 2.7e-3 * want[i].norm(), i
    assert (out[3] == 0).all() and torch.isnan(out[4]).all() and torch.isnan(out[5]).all()
    assert untouched(obuf, out)
    keep = out.clone()
    if ws.numel():
        ws.fill_(255)
    dps.dp_orthogonalize(xs, xs, ws, cfg)
    assert torch.equal(xs[:4], keep[:4]) and untouched(buf, xs)


def test_orthogonalize_batches_in_parts():
    """More memory than a part of the batch may take: the same as one by one."""
    rows, cols, P = 2560, 10240, 9
    x = torch.randn(P, rows, cols, device="cuda", dtype=BF)
    out = torch.empty_like(x)
    ws = dps.new_orthogonalize_workspace(P, rows, cols)
    # nine at once: X and the next in fp16, what it leaves out in 8 bits, G and Q in fp16
    assert ws.numel() < 9 * (5 * rows * cols + 4 * rows * rows)
    dps.dp_orthogonalize(x, out, ws, dps.newton_schulz_cfg(steps=2))
    y = x / x.double().flatten(1).norm(dim=1)[:, None, None]
    for r in (0, P - 1):
        want = ref.newton_schulz_wide(y[r], 2, ref.COEFS)
        assert (out[r].double() - want).norm() <= 2.7e-3 * want.norm()


# ---------------------------------------------------------------- Muon
MUON = {0: (61, 64), 2: (300, 260), 3: (260, 300), 5: (64, 61), 6: (300, 260), 7: (17, 1)}


def muon_state(P=3, seed=15):
    sizes = [61 * 64, 1000, 300 * 260, 260 * 300, 77, 64 * 61, 300 * 260, 17]
    plan = dps.Plan(sizes, 1 << 17, P)
    g = gen(seed)
    mean, master, buf = (torch.randn(plan.L, generator=g) * s for s in (1e-3, 0.02, 1e-3))
    params = torch.randn(P, plan.stride, generator=g).to(BF)
    return plan, mean, master, buf, params


@pytest.mark.parametrize("nesterov", [True, False])
@pytest.mark.parametrize("scale,lr", [(dps.DP_MUON_MATCH_RMS, 1e-3), (dps.DP_MUON_SPECTRAL, 0.02)])
@pytest.mark.parametrize("clip", [None, "workspace", "caller"])
def test_muon_step(nesterov, scale, lr, clip):
    plan, mean, master, buf, params = muon_state()
    ws = plan.new_workspace()
    m = dps.Muon(plan, MUON)
    dev = [t.cuda() for t in (mean, master, buf, params)]
    coef, kw = 1.0, {}
    if clip:
        kw = dict(use_clip_coef=True)
        coef = 0.37109375                       # exact in fp32
        if clip == "caller":
            kw["coef_dev"] = torch.tensor([coef], device="cuda")
        at = dps.workspace_result_offsets()[2]
        ws[at:at + 4].view(torch.float32).fill_(coef if clip == "workspace" else 9.0)
    cfg = dps.muon_cfg(lr=lr, momentum=0.9, weight_decay=0.1, nesterov=nesterov, scale=scale)
    dps.dp_muon_step(m, ws, m.new_workspace(), dev[0], dev[1], dev[2], dev[3], cfg, **kw)
    status = dps.dp_read_norm(plan, ws, raise_on_status=False)[2]
    assert status == 0
    got_mean, got_master, got_buf, got_params = (t.cpu() for t in dev)
    assert torch.equal(got_mean, mean)
    left = torch.ones(plan.L, dtype=torch.bool)
    for t, (r, c) in MUON.items():
        o = plan.tensor(t)[1]
        at = slice(o, o + r * c)
        left[at] = False
        s = 0.2 * max(r, c) ** 0.5 if scale else max(1.0, r / c) ** 0.5
        w, b, orth = ref.muon(*(v[at].double().view(r, c) for v in (mean, buf, master)), lr, 0.9, 0.1, nesterov, s, coef=coef)
        assert ((got_buf[at].view(r, c) - b).abs() <= 4 * U * (buf[at].abs() + mean[at].abs()).view(r, c)).all(), t
        # the update within 2e-3 (in shared memory 1e-4), the master's own roundings beside it
        d = (got_master[at].double().view(r, c) - w).norm()
        assert d <= lr * s * (1e-4 if r * c < 5000 else 2e-3) * orth.norm() + 4 * U * master[at].norm(), t
        for p in range(plan.P):
            assert torch.equal(got_params[p, at], got_master[at].to(BF)), t
    assert torch.equal(got_master[left], master[left]) and torch.equal(got_buf[left], buf[left])
    rest = torch.cat([left, torch.ones(plan.stride - plan.L, dtype=torch.bool)])
    assert torch.equal(got_params[:, rest].view(torch.int16), params[:, rest].view(torch.int16))


def test_muon_lr_on_the_device():
    plan, mean, master, buf, params = muon_state()
    ws = plan.new_workspace()
    m = dps.Muon(plan, MUON)
    outs = []
    for kw in (dict(lr=3e-3), dict(lr=0.5, lr_dev=torch.tensor([3e-3], device="cuda"))):
        dev = [t.cuda() for t in (mean, master, buf, params)]
        dps.dp_muon_step(m, ws, m.new_workspace(), *dev, dps.muon_cfg(**kw))
        outs.append(dev)
    for a, b in zip(*outs):
        assert torch.equal(a, b)


def test_muon_not_finite_is_reported_and_stays_in_its_matrix():
    for t in (0, 2):
        plan, mean, master, buf, params = muon_state()
        ws = plan.new_workspace()
        m = dps.Muon(plan, MUON)
        o = plan.tensor(t)[1]
        mean[o + 7] = float("inf")
        dev = [v.cuda() for v in (mean, master, buf, params)]
        dps.dp_muon_step(m, ws, m.new_workspace(), *dev)
        with pytest.raises(dps.DPError) as e:
            dps.dp_read_norm(plan, ws)
        assert e.value.code == dps.DP_ENONFINITE
        for k, (r, c) in MUON.items():
            at = plan.tensor(k)[1]
            good = torch.isfinite(dev[1][at:at + r * c])
            assert good.all() if k != t else not good.any()


def test_muon_refuses_another_plans_workspace():
    plan, mean, master, buf, params = muon_state()
    other = dps.Plan([5000, 300000], 1 << 20, 3).new_workspace()
    ws = torch.zeros(max(other.numel(), plan.info.workspace_bytes), dtype=torch.uint8, device="cuda")
    ws[:other.numel()] = other
    m = dps.Muon(plan, MUON)
    dev = [t.cuda() for t in (mean, master, buf, params)]
    dps.dp_muon_step(m, ws, m.new_workspace(), *dev)
    at = dps.workspace_result_offsets()[3]
    assert int(ws[at:at + 4].view(torch.int32)) == dps.DP_STATUS_PLAN_MISMATCH
    for a, b in zip(dev, (mean, master, buf, params)):
        a = a.cpu()
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))


# ---------------------------------------------------------------- streams and graphs
def test_captured_and_replayed():
    """A layer's step in one graph, replayed on other inputs, equals the eager calls."""
    P, T, K, N = 2, 260, 128, 320
    plan = dps.Plan([N * K, N], 1 << 20, P)
    params, grads = plan.new_replicas(), plan.new_replicas()
    master, buf, mean = (plan.new_state() for _ in range(3))
    g = gen(16)
    params.copy_(rnd(g, P, plan.stride, std=0.1))
    x, r = rnd(g, P, T, K).cuda(), rnd(g, P, T, N).cuda()
    y, z, dx = torch.empty_like(r), torch.empty_like(r), torch.empty_like(x)
    pws, m = plan.new_workspace(), dps.Muon(plan, {0: (N, K)})
    lr = torch.tensor([1e-2], device="cuda")
    w = plan.tensor_view(params, 0, (N, K))
    ws, bws, mws = dps.new_linear_workspace(x, w), dps.new_linear_workspace(x, w, True), m.new_workspace()
    cfg = dps.muon_cfg(lr=0.0, lr_dev=lr)

    def step():
        dps.dp_linear_forward(x, w, y, bias=plan.tensor_view(params, 1, (N,)), residual=r, z=z, act=dps.DP_ACT_GELU, ws=ws)
        dps.dp_linear_backward(y, x, w, dx=dx, dw=plan.tensor_view(grads, 0, (N, K)),
                               dbias=plan.tensor_view(grads, 1, (N,)), z=z, act=dps.DP_ACT_GELU, ws=bws)
        dps.dp_reduce_scatter_mean(plan, pws, grads, mean)
        dps.dp_muon_step(m, pws, mws, mean, master, buf, params, cfg)

    state = [t.clone() for t in (params, grads, master, buf)]

    def reset():
        for t, s in zip((params, grads, master, buf), state):
            t.copy_(s)

    step()                                     # every kernel known before the capture
    torch.cuda.synchronize()
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        step()
    for k in range(3):
        x.copy_(rnd(g, P, T, K))
        r.copy_(rnd(g, P, T, N))
        lr.fill_(0.01 * (k + 1))
        reset()
        step()
        eager = [t.clone() for t in (y, z, dx, params, grads, master, buf)]
        reset()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(eager, (y, z, dx, params, grads, master, buf)):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_two_streams_at_once():
    """Two calls with a workspace each on streams of their own."""
    g = gen(17)
    x = [rnd(g, 1, 900, 320).cuda() for _ in range(2)]
    w = [rnd(g, 1, 700, 320).cuda() for _ in range(2)]
    o = [rnd(g, 1, 400, 300).cuda() for _ in range(2)]
    alone = []
    for i in range(2):
        y, _ = forward(x[i], w[i], keep=False)
        q = torch.empty_like(o[i])
        dps.dp_orthogonalize(o[i], q, dps.new_orthogonalize_workspace(1, 400, 300))
        alone += [y, q]
    streams = [torch.cuda.Stream() for _ in range(2)]
    ys = [torch.zeros(1, 900, 700, dtype=BF, device="cuda") for _ in range(2)]
    qs = [torch.zeros_like(t) for t in o]
    wss = [(dps.new_linear_workspace(x[i], w[i]), dps.new_orthogonalize_workspace(1, 400, 300)) for i in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for i in range(2):
            dps.dp_linear_forward(x[i], w[i], ys[i], ws=wss[i][0], stream=streams[i])
            dps.dp_orthogonalize(o[i], qs[i], wss[i][1], stream=streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(ys[i], alone[2 * i]) and torch.equal(qs[i], alone[2 * i + 1])


def test_binding_refuses_wrong_extents():
    x, w = (torch.zeros(*s, dtype=BF, device="cuda") for s in ((2, 3, 8), (2, 5, 8)))
    y = torch.zeros(2, 3, 5, device="cuda")
    with pytest.raises(ValueError, match="w has extents"):
        dps.dp_linear_forward(x, w[:, :, :7], y)
    with pytest.raises(ValueError, match="y has extents"):
        dps.dp_linear_forward(x, w, y[:, :2])
    with pytest.raises(ValueError, match="bias has extents"):
        dps.dp_linear_forward(x, w, y, bias=y[:, 0, :4])
    with pytest.raises(ValueError, match="unit stride"):
        dps.dp_linear_forward(x.mT.contiguous().mT, w, y)
    with pytest.raises(dps.DPError, match="x must be DP_BF16"):
        dps.dp_linear_forward(x.float(), w, y)
    with pytest.raises(ValueError, match="dw has extents"):
        dps.dp_linear_backward(y, x, w, dw=torch.zeros(2, 5, 9, device="cuda"))
    with pytest.raises(dps.DPError, match="out must be DP_BF16"):
        dps.dp_orthogonalize(x, x.float(), None)
    plan = dps.Plan([40], 1 << 10, 2)
    m = dps.Muon(plan, {0: (8, 5)})
    s = plan.new_state()
    with pytest.raises(ValueError, match="master holds"):
        dps.dp_muon_step(m, plan.new_workspace(), None, s, s[:3], s, plan.new_replicas())


def test_first_calls_of_a_process_inside_a_capture():
    """Nothing that a first call sets up disturbs a capture."""
    code = """
import torch, gradient_sync_zero_gb300 as dps
x = torch.randn(2, 300, 96, device='cuda').bfloat16()
w = torch.randn(2, 200, 96, device='cuda').bfloat16()
y = torch.empty(2, 300, 200, device='cuda')
dx, o = torch.empty_like(x), torch.empty(2, 300, 96, dtype=torch.bfloat16, device='cuda')
s = torch.empty_like(x[:, :40])
ws, ow = dps.new_linear_workspace(x, w, True), dps.new_orthogonalize_workspace(2, 300, 96)
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    dps.dp_linear_forward(x, w, y, ws=ws)
    dps.dp_linear_backward(y, x, w, dx=dx, ws=ws)
    dps.dp_orthogonalize(x, o, ow)
    dps.dp_orthogonalize(x[:, :40], s, ow)
g.replay()
torch.cuda.synchronize()
a = [t.clone() for t in (y, dx, o, s)]
dps.dp_linear_forward(x, w, y, ws=ws)
dps.dp_linear_backward(y, x, w, dx=dx, ws=ws)
dps.dp_orthogonalize(x, o, ow)
dps.dp_orthogonalize(x[:, :40], s, ow)
assert all(torch.equal(p, q) for p, q in zip(a, (y, dx, o, s)))
print('same')
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stdout[-2000:] + r.stderr[-2000:]
