"""Paths of the dense layer, the orthogonalisation and the Muon step that the shapes of
test_layer_gpu.py do not take, and what each leaves alone."""
import pytest
import torch

import gradient_sync_zero_gb300 as dps
import layer_reference as ref
from layer_reference import U, stored
from test_layer_gpu import BF, F32, close, gen, no_timeouts   # noqa: F401

pytestmark = pytest.mark.gpu

# in shared memory, thin both ways, on the tensor cores with whole vectors and without
KINDS = [(61, 64), (131, 48), (40, 5000), (5000, 41), (320, 264), (264, 328), (300, 260)]


def device_gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def muon_case(shapes, P=3, seed=30, gap=77):
    """A plan with a tensor that is no matrix between any two, and its state."""
    sizes = [s for r, c in shapes for s in (r * c, gap)]
    plan = dps.Plan(sizes, 1 << 17, P)
    g = gen(seed)
    mean, master, buf = (torch.randn(plan.L, generator=g) * s for s in (1e-3, 0.02, 1e-3))
    params = torch.randn(P, plan.stride, generator=g).to(BF)
    return plan, {2 * i: s for i, s in enumerate(shapes)}, (mean, master, buf, params)


def test_muon_writes_nothing_after_a_timeout():
    """The bit that a product's wait leaves when it gives up: sums that were not waited for must not
    reach the weights, in no kernel of the step."""
    plan, matrices, state = muon_case(KINDS)
    ws, m = plan.new_workspace(), dps.Muon(plan, matrices)
    at = dps.workspace_result_offsets()[3]
    status = ws[at:at + 4].view(torch.int32)
    status.fill_(dps.DP_STATUS_TIMEOUT)
    dev = [t.cuda() for t in state]
    dps.dp_muon_step(m, ws, m.new_workspace(), *dev)
    for a, b in zip(dev, state):
        assert torch.equal(a.cpu().view(torch.int16), b.view(torch.int16))
    with pytest.raises(dps.DPError) as e:
        dps.dp_read_norm(plan, ws)
    assert e.value.code == dps.DP_ETIMEOUT and int(status) == dps.DP_STATUS_TIMEOUT
    status.zero_()
    dps.dp_muon_step(m, ws, m.new_workspace(), *dev)
    assert int(status) == 0
    for t, (r, c) in matrices.items():
        o = plan.tensor(t)[1]
        assert (dev[1][o:o + r * c].cpu() != state[1][o:o + r * c]).float().mean() > 0.9


def check_muon(plan, matrices, state, dev, lr, mu, decay, nesterov, scale, coef=1.0):
    """Every matrix against the formula, replicas against the master, and the rest untouched."""
    mean, master, buf, params = state
    got_mean, got_master, got_buf, got_params = (t.cpu() for t in dev)
    assert torch.equal(got_mean, mean)
    left = torch.ones(plan.L, dtype=torch.bool)
    for t, (r, c) in matrices.items():
        o = plan.tensor(t)[1]
        at = slice(o, o + r * c)
        left[at] = False
        s = 0.2 * max(r, c) ** 0.5 if scale else max(1.0, r / c) ** 0.5
        w, b, orth = ref.muon(*(v[at].double().cuda().view(r, c) for v in (mean, buf, master)), lr, mu, decay, nesterov, s,
                              coef=coef)
        w, b, orth = w.cpu(), b.cpu(), orth.cpu()
        # three roundings of terms of its two parts' size
        assert ((got_buf[at].view(r, c) - b).abs() <= 4 * U * (buf[at].abs() + mean[at].abs()).view(r, c)).all(), t
        # the documented 2e-3 of the update, and the master's two roundings
        d = (got_master[at].double().view(r, c) - w).norm()
        assert d <= lr * s * 2e-3 * orth.norm() + 4 * U * master[at].norm(), (t, r, c, d / (lr * s * orth.norm()))
        for p in range(plan.P):
            assert torch.equal(got_params[p, at], got_master[at].to(BF)), t
    assert torch.equal(got_master[left], master[left]) and torch.equal(got_buf[left], buf[left])
    rest = torch.cat([left, torch.ones(plan.stride - plan.L, dtype=torch.bool)])
    assert torch.equal(got_params[:, rest].view(torch.int16), params[:, rest].view(torch.int16))


def run_muon(shapes, nesterov=True, scale=dps.DP_MUON_MATCH_RMS, clip=False, P=3, gap=77):
    plan, matrices, state = muon_case(shapes, P, gap=gap)
    ws, m = plan.new_workspace(), dps.Muon(plan, matrices)
    dev = [t.cuda() for t in state]
    lr, coef, kw = 1e-2, 1.0, {}
    if clip:
        coef = 0.37109375                       # exact in fp32
        kw = dict(use_clip_coef=True, coef_dev=torch.tensor([coef], device="cuda"))
    cfg = dps.muon_cfg(lr=lr, momentum=0.9, weight_decay=0.1, nesterov=nesterov, scale=scale)
    mws = m.new_workspace()
    mws.fill_(255)
    dps.dp_muon_step(m, ws, mws, *dev, cfg, **kw)
    assert dps.dp_read_norm(plan, ws, raise_on_status=False)[2] == 0
    check_muon(plan, matrices, state, dev, lr, 0.9, 0.1, nesterov, scale, coef)


@pytest.mark.parametrize("nesterov,scale,clip", [(True, dps.DP_MUON_MATCH_RMS, False), (False, dps.DP_MUON_SPECTRAL, True),
                                                 (True, dps.DP_MUON_SPECTRAL, True), (False, dps.DP_MUON_MATCH_RMS, False)])
def test_muon_of_every_kind_of_matrix(nesterov, scale, clip):
    """Small, thin and large ones, stored in whole vectors and not, in one step."""
    run_muon(KINDS, nesterov, scale, clip)


@pytest.mark.parametrize("shapes", [
    [(320, 264)], [(264, 328), (264, 328)], [(257, 300)], [(300, 257)],      # one large shape: no other beside it
    [(2048, 256)], [(100, 5000)],                                            # whose G is summed in parts
    [(130, 70000), (320, 264)], [(70000, 130), (40, 5000), (264, 328)],      # in parts whatever the tiles, not together
    [(40, 5000)], [(5000, 41)], [(40, 5000), (40, 5000)],                    # thin alone and in a batch
    [(300, 260), (40, 5000), (264, 328), (5000, 41), (320, 264)],            # rounds parted by thin ones
], ids=str)
def test_muon_rounds(shapes):
    run_muon(shapes)


def test_muon_of_more_shapes_than_go_together():
    """Eleven large shapes: rounds of eight and three."""
    run_muon([(130 + 8 * i, 150 + 3 * i) for i in range(11)], clip=True)


def test_muon_of_more_small_matrices_than_a_launch_holds():
    """150 of them, of five shapes, in eight parts each since one is long."""
    run_muon([[(5, 7), (16, 24), (33, 31), (8, 8), (24, 320)][i % 5] for i in range(150)], nesterov=False)


def test_muon_of_sixty_four_ranks_and_of_one():
    for P in (1, 64):
        run_muon([(320, 264), (61, 64), (300, 260)], P=P)


def test_muon_state_goes_through_a_checkpoint(tmp_path):
    """master and momentum saved as AdamW's master and m after two steps; the third in fresh buffers has the bits
    of three steps in a row."""
    plan, matrices, (mean, master, buf, params) = muon_case([(61, 64), (320, 264), (40, 5000)])
    m, cfg = dps.Muon(plan, matrices), dps.muon_cfg(lr=1e-2)
    means = [mean.cuda().roll(k) for k in range(3)]

    def steps(which, ws, state, replicas):
        for k in which:
            dps.dp_muon_step(m, ws, m.new_workspace(), means[k], *state, replicas, cfg)
    through, p = [master.cuda(), buf.cuda()], params.cuda()
    steps((0, 1), plan.new_workspace(), through, p)
    path, v = str(tmp_path / "muon.ckpt"), plan.new_state()
    dps.dp_checkpoint_save(plan, path, *through, v, step=2)
    steps((2,), plan.new_workspace(), through, p)
    fresh = [torch.full((plan.L,), float("nan"), device="cuda") for _ in range(3)]
    assert dps.dp_checkpoint_load(plan, path, *fresh) == 2
    q = plan.new_replicas()
    steps((2,), plan.new_workspace(), fresh[:2], q)
    for t, (r, c) in matrices.items():
        o = plan.tensor(t)[1]
        at = slice(o, o + r * c)
        for a, b in zip(fresh[:2], through):
            assert torch.equal(a[at].view(torch.int32), b[at].view(torch.int32)), t
        assert torch.equal(q[:, at], p[:, at]), t


def orthogonal_fp32(x):
    """O of a CUDA matrix in fp32: master starts at 0 and ends as -lr s O (s = 0.2 sqrt(longer side))."""
    r, c = x.shape
    plan = dps.Plan([r * c], 1 << 20, 1)
    mean, master, buf = (plan.new_state() for _ in range(3))
    mean[:r * c] = x.flatten()
    m, ws = dps.Muon(plan, {0: (r, c)}), plan.new_workspace()
    cfg = dps.muon_cfg(lr=1.0, momentum=0.0, weight_decay=0.0, nesterov=False)
    dps.dp_muon_step(m, ws, m.new_workspace(), mean, master, buf, plan.new_replicas(), cfg)
    return -master[:r * c].view(r, c).double() / (0.2 * max(r, c) ** 0.5)


@pytest.mark.parametrize("shape", [(64, 320), (2, 900), (40, 1 << 16), (1 << 18, 64)], ids=str)
def test_muon_of_the_largest_values(shape):
    """Matrices of values around 3e38, whose norm's reciprocal fp32 holds in a few bits: small and thin matrices are
    within 1e-5."""
    r, c = shape
    g = device_gen(34)
    x = (torch.rand(r, c, generator=g, device="cuda") * 0.2 + 0.79) * 3.4e38
    x *= torch.randint(0, 2, (r, c), generator=g, device="cuda") * 2.0 - 1
    got, want = orthogonal_fp32(x), ref.newton_schulz(x.double())
    assert (got - want).norm() <= 1e-5 * want.norm(), (got - want).norm() / want.norm()


# ---------------------------------------------------------------- orthogonalisation
def kind_of(shape, kind, seed=37):
    g = device_gen(seed)
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.float64)
    if kind == "falling":                      # singular values about as 1, 1/2, 1/3 ..
        d = 1.0 / torch.arange(1, min(shape) + 1, device="cuda", dtype=torch.float64)
        x = x * (d[:, None] if shape[0] < shape[1] else d)
    if kind == "rank 1":
        x = torch.outer(x[:, 0], x[0])
    if kind == "few entries":                  # five entries hold nearly all of it
        big = torch.zeros_like(x).flatten()
        big[torch.randperm(x.numel(), generator=g, device="cuda")[:5]] = 1
        x = x * (big.view(shape) + 1e-4)
    return x.float()


IN_FP32 = [(1, 1), (1, 7), (9, 1), (3, 5), (16, 16), (48, 131), (131, 48), (64, 64), (61, 64), (2, 900), (64, 320), (100, 90),
           (100, 400), (2, 20000), (20000, 3), (64, 3001), (5000, 40)]


def fp32_bound(shape):
    """Five steps in fp32, norm against norm.  An entry of X is rounded once when it is scaled, and in each step, beside its
    terms (up to a + |b| + |c| = 10.3 times its magnitude), by sums of m terms whose roundings are as often up as down: by U and
    by 10.3 / 3.44 = 3 times sqrt(m) U before the growth by a = 3.4445 a step of what lies where the singular values are
    small: a^5 = 485 (the later steps' shares are a third each: in quadrature 1.05)."""
    return 1.05 * 485 * U * (1 + 3 * min(shape) ** 0.5)


@pytest.mark.parametrize("kind", ["noise", "falling", "rank 1", "few entries"])
@pytest.mark.parametrize("shape", IN_FP32, ids=str)
def test_small_and_thin_matrices(shape, kind):
    """What the Muon step's fp32 weights receive within fp32_bound, and the bf16 result within it and its rounding (2^-8 of
    every entry at most): a result of zeros, or one that is 1% off, fails at every shape."""
    x = kind_of(shape, kind)
    want, bound = ref.newton_schulz(x.double()), fp32_bound(shape)
    assert bound + 2.0 ** -8 < 0.01
    assert (orthogonal_fp32(x) - want).norm() <= bound * want.norm()
    out = torch.full((1, *shape), float("nan"), dtype=BF, device="cuda")
    for dt in (F32, BF):
        y = x.to(dt)
        want = ref.newton_schulz(y.double())
        dps.dp_orthogonalize(y[None], out, dps.new_orthogonalize_workspace(1, *shape))
        assert (out[0].double() - want).norm() <= (bound + 2.0 ** -8) * want.norm(), dt


@pytest.mark.parametrize("kind", ["rank 1", "falling", "few entries"])
@pytest.mark.parametrize("shape", [(128, 128), (130, 130), (257, 300), (300, 257), (600, 520), (264, 328), (300, 9001)], ids=str)
def test_large_matrices_of_uneven_spectra(shape, kind):
    """In fp32 before any rounding to bf16, as documented: 2e-3, and 6e-3 where a few entries hold the matrix.  Without the
    iterate's 8 low bits a matrix of rank 1 comes out 0.15 off, with an 8-bit float in their place 7e-3."""
    x = kind_of(shape, kind)
    got, want = orthogonal_fp32(x), ref.newton_schulz(x.double())
    off = (got - want).norm() / want.norm()
    assert off <= (6e-3 if kind == "few entries" else 2e-3), off


# K of G in parts, joined from memory with the mirrored half: wide and tall, more than one tile a side, a
# batch; and so long (above 65536) that it is cut whatever the tiles
@pytest.mark.parametrize("kind", ["noise", "falling"])
@pytest.mark.parametrize("shape", [(100, 5000), (5000, 100), (2048, 256), (256, 2051), (300, 9001), (9001, 300), (264, 5000),
                                   (530, 12000), (130, 70001), (70001, 130)], ids=str)
def test_orthogonalize_with_sums_in_parts(shape, kind):
    """Norm against norm, 2e-3 as documented and the rounding to bf16, 1.7e-3: together 2.7e-3."""
    r, c = shape
    x = torch.randn(2, r, c, generator=device_gen(36), device="cuda")
    if kind == "falling":                      # singular values about as 1, 1/2, 1/3 ..
        d = 1.0 / torch.arange(1, min(shape) + 1, device="cuda")
        x = x * (d[:, None] if r < c else d)
    out = torch.full((2, r, c), float("nan"), dtype=BF, device="cuda")
    dps.dp_orthogonalize(x, out, dps.new_orthogonalize_workspace(2, r, c))
    want = ref.newton_schulz(x.double())
    off = (out.double() - want).flatten(1).norm(dim=1) / want.flatten(1).norm(dim=1)
    assert (off <= 2.7e-3).all(), off
    # rows of one block: its share of those errors (twice 2e-3 is ample), where a wrong block is off by itself
    for b in range(0, min(r, 512), 128):
        e, w = (out[:, b:b + 128].double() - want[:, b:b + 128]), want[:, b:b + 128]
        assert (e.flatten(1).norm(dim=1) <= 4e-3 * w.flatten(1).norm(dim=1)).all(), b


# ---------------------------------------------------------------- long sums
def positive(g, *shape):
    """Between 0.5 and 1.5: running sums grow as their results, so that what is cut off adds up."""
    return (torch.rand(*shape, generator=g, device="cuda") + 0.5).to(BF)


def test_what_the_tensor_cores_cut_off():
    """The premise of the bounds below.  Beside 1, products below 2^-25 leave nothing, those above are whole, and the
    result is cut off at its own last place, 2^-23: with the sum so far as the 1 and with a product."""
    for first, n in ((16, 16), (1, 15)):         # the 1 in a step of its own, or with 15 others
        for j in range(22, 28):
            x, w = torch.zeros(1, 200, first + n), torch.zeros(1, 64, first + n)
            x[..., 0] = w[..., 0] = 1
            x[..., first:], w[..., first:] = 2.0 ** -(j // 2), 2.0 ** -(j - j // 2)
            x, w = x.to(BF).cuda(), w.to(BF).cuda()
            y = torch.empty(1, 200, 64, device="cuda")
            dps.dp_linear_forward(x, w, y, ws=dps.new_linear_workspace(x, w))
            places = n * 2.0 ** (23 - j) // 1 if j <= 25 else 0
            assert (y == 1 + places * 2.0 ** -23).all(), (first, j)


# So a step of 16 products loses, in places of the sum's last bit, at most 16 / 4 + 3 / 4 and on average half of
# that, D = 2.375.  A sum that grows steadily to r takes its steps at a last place of 2^-23 of the binade it is in:
# over all binades the integral of that to r is at most 0.375 * 2^-23 r^2.  K / 16 steps: on average
# K / 16 * D * 0.375 * 2^-23 = 6.63e-9 K of the result, and never more than twice that.
# (First run: a bound of 1.34e-9 K, from one cut for a step instead of one for each of its 16 products.)
CUT = 6.63e-9


@pytest.mark.parametrize("T,K,N", [
    (2304, 8192, 1200),      # two accumulators of 4096, not cut
    (2304, 16384, 1200),     # four
    (2304, 65536, 1200),     # parts of K that four accumulators hold
    (300, 40000, 72),        # few tiles
    (9, 100000, 300),        # tokens as columns
])
def test_fp32_results_of_long_sums(T, K, N):
    """Accumulators of 4096 products: CUT * 4096 = 2.7e-5 low at most (one accumulator for 16384 products
    measured 6.5e-5)."""
    g = device_gen(31)
    x, w = positive(g, 1, T, K), positive(g, 1, N, K)
    y = torch.empty(1, T, N, device="cuda")
    dps.dp_linear_forward(x, w, y, ws=dps.new_linear_workspace(x, w))
    off = y.double() / (x.double() @ w.double().mT) - 1
    assert off.mean().abs() <= 4096 * CUT and off.abs().max() <= 2 * 4096 * CUT, (off.mean(), off.abs().max())


@pytest.mark.parametrize("T", [16384, 262144])
def test_fp32_gradients_of_many_tokens(T):
    g = device_gen(32)
    N, K = 1200, 2304
    x, dy, w = positive(g, 1, T, K), positive(g, 1, T, N), positive(g, 1, N, K)
    dw = torch.full((1, N, K), 3.0, device="cuda")
    ws = dps.new_linear_workspace(x, w, True)
    dps.dp_linear_backward(dy, x, w, dw=dw, accumulate=True, ws=ws)
    rows = slice(0, N, 40)
    want = sum(a.double().T @ b.double() for a, b in zip(dy[0, :, rows].split(1 << 15), x[0].split(1 << 15)))
    off = (dw[0, rows].double() - 3) / want - 1
    assert off.mean().abs() <= 4096 * CUT and off.abs().max() <= 2 * 4096 * CUT, (off.mean(), off.abs().max())


def test_bf16_results_of_very_long_sums():
    """2^20 products to a result: the mean over the entries, whose roundings to bf16 are as often up as down (2^-9 /
    sqrt(30 * 2304) = 8e-6), shows what was cut off: CUT * 65536 = 4.3e-4 at most in parts of that length."""
    g = device_gen(33)
    T, N, K = 1 << 20, 1200, 2304
    x, dy, w = positive(g, 1, T, K), positive(g, 1, T, N), positive(g, 1, N, K)
    dw = torch.empty(1, N, K, device="cuda", dtype=BF)
    dps.dp_linear_backward(dy, x, w, dw=dw, ws=dps.new_linear_workspace(x, w, True))
    rows = slice(0, N, 40)
    want = sum(a.double().T @ b.double() for a, b in zip(dy[0, :, rows].split(1 << 15), x[0].split(1 << 15)))
    off = dw[0, rows].double() / want - 1
    assert off.mean().abs() <= 65536 * CUT + 3e-5, off.mean()


@pytest.mark.parametrize("T", [1, 2])
def test_one_row_shown_to_two_tokens_and_every_weight_row(T):
    g = gen(35)
    x, w = torch.randn(3, 1, 264, generator=g).to(BF), torch.randn(3, 40, 264, generator=g).to(BF)
    xs, ws_, y = x.cuda().expand(3, T, 264), w.cuda(), torch.empty(3, T, 40, device="cuda")
    dps.dp_linear_forward(xs, ws_, y)                        # no workspace
    want, _, err, _ = ref.linear(x.double().expand(3, T, 264), w.double())
    close(y, want, stored(want, err, F32))
    same = ws_[:, :1].expand(3, 40, 264)
    dps.dp_linear_forward(xs, same, y)
    want, _, err, _ = ref.linear(x.double().expand(3, T, 264), w[:, :1].double().expand(3, 40, 264))
    close(y, want, stored(want, err, F32))


@pytest.mark.parametrize("T", [2, 40, 300])
def test_a_vocabulary_head(T):
    """Rows of 50257 columns lie off 16-byte boundaries: fp32 logits, and the gradients of a sum that long."""
    g, N, K = device_gen(38), 50257, 72
    x, w = torch.randn(2, T, K, generator=g, device="cuda").to(BF), torch.randn(2, N, K, generator=g, device="cuda").to(BF)
    y = torch.full((2, T, N), float("nan"), device="cuda")
    dps.dp_linear_forward(x, w, y, ws=dps.new_linear_workspace(x, w))
    want, _, err, _ = ref.linear(x.double(), w.double())
    assert ((y.double() - want).abs() <= stored(want, err, F32)).all()
    dx, dw = torch.empty(2, T, K, device="cuda"), torch.zeros(2, N, K, device="cuda", dtype=BF)
    dps.dp_linear_backward(y, x, w, dx=dx, dw=dw, ws=dps.new_linear_workspace(x, w, True))
    wants, errs = ref.linear_grad(y.double(), None, x.double(), w.double(), rounds=True)
    for got, want, err, t in ((dx, wants[0], errs[0], F32), (dw, wants[1], errs[1], BF)):
        assert ((got.double() - want).abs() <= stored(want, err, t)).all()
