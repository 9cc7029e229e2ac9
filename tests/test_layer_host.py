"""The dense layer, the orthogonalisation and the Muon step without a GPU: the 64-bit
reference against differences and singular values, and every refusal of the C ABI and of
the binding (made before any device work)."""
import ctypes as C

import pytest
import torch

import gradient_sync_zero_gb300 as dps
import layer_reference as ref
from gradient_sync_zero_gb300 import build as dbuild


@pytest.fixture(scope="module", autouse=True)
def built():
    dbuild.build()


# ---- the reference ----
@pytest.mark.parametrize("kind", ref.ACTS)
def test_reference_gradients_equal_differences(kind):
    """Central differences in 64 bits: truncation ~h^2 = 1e-12, cancellation ~1e-16 / h = 1e-10."""
    g = torch.Generator().manual_seed(1)
    P, T, K, N, h = 2, 4, 5, 3, 1e-6
    x, w, b = (torch.randn(P, *s, generator=g, dtype=torch.float64) for s in ((T, K), (N, K), (N,)))
    dy = torch.randn(P, T, N, generator=g, dtype=torch.float64)
    z = ref.linear(x, w, b)[1]
    assert z.abs().min() > 1e-3       # no kink of relu within a step
    grads, _ = ref.linear_grad(dy, z, x, w, kind)
    for at, got in zip((x, w, b), grads):
        for i in range(at.numel()):
            keep = at.view(-1)[i].item()
            vals = []
            for s in (h, -h):
                at.view(-1)[i] = keep + s
                vals.append((ref.linear(x, w, b, kind=kind)[0] * dy).sum())
            at.view(-1)[i] = keep
            num = (vals[0] - vals[1]) / (2 * h)
            assert abs(num - got.reshape(-1)[i]) < 1e-7, (kind, i)


@pytest.mark.parametrize("shape", [(4, 9), (9, 4), (6, 6), (1, 5)], ids=str)
def test_reference_orthogonalisation_acts_on_singular_values(shape):
    x = torch.randn(*shape, generator=torch.Generator().manual_seed(2), dtype=torch.float64)
    u, s, v = torch.linalg.svd(x, full_matrices=False)
    s = s / x.norm()
    a, b, c = ref.COEFS
    for _ in range(5):
        s = a * s + b * s ** 3 + c * s ** 5
    assert (ref.newton_schulz(x) - u @ torch.diag(s) @ v).abs().max() < 1e-12


# ---- refusals of the C ABI (fake device addresses: nothing may be launched) ----
def R(addr=1 << 30, rs=1 << 20, ws=64, dtype=dps.DP_BF16):
    return C.byref(dps.Rows(addr, rs, ws, dtype, 0))


WS = C.c_void_p(1 << 44)
BIG = 1 << 40
X, W, Y, Z, Q, B = (dict(addr=(i + 1) << 36) for i in range(6))


def _err():
    return dps.lib().dp_last_error().decode()


def _forward(x=None, w=None, bias=None, res=None, z=None, y=None, P=2, T=300, K=64, N=64, act=0, ws=WS, n=BIG):
    return dps.lib().dp_linear_forward(x or R(**X), w or R(**W), bias, res, z, y or R(**Y), P, T, K, N, act, ws,
                                       n, None)


@pytest.mark.parametrize("kw,code,word", [
    (dict(P=0), dps.DP_EINVAL, "P outside"),
    (dict(P=65), dps.DP_EINVAL, "P outside"),
    (dict(T=-1), dps.DP_EINVAL, "T is negative"),
    (dict(T=1 << 31), dps.DP_EINVAL, "2^31"),
    (dict(K=0), dps.DP_EINVAL, "in_dim outside"),
    (dict(K=1 << 31), dps.DP_EINVAL, "in_dim outside"),
    (dict(N=0), dps.DP_EINVAL, "out_dim outside"),
    (dict(T=1 << 29, K=1 << 30), dps.DP_EINVAL, "1e12"),
    (dict(P=1, T=(1 << 31) - 1000, K=1, N=1), dps.DP_EINVAL, "2^31 - 1024"),
    (dict(act=5), dps.DP_EINVAL, "unknown activation"),
    (dict(act=-1), dps.DP_EINVAL, "unknown activation"),
    (dict(x=R(dtype=dps.DP_F32, **X)), dps.DP_EINVAL, "x must be DP_BF16"),
    (dict(w=R(dtype=dps.DP_F32, **W)), dps.DP_EINVAL, "w must be DP_BF16"),
    (dict(y=R(dtype=9, **Y)), dps.DP_EINVAL, "unknown type"),
    (dict(x=R(addr=0)), dps.DP_EINVAL, "NULL data in x"),
    (dict(x=R(addr=(1 << 36) + 1)), dps.DP_EALIGN, "aligned"),
    (dict(x=R(ws=-64, **X)), dps.DP_EINVAL, "negative"),
    (dict(y=R(ws=63, **Y)), dps.DP_EINVAL, "overlap"),
    (dict(y=R(rs=0, **Y)), dps.DP_EINVAL, "overlap"),
    (dict(z=R(ws=63, **Z)), dps.DP_EINVAL, "overlap"),
    (dict(y=R(**X)), dps.DP_EINVAL, "y overlaps x"),
    (dict(y=R(**W)), dps.DP_EINVAL, "y overlaps w"),
    (dict(z=R(**X)), dps.DP_EINVAL, "z overlaps x"),
    (dict(z=R(**Y)), dps.DP_EINVAL, "z overlaps y"),
    (dict(bias=R(rs=64, **Y)), dps.DP_EINVAL, "y overlaps bias"),
    (dict(res=R(**Z), z=R(**Z)), dps.DP_EINVAL, "z overlaps residual"),
    (dict(res=R(addr=(3 << 36) + 64)), dps.DP_EINVAL, "without being it"),
    (dict(res=R(dtype=dps.DP_F32, **Y)), dps.DP_EINVAL, "without being it"),
    (dict(x=R(addr=(1 << 36) + 2), ws=None), dps.DP_EINVAL, "NULL workspace"),
    (dict(x=R(addr=(1 << 36) + 2), ws=C.c_void_p((1 << 44) + 16)), dps.DP_EALIGN, "32-byte"),
    (dict(x=R(addr=(1 << 36) + 2), n=100), dps.DP_EINVAL, "workspace holds 100"),
    (dict(x=R(addr=(1 << 36) + 2), ws=C.c_void_p(1 << 36)), dps.DP_EINVAL, "workspace overlaps x"),
    (dict(x=R(addr=(1 << 36) + 2), ws=C.c_void_p(3 << 36)), dps.DP_EINVAL, "workspace overlaps y"),
])
def test_forward_refusals(kw, code, word):
    assert _forward(**kw) == code
    assert word in _err() and "dp_linear_forward" in _err()


def test_forward_null_arguments_and_empty():
    f = dps.lib().dp_linear_forward
    assert f(None, R(**W), None, None, None, R(**Y), 1, 1, 8, 8, 0, WS, BIG, None) == dps.DP_EINVAL
    assert f(R(**X), None, None, None, None, R(**Y), 1, 1, 8, 8, 0, WS, BIG, None) == dps.DP_EINVAL
    assert f(R(**X), R(**W), None, None, None, None, 1, 1, 8, 8, 0, WS, BIG, None) == dps.DP_EINVAL
    assert f(R(addr=0), R(**W), None, None, None, R(addr=0), 1, 0, 8, 8, 0, None, 0, None) == dps.DP_OK


def _backward(dy=None, z=None, x=None, w=None, dx=R(**Y), dw=R(**Z), db=None, P=2, T=300, K=64, N=64, act=0, acc=0,
              ws=WS, n=BIG):
    return dps.lib().dp_linear_backward(dy or R(**Q), z, x or R(**X), w or R(**W), dx, dw, db, P, T, K, N, act, acc,
                                        ws, n, None)


@pytest.mark.parametrize("kw,code,word", [
    (dict(P=0), dps.DP_EINVAL, "P outside"),
    (dict(N=1 << 31), dps.DP_EINVAL, "out_dim outside"),
    (dict(act=7), dps.DP_EINVAL, "unknown activation"),
    (dict(act=dps.DP_ACT_GELU), dps.DP_EINVAL, "NULL z"),
    (dict(dx=None, dw=None), dps.DP_EINVAL, "all NULL"),
    (dict(x=R(dtype=dps.DP_F32, **X)), dps.DP_EINVAL, "x must be DP_BF16"),
    (dict(w=R(dtype=dps.DP_F32, **W)), dps.DP_EINVAL, "w must be DP_BF16"),
    (dict(dy=R(dtype=3, **Q)), dps.DP_EINVAL, "unknown type"),
    (dict(dx=R(rs=0, **Y)), dps.DP_EINVAL, "overlap"),
    (dict(dw=R(rs=0, **Z)), dps.DP_EINVAL, "overlap"),
    (dict(db=R(rs=63, **B)), dps.DP_EINVAL, "overlap"),
    (dict(dx=R(**Q)), dps.DP_EINVAL, "dx overlaps dy"),
    (dict(dw=R(**W)), dps.DP_EINVAL, "dw overlaps w"),
    (dict(dw=R(**Y)), dps.DP_EINVAL, "dw overlaps dx"),
    (dict(db=R(**Z)), dps.DP_EINVAL, "dbias overlaps dw"),
    (dict(db=R(**B), z=R(**B), act=1), dps.DP_EINVAL, "dbias overlaps z"),
    (dict(ws=None), dps.DP_EINVAL, "NULL workspace"),
    (dict(n=64), dps.DP_EINVAL, "workspace holds 64"),
    (dict(ws=C.c_void_p(4 << 36)), dps.DP_EINVAL, "workspace overlaps dw"),
])
def test_backward_refusals(kw, code, word):
    assert _backward(**kw) == code
    assert word in _err() and "dp_linear_backward" in _err()


def _bytes(x, w, P, T, K, N, back):
    out = C.c_int64(-1)
    assert dps.lib().dp_linear_workspace_bytes(x, w, P, T, K, N, back, C.byref(out)) == dps.DP_OK
    return out.value


def test_linear_workspace_holds_copies_and_parts():
    a = dict(rs=1 << 24, ws=2048)
    # enough tiles, rows on 16-byte boundaries: nothing
    assert _bytes(R(**X, **a), R(**W, **a), 8, 4096, 2048, 2048, 0) == 0
    # a copy of x, of w
    odd = dict(rs=1 << 24, ws=2049)
    assert _bytes(R(**X, **odd), R(**W, **a), 8, 4096, 2048, 2048, 0) == 2 * 8 * 4096 * 2048
    assert _bytes(R(**X, **a), R(**W, **odd), 8, 4096, 2048, 2048, 0) == 2 * 8 * 2048 * 2048
    # few tiles: parts of K, and in the backward dz and the column sums beside them
    assert _bytes(R(**X, **a), R(**W, **a), 1, 48, 2048, 2048, 0) >= 4 * 2 * 48 * 2048
    assert _bytes(R(**X, **a), R(**W, **a), 8, 4096, 2048, 2048, 1) >= 2 * 8 * 4096 * 2048
    out = C.c_int64()
    assert dps.lib().dp_linear_workspace_bytes(R(**X), R(**W), 1, 1, 8, 8, 0, None) == dps.DP_EINVAL
    assert dps.lib().dp_linear_workspace_bytes(R(**X), R(**W), 0, 1, 8, 8, 0, C.byref(out)) == dps.DP_EINVAL


def _orth(x=None, out=None, P=2, rows=300, cols=300, cfg=None, ws=WS, n=BIG):
    big = dict(rs=1 << 24, ws=300)
    return dps.lib().dp_orthogonalize(x or R(**X, **big), out or R(**Y, **big), P, rows, cols,
                                      C.byref(cfg or dps.newton_schulz_cfg()), ws, n, None)


@pytest.mark.parametrize("kw,code,word", [
    (dict(P=0), dps.DP_EINVAL, "P outside"),
    (dict(P=65), dps.DP_EINVAL, "P outside"),
    (dict(rows=0), dps.DP_EINVAL, "rows or cols"),
    (dict(cols=(1 << 20) + 1), dps.DP_EINVAL, "rows or cols"),
    (dict(out=R(dtype=dps.DP_F32, rs=1 << 24, ws=300, **Y)), dps.DP_EINVAL, "out must be DP_BF16"),
    (dict(out=R(rs=1 << 24, ws=299, **Y)), dps.DP_EINVAL, "overlap"),
    (dict(out=R(addr=(1 << 36) + 2, rs=1 << 24, ws=300)), dps.DP_EINVAL, "without being it"),
    (dict(cfg=dps.newton_schulz_cfg(steps=0)), dps.DP_EINVAL, "steps"),
    (dict(cfg=dps.newton_schulz_cfg(steps=65)), dps.DP_EINVAL, "steps"),
    (dict(cfg=dps.newton_schulz_cfg(eps=0.0)), dps.DP_EINVAL, "eps"),
    (dict(cfg=dps.newton_schulz_cfg(eps=float("nan"))), dps.DP_EINVAL, "eps"),
    (dict(cfg=dps.newton_schulz_cfg(a=float("inf"))), dps.DP_EINVAL, "not finite"),
    (dict(cfg=dps.newton_schulz_cfg(c=1e39)), dps.DP_EINVAL, "not finite"),
    (dict(ws=None), dps.DP_EINVAL, "NULL workspace"),
    (dict(ws=C.c_void_p((1 << 44) + 8)), dps.DP_EALIGN, "32-byte"),
    (dict(n=1000), dps.DP_EINVAL, "workspace holds 1000"),
    (dict(ws=C.c_void_p(1 << 36)), dps.DP_EINVAL, "workspace overlaps"),
])
def test_orthogonalize_refusals(kw, code, word):
    assert _orth(**kw) == code
    assert word in _err() and "dp_orthogonalize" in _err()
    assert dps.lib().dp_orthogonalize(R(), R(), 1, 4, 4, None, WS, BIG, None) == dps.DP_EINVAL


def test_orthogonalize_workspace():
    out = C.c_int64(-1)
    f = dps.lib().dp_orthogonalize_workspace_bytes
    assert f(2, 2048, 5632, C.byref(out)) == dps.DP_OK
    # the iterate and the next in fp16, what it leaves out in 8 bits, G and Q in fp16
    assert out.value >= 2 * (5 * 2048 * 5632 + 4 * 2048 * 2048)
    assert f(64, 48, 131, C.byref(out)) == dps.DP_OK and out.value == 0     # in shared memory
    assert f(0, 8, 8, C.byref(out)) == dps.DP_EINVAL and f(1, 8, 8, None) == dps.DP_EINVAL
    # large batches go through in parts: bounded
    assert f(64, 8192, 8192, C.byref(out)) == dps.DP_OK and out.value < 3 << 30


def test_muon_handle_refusals():
    plan = dps.Plan([12, 20, 64 * 64], 1 << 20, 2)
    with pytest.raises(dps.DPError, match="not in the plan"):
        dps.Muon(plan, {3: (3, 4)})
    with pytest.raises(dps.DPError, match="not in the plan"):
        dps.Muon(plan, {-1: (3, 4)})
    with pytest.raises(dps.DPError, match="holds 20 elements, not 3 x 4"):
        dps.Muon(plan, {1: (3, 4)})
    with pytest.raises(dps.DPError, match="rows or cols"):
        dps.Muon(plan, {0: (0, 4)})
    with pytest.raises(ValueError, match="rows, cols"):
        dps.Muon(plan, {0: (3, 2, 2)})
    h = C.c_void_p(5)
    ids, r = (C.c_int32 * 2)(0, 0), (C.c_int64 * 2)(3, 3)
    c = (C.c_int64 * 2)(4, 4)
    assert dps.lib().dp_muon_create(plan.handle, ids, r, c, 2, C.byref(h)) == dps.DP_EINVAL
    assert "listed twice" in _err() and not h.value
    assert dps.lib().dp_muon_create(None, ids, r, c, 1, C.byref(h)) == dps.DP_EINVAL
    assert dps.lib().dp_muon_create(plan.handle, ids, None, c, 1, C.byref(h)) == dps.DP_EINVAL
    assert dps.lib().dp_muon_create(plan.handle, ids, r, c, -1, C.byref(h)) == dps.DP_EINVAL
    assert dps.lib().dp_muon_create(plan.handle, ids, r, c, 1, None) == dps.DP_EINVAL
    assert dps.Muon(plan, {0: (3, 4), 2: (64, 64)}).workspace_bytes == 0
    assert dps.Muon(plan, {}).workspace_bytes == 0


def test_muon_handle_outlives_its_plan():
    plan = dps.Plan([600 * 700], 1 << 20, 2)
    m = dps.Muon(plan, {0: (600, 700)})
    m.plan = None
    del plan
    assert m.workspace_bytes > 5 * 600 * 700


@pytest.mark.parametrize("kw,code,word", [
    (dict(pw=None), dps.DP_EINVAL, "NULL plan_workspace"),
    (dict(mean=None), dps.DP_EINVAL, "NULL device pointer"),
    (dict(master=(2 << 36) + 4), dps.DP_EALIGN, "32-byte"),
    (dict(momentum=2 << 36), dps.DP_EINVAL, "momentum overlaps master"),
    (dict(params=(1 << 36) + 64), dps.DP_EINVAL, "params overlaps mean"),
    (dict(ws=4 << 36), dps.DP_EINVAL, "workspace overlaps params"),
    (dict(ws=None), dps.DP_EINVAL, "NULL workspace"),
    (dict(n=10), dps.DP_EINVAL, "workspace holds 10"),
    (dict(coef=64, use=0), dps.DP_EINVAL, "use_clip_coef = 0"),
    (dict(coef=66, use=1), dps.DP_EALIGN, "coef_dev"),
    (dict(lr=float("nan")), dps.DP_EINVAL, "lr"),
    (dict(lr=-1.0), dps.DP_EINVAL, "lr"),
    (dict(momentum_factor=1.0), dps.DP_EINVAL, "momentum"),
    (dict(momentum_factor=-0.1), dps.DP_EINVAL, "momentum"),
    (dict(decay=float("inf")), dps.DP_EINVAL, "weight_decay"),
    (dict(scale=2), dps.DP_EINVAL, "unknown scale"),
    (dict(ns=dps.newton_schulz_cfg(steps=0)), dps.DP_EINVAL, "steps"),
    (dict(lr_dev=3), dps.DP_EALIGN, "lr_dev"),
])
def test_muon_step_refusals(kw, code, word):
    plan = dps.Plan([600 * 700], 1 << 20, 2)
    m = dps.Muon(plan, {0: (600, 700)})
    a = dict(pw=7 << 36, mean=1 << 36, master=2 << 36, momentum=3 << 36, params=4 << 36, ws=5 << 36, n=BIG, coef=None,
             use=0, lr=1e-3, momentum_factor=0.9, decay=0.1, scale=1, ns=None, lr_dev=None)
    a.update(kw)
    cfg = dps.muon_cfg(lr=a["lr"], momentum=a["momentum_factor"], weight_decay=a["decay"], scale=a["scale"],
                       newton_schulz=a["ns"])
    cfg.lr_dev = a["lr_dev"]
    f = dps.lib().dp_muon_step
    assert f(m.handle, a["pw"], a["mean"], a["master"], a["momentum"], a["params"], a["use"], a["coef"], C.byref(cfg),
             a["ws"], a["n"], None) == code
    assert word in _err() and "dp_muon_step" in _err()
    assert f(None, 1 << 36, 1, 1, 1, 1, 0, None, C.byref(cfg), 1, 1, None) == dps.DP_EINVAL
    assert f(m.handle, 1 << 36, 1 << 37, 1 << 38, 1 << 39, 1 << 40, 0, None, None, 1 << 41, BIG, None) == dps.DP_EINVAL


def test_binding_refuses_what_it_sees():
    x = torch.zeros(2, 3, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="x must be a CUDA tensor"):
        dps.dp_linear_forward(x, x, x)
    with pytest.raises(TypeError, match="x must be a torch.Tensor"):
        dps.dp_orthogonalize([1], x, None)
    with pytest.raises(TypeError, match="lr_dev"):
        dps.muon_cfg(lr_dev=3)
    with pytest.raises(TypeError, match="dbias must be"):
        dps._bias(3, 2, 8, "dbias")
    with pytest.raises(ValueError, match="needs \\(2, 8\\)"):
        dps._bias(torch.zeros(3, 8), 2, 8, "bias")


def test_muon_step_refuses_a_workspace_that_is_the_plans():
    """Its kernels would write over the image that they check."""
    plan = dps.Plan([600 * 700], 1 << 20, 2)
    m, cfg, n = dps.Muon(plan, {0: (600, 700)}), dps.muon_cfg(), plan.info.workspace_bytes
    a = dict(pw=1 << 36, mean=2 << 36, master=3 << 36, momentum=4 << 36, params=5 << 36, ws=6 << 36)

    def call(**kw):
        b = {**a, **kw}
        return dps.lib().dp_muon_step(m.handle, b["pw"], b["mean"], b["master"], b["momentum"], b["params"], 0, None,
                                      C.byref(cfg), b["ws"], BIG, None)
    for name, word in (("ws", "workspace"), ("master", "master"), ("momentum", "momentum"), ("params", "params")):
        for at in (0, 256, n - 32):
            assert call(**{name: (1 << 36) + at}) == dps.DP_EINVAL
            assert f"plan_workspace overlaps {word}" in _err()


def test_long_sums_are_formed_in_parts():
    """What a tile's accumulators cut off grows with the products they add: fp32 results take 16384 in one go at
    most, however many tiles there are (the workspace has room for the parts)."""
    a = dict(rs=1 << 40, ws=4096)
    least = _bytes(R(**X, **a), R(**W, **a), 1, 16384, 4096, 4096, 1)
    long = _bytes(R(**X, **a), R(**W, **a), 1, 65536, 4096, 4096, 1)
    assert least < 4 * 4096 * 4096 + 2 * 16384 * 4096 + 4 * 512 * 4096 + 1024      # dz, the column sums: no parts
    assert long >= 4 * 4 * 4096 * 4096 + 2 * 65536 * 4096
    b = dict(rs=1 << 40, ws=65536)
    assert _bytes(R(**X, **b), R(**W, **b), 1, 4096, 65536, 4096, 0) >= 4 * 4 * 4096 * 4096


def test_two_tokens_need_no_copies():
    """Ordinary loads read rows that are shown twice, which the tensor cores' copies cannot."""
    a = dict(rs=1 << 24, ws=2048)
    once = dict(rs=1 << 24, ws=0)
    assert _bytes(R(**X, **once), R(**W, **a), 8, 2, 2048, 2048, 0) == 0
    assert _bytes(R(**X, **a), R(**W, **once), 8, 1, 2048, 2048, 0) == 0
    assert _bytes(R(**X, **once), R(**W, **a), 8, 3, 2048, 2048, 0) >= 2 * 8 * 3 * 2048
    assert _bytes(R(**X, **once), R(**W, **a), 8, 2, 2044, 2048, 0) >= 2 * 8 * 2 * 2048      # rows of no whole vectors
