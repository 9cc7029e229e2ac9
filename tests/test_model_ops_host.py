"""The operators at the ends of a training step, without a GPU: the generator
against its published vectors, the 64-bit reference against differences, and every
refusal of the C ABI and of the binding (made before any device work)."""
import ctypes as C

import numpy as np
import pytest
import torch

import gradient_sync_zero_gb300 as dps
import model_reference as ref
from gradient_sync_zero_gb300 import build as dbuild


@pytest.fixture(scope="module", autouse=True)
def built():
    dbuild.build()


@pytest.mark.parametrize("counter,key,want", [
    ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
    ((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
    ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
     (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1))])
def test_generator_gives_the_published_vectors(counter, key, want):
    got = ref.philox4x32([np.array([c]) for c in counter], key)
    assert tuple(int(x[0]) for x in got) == want


def _small_policy(seed=0, P=2, T=5, V=7):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)   # noqa: E731
    logits, tokens = r(P, T, V), torch.randint(0, V, (P, T), generator=g)
    tokens[0, 1] = -100
    old = ref.logprob(logits, tokens, 1.3)[0] - 0.4 * r(P, T)
    w = torch.rand(P, T, generator=g, dtype=torch.float64)
    w[1, 2] = 0.0
    return logits, tokens, old, old + 0.3 * r(P, T), r(P, T), w


def test_reference_gradients_equal_differences():
    """The reference's formulas for dlogits, against central differences of its loss
    in 64 bits (step 1e-6: truncation ~1e-12, cancellation ~1e-10)."""
    logits, tokens, old, rf, adv, w = _small_policy()
    kw = dict(lo=0.2, hi=0.3, beta=0.1, alpha=1.3)
    _, _, _, g, _ = ref.policy(logits, tokens, old, rf, adv, w, **kw)
    h = 1e-6
    for idx in np.ndindex(*logits.shape):
        lossp, lossm = [], []
        for s, to in ((h, lossp), (-h, lossm)):
            z = logits.clone()
            z[idx] += s
            to.append(ref.policy(z, tokens, old, rf, adv, w, **kw)[0][:, 0].sum())
        num = (lossp[0] - lossm[0]) / (2 * h)
        assert abs(num - g[idx]) < 1e-8, idx


def test_reference_lookup_gradient_is_the_adjoint():
    g = torch.Generator().manual_seed(3)
    P, T, V, D = 2, 9, 5, 6
    table = torch.randn(P, V, D, generator=g, dtype=torch.float64)
    dout = torch.randn(P, T, D, generator=g, dtype=torch.float64)
    tokens = torch.randint(-1, V + 1, (P, T), generator=g)
    drop = (0.3, 77, 5)
    a = (ref.lookup(table, tokens, 1.7, drop) * dout).sum()
    b = (ref.lookup_grad(dout, tokens, V, 1.7, drop)[0] * table).sum()
    assert abs(a - b) < 1e-12 * abs(a) + 1e-12


# ---- refusals of the C ABI (fake device addresses: nothing may be launched) ----
def R(addr=1 << 30, rs=1 << 20, ws=64, dtype=dps.DP_BF16):
    return C.byref(dps.Rows(addr, rs, ws, dtype, 0))


TOK, VEC, WS = C.c_void_p(1 << 34), C.c_void_p(1 << 35), C.c_void_p(1 << 36)
FAR = dict(addr=1 << 40)


def _err():
    return dps.lib().dp_last_error().decode()


def _dropout(x=None, res=None, out=None, P=2, T=3, D=64, cfg=None):
    return dps.lib().dp_dropout(x or R(), res, out or R(**FAR), P, T, D,
                                C.byref(cfg or dps.dropout_cfg(0.1)), None)


@pytest.mark.parametrize("kw,code,word", [
    (dict(P=0), dps.DP_EINVAL, "P outside"),
    (dict(P=65), dps.DP_EINVAL, "P outside"),
    (dict(T=-1), dps.DP_EINVAL, "T is negative"),
    (dict(T=1 << 31), dps.DP_EINVAL, "2^31"),
    (dict(D=0), dps.DP_EINVAL, "dim outside"),
    (dict(D=1 << 31), dps.DP_EINVAL, "dim outside"),
    (dict(x=R(dtype=7)), dps.DP_EINVAL, "unknown type"),
    (dict(x=R(addr=0)), dps.DP_EINVAL, "NULL data in x"),
    (dict(x=R(addr=(1 << 30) + 1)), dps.DP_EALIGN, "aligned"),
    (dict(x=R(addr=(1 << 30) + 2, dtype=dps.DP_F32)), dps.DP_EALIGN, "aligned"),
    (dict(x=R(ws=-64)), dps.DP_EINVAL, "negative"),
    (dict(x=R(rs=1 << 62)), dps.DP_EINVAL, "address space"),
    (dict(out=R(ws=63, **FAR)), dps.DP_EINVAL, "overlap"),
    (dict(out=R(rs=0, **FAR)), dps.DP_EINVAL, "overlap"),
    (dict(out=R(rs=191, **FAR)), dps.DP_EINVAL, "overlap"),
    (dict(out=R(addr=(1 << 30) + 64)), dps.DP_EINVAL, "without being it"),
    (dict(out=R(dtype=dps.DP_F32)), dps.DP_EINVAL, "without being it"),
    (dict(cfg=dps.dropout_cfg(-0.1)), dps.DP_EINVAL, "dropout p"),
    (dict(cfg=dps.dropout_cfg(1.1)), dps.DP_EINVAL, "dropout p"),
    (dict(cfg=dps.dropout_cfg(float("nan"))), dps.DP_EINVAL, "dropout p"),
    (dict(cfg=dps.DropoutCfg(0.1, 0, 0, 0, 4)), dps.DP_EALIGN, "seed_dev"),
])
def test_dropout_refusals(kw, code, word):
    assert _dropout(**kw) == code
    assert word in _err() and "dp_dropout" in _err()


def test_dropout_null_arguments_and_empty():
    lib = dps.lib()
    assert lib.dp_dropout(None, None, R(), 1, 1, 4, None, None) == dps.DP_EINVAL
    assert lib.dp_dropout(R(), None, None, 1, 1, 4, None, None) == dps.DP_EINVAL
    assert lib.dp_dropout(R(addr=0), None, R(addr=0), 1, 0, 4, None, None) == dps.DP_OK


def _lookup(table=None, V=100, D=64, tok=TOK, ty=dps.DP_I64, P=2, T=3, drop=None, out=None):
    return dps.lib().dp_embedding_forward(table or R(), V, D, tok, ty, P, T, 1.0, drop,
                                          out or R(**FAR), None)


@pytest.mark.parametrize("kw,code,word", [
    (dict(V=0), dps.DP_EINVAL, "vocab outside"),
    (dict(D=0), dps.DP_EINVAL, "dim outside"),
    (dict(ty=2), dps.DP_EINVAL, "token type"),
    (dict(tok=None), dps.DP_EINVAL, "NULL tokens"),
    (dict(tok=C.c_void_p((1 << 34) + 4)), dps.DP_EALIGN, "tokens not aligned"),
    (dict(out=R(addr=(1 << 30) + 4096)), dps.DP_EINVAL, "overlaps table"),
    (dict(drop=C.byref(dps.dropout_cfg(2.0))), dps.DP_EINVAL, "dropout p"),
    (dict(P=0), dps.DP_EINVAL, "P outside"),
])
def test_lookup_refusals(kw, code, word):
    assert _lookup(**kw) == code
    assert word in _err()


def _grad(dout=None, tok=TOK, ty=dps.DP_I64, P=2, T=3, drop=None, grad=None, V=100, D=64, ws=WS,
          nbytes=1 << 40):
    return dps.lib().dp_embedding_backward(dout or R(), tok, ty, P, T, 1.0, drop, grad or R(**FAR),
                                           V, D, 0, ws, nbytes, None)


@pytest.mark.parametrize("kw,code,word", [
    (dict(ws=None), dps.DP_EINVAL, "NULL workspace"),
    (dict(ws=C.c_void_p((1 << 36) + 16)), dps.DP_EALIGN, "32-byte"),
    (dict(nbytes=8), dps.DP_EINVAL, "needs"),
    (dict(grad=R(rs=6399, **FAR)), dps.DP_EINVAL, "overlap"),
    (dict(grad=R(addr=(1 << 30) + 64)), dps.DP_EINVAL, "grad overlaps dout"),
    (dict(V=0), dps.DP_EINVAL, "vocab outside"),
    (dict(T=1 << 31), dps.DP_EINVAL, "2^31"),
    (dict(tok=None), dps.DP_EINVAL, "NULL tokens"),
])
def test_lookup_gradient_refusals(kw, code, word):
    assert _grad(**kw) == code
    assert word in _err()


def test_workspace_query():
    assert dps.dp_embedding_workspace_bytes(8, 1024, 50257, 768) > 0
    for args in ((0, 1, 1, 1), (1, -1, 1, 1), (1, 1, 0, 1), (1, 1, 1, 0)):
        with pytest.raises(dps.DPError) as e:
            dps.dp_embedding_workspace_bytes(*args)
        assert e.value.code == dps.DP_EINVAL
    assert dps.lib().dp_embedding_workspace_bytes(1, 1, 1, 1, None) == dps.DP_EINVAL


def _policy(logits=None, V=64, tok=TOK, ty=dps.DP_I32, old=VEC, rf=VEC, adv=VEC, w=VEC, cfg=None,
            logp=VEC, stats=VEC, dl=None, P=2, T=3):
    return dps.lib().dp_policy_loss(logits or R(), P, T, V, tok, ty, old, rf, adv, w,
                                    C.byref(cfg or dps.policy_cfg(kl_beta=0.1)), logp, stats,
                                    dl or R(**FAR), None)


@pytest.mark.parametrize("kw,code,word", [
    (dict(old=None), dps.DP_EINVAL, "NULL old_logp"),
    (dict(adv=None), dps.DP_EINVAL, "NULL advantage"),
    (dict(logp=None), dps.DP_EINVAL, "NULL logp"),
    (dict(stats=None), dps.DP_EINVAL, "NULL stats"),
    (dict(stats=None, T=0), dps.DP_EINVAL, "NULL stats"),
    (dict(rf=None), dps.DP_EINVAL, "needs ref_logp"),
    (dict(w=C.c_void_p(6)), dps.DP_EALIGN, "weight"),
    (dict(dl=R(dtype=dps.DP_F32, **FAR)), dps.DP_EINVAL, "logits' type"),
    (dict(dl=R(addr=(1 << 30) + 32)), dps.DP_EINVAL, "without being it"),
    (dict(cfg=dps.policy_cfg(clip_low=1.5)), dps.DP_EINVAL, "clip_low"),
    (dict(cfg=dps.policy_cfg(clip_low=-0.1)), dps.DP_EINVAL, "clip_low"),
    (dict(cfg=dps.policy_cfg(clip_high=-0.1)), dps.DP_EINVAL, "clip_high"),
    (dict(cfg=dps.policy_cfg(clip_high=float("inf"))), dps.DP_EINVAL, "clip_high"),
    (dict(cfg=dps.policy_cfg(kl_beta=-1.0)), dps.DP_EINVAL, "kl_beta"),
    (dict(cfg=dps.policy_cfg(logit_scale=0.0)), dps.DP_EINVAL, "logit_scale"),
    (dict(cfg=dps.policy_cfg(logit_scale=1e300)), dps.DP_EINVAL, "logit_scale"),
    (dict(V=0), dps.DP_EINVAL, "vocab outside"),
])
def test_policy_refusals(kw, code, word):
    assert _policy(**kw) == code
    assert word in _err()


def test_policy_needs_a_cfg():
    lib = dps.lib()
    assert lib.dp_policy_loss(R(), 1, 1, 4, TOK, 0, VEC, None, VEC, None, None, VEC, VEC, None,
                              None) == dps.DP_EINVAL
    assert "NULL cfg" in _err()


def test_logprob_refusals():
    lib = dps.lib()
    f = lib.dp_token_logprob
    assert f(R(), 2, 3, 64, TOK, 1, 1.0, None, None, None) == dps.DP_EINVAL
    assert "NULL logp" in _err()
    assert f(R(), 2, 3, 64, TOK, 1, -1.0, VEC, None, None) == dps.DP_EINVAL
    assert "logit_scale" in _err()
    assert f(R(), 2, 3, 64, TOK, 1, float("nan"), VEC, None, None) == dps.DP_EINVAL
    b = lib.dp_token_logprob_backward
    assert b(R(), 2, 3, 64, TOK, 1, 1.0, None, VEC, R(**FAR), None) == dps.DP_EINVAL
    assert b(R(), 2, 3, 64, TOK, 1, 1.0, VEC, None, R(**FAR), None) == dps.DP_EINVAL
    assert b(R(), 2, 3, 64, TOK, 1, 1.0, VEC, VEC, R(ws=32, **FAR), None) == dps.DP_EINVAL
    assert b(R(), 2, 3, 64, TOK, 1, 1.0, VEC, VEC, R(dtype=1, **FAR), None) == dps.DP_EINVAL
    assert b(R(), 2, 3, 64, TOK, 1, 1.0, VEC, VEC, R(ws=128), None) == dps.DP_EINVAL
    assert "without being it" in _err()


def test_column_slices_of_one_buffer_are_no_overlap():
    """[T][2 * 64] holds x in its left and out in its right half: refused only when the
    halves meet (the accepted form is not launched here: T = 0)."""
    lib = dps.lib()
    left = dict(addr=1 << 30, rs=1 << 20, ws=128)
    meet = dict(left, addr=(1 << 30) + 2 * 63)
    assert lib.dp_dropout(R(**left), None, R(**meet), 2, 3, 64, None, None) == dps.DP_EINVAL
    assert "without being it" in _err()


def test_binding_refusals():
    x = torch.zeros(2, 3, 8)
    with pytest.raises(ValueError, match="CUDA tensor"):
        dps.dp_dropout(x, x, None)
    with pytest.raises(TypeError, match="torch.Tensor"):
        dps.dp_dropout(x.numpy(), x, None)
    with pytest.raises(ValueError, match="CUDA tensor"):
        dps.dp_token_logprob(x, torch.zeros(2, 3, dtype=torch.int64), torch.zeros(2, 3))
    plan = dps.Plan([12, 30], 1 << 20, 2)
    buf = torch.arange(2 * plan.stride, dtype=torch.float32).view(2, plan.stride)
    v = plan.tensor_view(buf, 1, (5, 6))
    assert v.shape == (2, 5, 6) and v.stride() == (plan.stride, 6, 1)
    assert v[1, 2, 3] == plan.stride + plan.tensor(1)[1] + 15
    assert plan.tensor_view(buf[0], 0, (3, 4)).shape == (3, 4)
    with pytest.raises(ValueError, match="holds 30"):
        plan.tensor_view(buf, 1, (5, 7))
