"""Sizes and factors of the step's operators that no kernel can take: refused before anything is
enqueued (fake device addresses)."""
import ctypes as C

import pytest

import gradient_sync_zero_gb300 as dps
from gradient_sync_zero_gb300 import build as dbuild

TOK, WS = C.c_void_p(1 << 34), C.c_void_p(1 << 36)


@pytest.fixture(scope="module", autouse=True)
def built():
    dbuild.build()


def R(addr, rs, ws, dtype=dps.DP_BF16):
    return C.byref(dps.Rows(addr, rs, ws, dtype, 0))


def _refused(rc, word):
    assert rc == dps.DP_EINVAL
    assert word in dps.lib().dp_last_error().decode()


@pytest.mark.parametrize("T,D", [(1 << 30, 1 << 23), (0x7FFFFFFF, 1 << 20)])
def test_embedding_gradient_of_more_ctas_than_a_grid_has(T, D):
    """One row of dout for every token (a row stride of 0)."""
    _refused(dps.lib().dp_embedding_backward(R(1 << 30, 0, 0), TOK, dps.DP_I32, 1, T, 1.0, None, R(1 << 50, 0, D), 100, D,
                                             0, WS, 1 << 61, None), "CTAs per rank")


def test_dropout_of_more_ctas_than_a_grid_has():
    T, D = 1 << 20, 1 << 30
    cfg = dps.dropout_cfg(0.5)
    _refused(dps.lib().dp_dropout(R(1 << 30, 0, 0), None, R(1 << 50, 0, D), 1, T, D, C.byref(cfg), None),
             "CTAs per rank")


@pytest.mark.parametrize("scale,p", [(float("inf"), 0.0), (float("nan"), 0.0), (-1e39, 0.1), (2e38, 0.5), (-2e38, 0.5),
                                     (float("inf"), 1.0)])
def test_embedding_scales_beyond_fp32(scale, p):
    lib, cfg = dps.lib(), dps.dropout_cfg(p)
    table, act = R(1 << 30, 1 << 20, 64), R(1 << 40, 1 << 20, 64)
    _refused(lib.dp_embedding_forward(table, 100, 64, TOK, dps.DP_I64, 2, 3, scale, C.byref(cfg), act, None), "finite")
    _refused(lib.dp_embedding_backward(act, TOK, dps.DP_I64, 2, 3, scale, C.byref(cfg), table, 100, 64, 0, WS, 1 << 40,
                                       None), "finite")
