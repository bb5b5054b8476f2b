"""Host checks of the AdamW entry points, and the plan that they write: no
device (the addresses here are never dereferenced)."""
import ctypes as C

import pytest

from grouped_gemm_glu_gb300 import build as B
from grouped_gemm_glu_gb300 import lib as L

A = 0x10000


@pytest.fixture(scope="module")
def lib():
    B.build()
    return L.load()


def _row(n=100, w=A, m=A, v=A, **kw):
    return L.AdamwTensor(w=w, m=m, v=v, n=n, **kw)


def _rows(*rows):
    return (L.AdamwTensor * max(1, len(rows)))(*rows)


def test_plan(lib):
    rows = _rows(_row(1), _row(0), _row(4097), _row(2048))
    size = lib.moe_adamw_plan_size(rows, 4)
    assert size == 4 * C.sizeof(L.AdamwTensor) + 8 * (1 + 0 + 3 + 1)
    buf = (C.c_uint8 * size)()
    assert lib.moe_adamw_plan(rows, 4, 0, C.addressof(buf), size) == L.MOE_OK
    table = (C.c_uint32 * 10).from_buffer(buf, 4 * C.sizeof(L.AdamwTensor))
    assert list(table) == [0, 0, 2, 0, 2, 1, 2, 2, 3, 0]
    assert lib.moe_adamw_plan(rows, 4, 0, C.addressof(buf), size - 1) == L.MOE_ERR_ARG
    assert lib.moe_adamw_plan(rows, 4, 2, C.addressof(buf), size) == L.MOE_ERR_ARG
    assert lib.moe_adamw_plan(None, 0, 0, None, 0) == L.MOE_OK
    for bad, state in ((_row(w=None), 0), (_row(m=None), 0), (_row(v=None), 0), (_row(n=-1), 0), (_row(n=1 << 43), 0),
                       (_row(w_bf16=1), 0), (_row(w=A + 2), 0), (_row(w=A + 1, master=A, w_bf16=1), 0),
                       (_row(m=A + 2), 0), (_row(), 1), (_row(m=A + 4, m_scale=A, v_scale=A), 1),
                       (_row(weight_decay=-1.0), 0), (_row(weight_decay=float("nan")), 0)):
        assert lib.moe_adamw_plan(_rows(bad), 1, state, C.addressof(buf), size) == L.MOE_ERR_ARG
    assert lib.moe_adamw_plan(_rows(_row(m_scale=A + 1, v_scale=A + 3)), 1, 1, C.addressof(buf), size) == L.MOE_OK


def test_step(lib):
    rows = _rows(_row(100))
    n_ws = lib.moe_adamw_workspace_size(1)

    def f(rows=rows, grads=(A,), n=1, plan=A, p=None, lr=A, t=A, ws=A, nbytes=n_ws):
        p = p or L.AdamwParams(0.9, 0.99, 1e-8, 0.0, 0, 0)
        g = (C.c_void_p * max(1, len(grads)))(*grads) if grads is not None else None
        return lib.moe_adamw_step(rows, g, n, plan, C.byref(p), lr, t, None, ws, nbytes, None)

    P = lambda b1=0.9, b2=0.99, eps=1e-8, mx=0.0, state=0: L.AdamwParams(b1, b2, eps, mx, state, 0)
    nan = float("nan")
    for kw in (dict(rows=None), dict(grads=None), dict(n=-1), dict(plan=None), dict(plan=A + 4), dict(lr=None), dict(t=None),
               dict(ws=None), dict(ws=A + 8), dict(nbytes=n_ws - 1), dict(grads=(None,)), dict(grads=(A + 2,)),
               dict(p=P(b1=1.0)), dict(p=P(b1=nan)), dict(p=P(b2=-0.1)), dict(p=P(eps=-1.0)), dict(p=P(mx=-1.0)),
               dict(p=P(mx=nan)), dict(p=P(state=3)), dict(p=P(state=1)), dict(rows=_rows(_row(w=None)))):
        assert f(**kw) == L.MOE_ERR_ARG, kw
    assert lib.moe_adamw_step(rows, None, 1, A, None, A, A, None, A, n_ws, None) == L.MOE_ERR_ARG
    assert lib.moe_adamw_workspace_size(9000) > n_ws and lib.moe_adamw_workspace_size(-1) == 0
