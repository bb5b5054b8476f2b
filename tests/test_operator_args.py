"""Host checks of the norm's, the router's and the MXFP4 entry points: what
they refuse, they refuse without a device and before anything is launched
(the addresses here are never dereferenced)."""
import ctypes as C

import pytest

from grouped_gemm_glu_gb300 import build as B
from grouped_gemm_glu_gb300 import lib as L

A, A8, A4 = 0x10000, 0x10008, 0x10004  # 16-, 8- and 4-byte aligned


@pytest.fixture(scope="module")
def lib():
    B.build()
    return L.load()


def test_rmsnorm(lib):
    f = lambda x=A, res=None, g=A, eps=1e-5, T=4, H=64, h=None, y=A, q=None, s=None: lib.moe_rmsnorm_fwd(
        x, res, g, eps, T, H, h, y, q, s, None, None)
    for kw in (dict(x=None), dict(g=None), dict(eps=-1.0), dict(eps=float("nan")), dict(T=-1), dict(T=(1 << 30) + 1),
               dict(H=0), dict(H=60), dict(res=A), dict(h=A), dict(y=None), dict(q=A), dict(q=A, s=A, H=40),
               dict(x=A8), dict(y=A8), dict(q=A4, s=A)):
        assert f(**kw) == L.MOE_ERR_ARG, kw
    assert f(H=16392) == L.MOE_ERR_UNSUPPORTED
    assert f(T=0, x=None, g=None, y=None) == L.MOE_OK
    b = lambda dy=A, h=A, g=A, r=A, T=4, H=64, dx=A, dg=None, ws=None, n=0, dres=None: lib.moe_rmsnorm_bwd(
        dy, dres, h, g, r, T, H, dx, dg, ws, n, None)
    for kw in (dict(dy=None), dict(h=None), dict(g=None), dict(r=None), dict(dx=None), dict(H=12), dict(dy=A8),
               dict(dres=A8), dict(dg=A), dict(dg=A, ws=A, n=64), dict(dg=A, ws=A8, n=1 << 20)):
        assert b(**kw) == L.MOE_ERR_ARG, kw
    assert b(T=0) == L.MOE_OK
    assert lib.moe_rmsnorm_bwd_workspace_size(4, 64) >= 4 * 64 * 4
    assert lib.moe_rmsnorm_bwd_workspace_size(0, 64) == 0
    assert lib.moe_dequantize_mxfp8(A, A, 0, A, None) == L.MOE_OK
    assert lib.moe_dequantize_mxfp8(A8, A, 4, A, None) == L.MOE_ERR_ARG


def test_router(lib):
    def f(n=16, k=2, T=4, p=None, x=A):
        p = p or L.router_params()
        return lib.moe_router_fwd(x, 0, None, None, T, n, k, C.byref(p), A, A, None, None)
    for kw in (dict(n=0), dict(n=1025), dict(k=0), dict(k=17), dict(n=64, k=33), dict(T=-1), dict(x=None),
               dict(T=1 << 30), dict(p=L.router_params(n_group=3)), dict(p=L.router_params(n_group=4, topk_group=5)),
               dict(p=L.router_params(n_group=4, topk_group=1), k=5), dict(p=L.router_params(group_top=0)),
               dict(n=64, p=L.router_params(n_group=64)), dict(p=L.router_params(scale=float("nan"))),
               dict(p=L.RouterParams(7, 0, 1, 1, 1, 1.0))):
        assert f(**kw) == L.MOE_ERR_ARG, kw
    assert lib.moe_router_fwd(A, 0, None, None, 4, 16, 2, None, A, A, None, None) == L.MOE_ERR_ARG
    assert f(T=0, x=None) == L.MOE_OK
    p = L.router_params()
    assert lib.moe_router_bwd(A, 0, A, None, 4, 16, 2, C.byref(p), A, None) == L.MOE_ERR_ARG
    assert lib.moe_router_bwd(None, 0, None, None, 0, 16, 2, C.byref(p), None, None) == L.MOE_OK


def test_mxfp4(lib):
    for args in ((None, 1, 32, 32, 0, A, A), (A, 1, 48, 32, 0, A, A), (A, 1, 32, 40, 1, A, A), (A8, 1, 32, 32, 0, A, A),
                 (A, 0, 32, 32, 0, A, A), (A, 1, 32, 32, 0, A8, A), (A, 1, 32, 32, 0, A, A8)):
        assert lib.moe_quantize_mxfp4(*args, None, None) == L.MOE_ERR_ARG, args
    assert lib.moe_dequantize_mxfp4(A, A, 1, 32, 40, A, None) == L.MOE_ERR_ARG
    assert lib.moe_mxfp4_code_bytes(2, 32, 160) == 2 * 32 * 128 and lib.moe_mxfp4_scale_bytes(2, 32, 160) == 2 * 2 * 1024
    n = lib.moe_grouped_mxfp4_workspace_size(4, 256, 1152)
    assert n > 0 and lib.moe_grouped_mxfp4_workspace_size(0, 256, 1152) == 0
    out = L.ActOut(y=A)

    def fc2(a=(L.IN_MXFP8, A, A, None), w=(L.IN_MXFP4, A, A, None), ws=A, nb=n, K=256, N=64):
        return lib.moe_grouped_fc2_fwd(C.byref(L.InT(*a)), C.byref(L.InT(*w)), A, A, 4, K, N, 1152, 0, C.byref(out), ws,
                                       nb, 0, None, None)
    for kw in (dict(a=(L.IN_BF16, A, None, None)), dict(a=(L.IN_MXFP4, A, A, None)), dict(w=(L.IN_MXFP4, 0x10010, A, None)),
               dict(w=(L.IN_MXFP4, A, A8, None)), dict(w=(L.IN_MXFP4, A, None, None)), dict(ws=None), dict(nb=n - 1),
               dict(K=250), dict(N=40)):
        assert fc2(**kw) == L.MOE_ERR_ARG, kw
    p = L.glu_params("swiglu")
    f = lambda w=A, ws=A, nb=n: lib.moe_grouped_fc1_glu_quant_fwd_mxfp4(
        A, A, w, A, None, None, A, A, 4, 256, 64, 1152, C.byref(p), 0, C.byref(out), ws, nb, 0, None, None)
    assert f(w=0x10010) == L.MOE_ERR_ARG and f(ws=None) == L.MOE_ERR_ARG and f(nb=n - 1) == L.MOE_ERR_ARG


def test_route_permute_mxfp8(lib):
    f = lambda x=A, H=64, R=128, ws=A, n=1 << 16: lib.moe_route_permute_mxfp8(
        x, A, A, A, 4, H, 2, 0, 4, R, A, A, A, A, A, A, A, ws, n, None, None)
    for kw in (dict(x=None), dict(x=A8), dict(H=48), dict(R=100), dict(ws=None), dict(n=16)):
        assert f(**kw) == L.MOE_ERR_ARG, kw
