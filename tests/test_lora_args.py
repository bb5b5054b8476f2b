"""Host checks of the adapters' entry points: no device (the addresses here are
never dereferenced)."""
import pytest

from grouped_gemm_glu_gb300 import build as B
from grouped_gemm_glu_gb300 import lib as L

A = 0x100000


@pytest.fixture(scope="module")
def lib():
    B.build()
    return L.load()


def test_forward(lib):
    n = lib.moe_lora_fwd_workspace_size(1000, 16, 4)
    assert n > 1000 * 4 + 1000 * 32
    assert lib.moe_lora_fwd_workspace_size(-1, 16, 4) == lib.moe_lora_fwd_workspace_size(400, 0, 4) == 0
    assert lib.moe_lora_fwd_workspace_size(1, 16, 4) == 0  # few rows need none
    P = [A + (i << 24) for i in range(9)]

    def f(x=P[0], a=P[1], b=P[2], idx=P[3], scale=P[4], base=None, T=1000, K=64, N=64, r=16, G=4, y=P[5], h=P[6], ws=P[7],
          nbytes=n):
        return lib.moe_lora_fwd(x, a, b, idx, scale, base, T, K, N, r, G, y, h, ws, nbytes, None, None)

    for kw in (dict(x=None), dict(a=None), dict(b=None), dict(idx=None), dict(scale=None), dict(y=None), dict(ws=None),
               dict(nbytes=n - 1), dict(T=-1), dict(T=(1 << 27) + 1), dict(K=0), dict(K=60), dict(N=12), dict(r=0),
               dict(r=4), dict(G=0), dict(K=(1 << 20) + 8), dict(x=P[0] + 8), dict(a=P[1] + 2), dict(b=P[2] + 8),
               dict(base=P[8] + 8), dict(y=P[5] + 8), dict(h=P[6] + 8), dict(ws=P[7] + 16), dict(y=P[0]), dict(y=P[1]),
               dict(y=P[2] + 16), dict(base=P[5] + 16), dict(y=P[3]), dict(y=P[4]), dict(y=P[6] - 1024), dict(h=P[0]),
               dict(h=P[3]), dict(h=P[8], base=P[8])):
        assert f(**kw) == L.MOE_ERR_ARG, kw
    assert f(r=136) == f(G=32768) == L.MOE_ERR_UNSUPPORTED
    assert f(T=0, x=None, y=None, ws=None) == L.MOE_OK


def test_backward(lib):
    n = lib.moe_lora_bwd_workspace_size(100, 16, 4)
    P = [A + (i << 24) for i in range(12)]

    def f(dy=P[0], x=P[1], h=P[2], a=P[3], b=P[4], idx=P[5], scale=P[6], base=None, T=100, K=64, N=64, r=16, G=4, dx=P[7],
          da=P[8], db=P[9], ws=P[10], nbytes=n):
        return lib.moe_lora_bwd(dy, x, h, a, b, idx, scale, base, T, K, N, r, G, dx, da, db, ws, nbytes, None, None)

    for kw in (dict(dy=None), dict(x=None), dict(h=None), dict(a=None), dict(b=None), dict(idx=None), dict(scale=None),
               dict(dx=None), dict(da=None), dict(db=None), dict(ws=None), dict(nbytes=n - 1), dict(T=-1), dict(K=4),
               dict(N=0), dict(r=12), dict(G=-1), dict(dy=P[0] + 8), dict(x=P[1] + 8), dict(h=P[2] + 8), dict(da=P[8] + 8),
               dict(dx=P[7] + 2), dict(ws=P[10] + 128), dict(dx=P[0]), dict(dx=P[1]), dict(dx=P[2]), dict(dx=P[3]),
               dict(da=P[3]), dict(db=P[4]), dict(base=P[7] + 32), dict(dx=P[4]), dict(dx=P[5]), dict(da=P[1]), dict(da=P[4]),
               dict(da=P[7]), dict(db=P[0] + 64), dict(db=P[2]), dict(db=P[8]), dict(db=P[6])):
        assert f(**kw) == L.MOE_ERR_ARG, kw
    assert f(r=136) == L.MOE_ERR_UNSUPPORTED
