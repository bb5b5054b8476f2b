"""The norm written over its inputs, which the header allows: h over x or over
the residual, dx over dy or over dres.  The bits are those of separate outputs,
on both sides of the few-rows rule and with more rows than a CTA has in flight
(4000 x 2880: 760 row groups on 152 CTAs, three rows ahead; 9000 x 256: 2432
groups of one warp)."""
import ctypes as C

import pytest
import torch

from grouped_gemm_glu_gb300 import lib as L
from grouped_gemm_glu_gb300 import ops

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
SIZES = [(1, 8), (100, 2880), (405, 2880), (4000, 2880), (9000, 256), (700, 16384), (3000, 1032)]


def _rand(T, H, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return [torch.randn(T, H, generator=g, device=DEV).to(torch.bfloat16) for _ in range(3)]


def _p(t):
    return None if t is None else C.c_void_p(t.data_ptr())


@pytest.mark.parametrize("T,H", SIZES)
@pytest.mark.parametrize("over", ["x", "residual"])
def test_forward(T, H, over):
    x, res, gm = _rand(T, H, T + H)
    gamma, mx = gm[0].contiguous(), H % 32 == 0
    want = ops.rmsnorm(x, gamma, residual=res, mxfp8=mx)
    a = {"x": x.clone(), "residual": res.clone()}
    h = a[over]
    y, r = torch.empty_like(x), torch.empty(T, dtype=torch.float32, device=DEV)
    q = torch.empty(T, H, dtype=torch.uint8, device=DEV) if mx else None
    s = torch.empty(T, H // 32, dtype=torch.uint8, device=DEV) if mx else None
    L.check(L.load().moe_rmsnorm_fwd(_p(a["x"]), _p(a["residual"]), _p(gamma), 1e-5, T, H, _p(h), _p(y), _p(q), _p(s),
                                     _p(r), torch.cuda.current_stream().cuda_stream), "moe_rmsnorm_fwd")
    for k, v in (("h", h), ("y", y), ("rstd", r)) + ((("q", q), ("s", s)) if mx else ()):
        assert torch.equal(v, want[k]), k


@pytest.mark.parametrize("T,H", SIZES)
@pytest.mark.parametrize("over,dres", [("dy", True), ("dy", False), ("dres", True)])
def test_backward(T, H, over, dres):
    dy, e, h = _rand(T, H, T * 3 + H)
    gamma = (1 + 0.1 * _rand(1, H, 7)[0][0].float()).to(torch.bfloat16)
    rstd = torch.rsqrt(h.float().square().mean(1) + 1e-5)
    want, wg = ops.rmsnorm_bwd(dy, h, gamma, rstd, dres=e if dres else None)
    a = {"dy": dy.clone(), "dres": e.clone() if dres else None}
    dg, lib = torch.empty(H, dtype=torch.float32, device=DEV), L.load()
    n = lib.moe_rmsnorm_bwd_workspace_size(T, H)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    L.check(lib.moe_rmsnorm_bwd(_p(a["dy"]), _p(a["dres"]), _p(h), _p(gamma), _p(rstd), T, H, _p(a[over]), _p(dg), _p(ws),
                                n, torch.cuda.current_stream().cuda_stream), "moe_rmsnorm_bwd")
    assert torch.equal(a[over], want) and torch.equal(dg, wg)
