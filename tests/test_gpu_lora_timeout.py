"""The adapters' kernels with waits that give up: under the least limit every
wait does that would have to wait.  A call then ends, reports it, writes nothing
outside its outputs, and leaves no copy under way: the calls behind it are right."""
import pytest
import torch

from grouped_gemm_glu_gb300 import lib as L
from grouped_gemm_glu_gb300 import ops
from test_gpu_lora import DEV, Case

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
DEFAULT_LIMIT_NS = 2_000_000_000


def _guarded(*shape):
    n = 1
    for s in shape:
        n *= s
    full = torch.full((n + 512,), 3.0, dtype=BF, device=DEV)
    return full, full[256:-256].view(*shape)


# one stage and many, ranks with base loaded ahead and without, one box and single rows, one CTA and clusters
@pytest.mark.parametrize("T,K,N,r,G,order", [(300, 64, 128, 16, 1, "one"), (700, 2048, 1048, 16, 3, "runs"),
                                             (700, 2048, 1048, 16, 3, "rows"), (600, 4096, 264, 40, 40, "rows"),
                                             (513, 1000, 520, 64, 2, "runs"), (700, 520, 2048, 128, 3, "rows"),
                                             (3000, 2048, 2048, 128, 4, "runs"), (8192, 2048, 2048, 32, 8, "runs")])
def test_waits_that_give_up(T, K, N, r, G, order):
    lib = L.load()
    c = Case(T, K, N, r, G, order, seed=T + r)
    want = ops.lora(c.x_, c.A_, c.B_, c.idx_, c.scale_, base=c.yb_)
    back = ops.lora_bwd(c.dy_, c.x_, want["h"], c.A_, c.B_, c.idx_, c.scale_, base=c.xb_)
    torch.cuda.synchronize()
    p = lambda t: None if t is None else t.data_ptr()
    stream = torch.cuda.current_stream().cuda_stream
    n, nb = lib.moe_lora_fwd_workspace_size(T, r, G), lib.moe_lora_bwd_workspace_size(T, r, G)
    ws = torch.full((max(n, nb) + 512,), 0xFF, dtype=torch.uint8, device=DEV)
    seen = []
    for _ in range(4):
        fy, y = _guarded(T, N)
        fh, h = _guarded(T, r)
        outs = [_guarded(*s) for s in ((T, K), (G, r, K), (G, r, N))]
        status = ops.new_status(DEV)
        ws.fill_(0xFF)
        lib.moe_set_wait_limit_ns(1)
        try:
            assert lib.moe_lora_fwd(p(c.x_), p(c.A_), p(c.B_), p(c.idx_), p(c.scale_), p(c.yb_), T, K, N, r, G, p(y), p(h), p(ws),
                                    n, p(status), stream) == L.MOE_OK
            forward = ops.read_status(status)
            assert bool((ws[n:] == 0xFF).all())
            ws.fill_(0xFF)
            assert lib.moe_lora_bwd(p(c.dy_), p(c.x_), p(want["h"]), p(c.A_), p(c.B_), p(c.idx_), p(c.scale_), p(c.xb_), T, K, N,
                                    r, G, *(p(v) for _, v in outs), p(ws), nb, p(status), stream) == L.MOE_OK
            backward = ops.read_status(status)
            assert bool((ws[nb:] == 0xFF).all())
        finally:
            lib.moe_set_wait_limit_ns(DEFAULT_LIMIT_NS)
        assert forward in (L.MOE_OK, L.MOE_ERR_TIMEOUT) and backward in (L.MOE_OK, L.MOE_ERR_TIMEOUT)
        seen += [forward, backward]
        for full in (fy, fh, *(f for f, _ in outs)):
            assert bool((full[:256] == 3).all()) and bool((full[-256:] == 3).all())
        if forward == L.MOE_OK:
            assert torch.equal(y, want["y"]) and torch.equal(h, want["h"])
        if backward == L.MOE_OK:
            assert all(torch.equal(v, w) for (_, v), w in zip(outs, back))
        o = ops.lora(c.x_, c.A_, c.B_, c.idx_, c.scale_, base=c.yb_)
        g = ops.lora_bwd(c.dy_, c.x_, o["h"], c.A_, c.B_, c.idx_, c.scale_, base=c.xb_)
        assert torch.equal(o["y"], want["y"]) and torch.equal(o["h"], want["h"])
        assert all(torch.equal(a, b) for a, b in zip(g, back))
    assert L.MOE_ERR_TIMEOUT in seen
