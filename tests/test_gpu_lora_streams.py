"""Adapter calls of every kind at once on streams of their own, next to a layer's
step on another: kernels that hold tensor memory side by side, and the results
of each call alone."""
import numpy as np
import pytest
import torch

from grouped_gemm_glu_gb300 import lib as L
from grouped_gemm_glu_gb300 import ops, synth
from grouped_gemm_glu_gb300.layer import MoeLayer
from test_gpu_lora import DEV, Case

pytestmark = pytest.mark.gpu


def _call(c):
    o = ops.lora(c.x_, c.A_, c.B_, c.idx_, c.scale_, base=c.yb_)
    return [o["y"], o["h"], *ops.lora_bwd(c.dy_, c.x_, o["h"], c.A_, c.B_, c.idx_, c.scale_, base=c.xb_)]


def test_at_once():
    cases = [Case(700, 2048, 1024, 16, 3, "runs", seed=1), Case(900, 1024, 2048, 64, 3, "runs", seed=2),
             Case(600, 1032, 1024, 128, 2, "rows", seed=3), Case(512, 512, 2048, 48, 40, "rows", seed=4),
             Case(1500, 2048, 1032, 32, 5, "runs", seed=5), Case(60, 1024, 1024, 16, 9, "rows", seed=6)]
    rng = np.random.default_rng(7)
    T, H, E, k, F = 512, 512, 8, 2, 256
    bf = lambda *s, sc=1.0: synth._bf16(sc * rng.standard_normal(s)).to(DEV)
    layer = MoeLayer(bf(E, 2 * F, H, sc=H ** -0.5), bf(E, F, H, sc=F ** -0.5), T, k, (T * k + 31 * E + 127) // 128 * 128,
                     L.glu_params("swiglu"))
    x, dout = bf(T, H), bf(T, H)
    idx = torch.from_numpy(np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)).to(DEV)
    prob = torch.full((T, k), 0.5, device=DEV)
    want = [_call(c) for c in cases]
    layer.step(x, idx, prob, dout)
    torch.cuda.synchronize()
    kept = [layer.out.clone(), layer.dx.clone(), layer.dW1.clone(), layer.dW2.clone()]
    streams = [torch.cuda.Stream() for _ in range(len(cases) + 1)]
    for _ in range(20):
        got = []
        for s, c in zip(streams, cases):
            with torch.cuda.stream(s):
                got.append(_call(c))
        with torch.cuda.stream(streams[-1]):
            layer.step(x, idx, prob, dout)
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert all(torch.equal(a, b) for a, b in zip(g, w))
        assert all(torch.equal(a, b) for a, b in zip((layer.out, layer.dx, layer.dW1, layer.dW2), kept))
    assert ops.read_status(layer.status) == L.MOE_OK
