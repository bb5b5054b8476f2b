"""Shards of MoeServer: servers that hold a part of the experts each add up to
the server that holds them all.

The shards' rows are the whole server's (the same bf16 rows of every expert),
each output is an fp32 sum rounded to bf16 (2^-8 of its magnitude at most), so
|sum of the shards - whole| <= 2^-8 (sum |shard| + |whole|) and, for the fp32
sums in another order, 2^-20 of the same."""
import numpy as np
import pytest
import torch

from grouped_gemm_glu_gb300 import lib as L
from grouped_gemm_glu_gb300 import ops, synth
from grouped_gemm_glu_gb300.block import MoeServer
from parity import np_

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("T,cuts", [(1, (0, 4, 8)), (5, (0, 3, 8)), (200, (0, 2, 6, 8))])
def test_shards_add_up(T, cuts):
    H, n, k, F = 320, 8, 3, 192
    rng = np.random.default_rng(T)
    bf = lambda *s, sc=1.0: synth._bf16(sc * rng.standard_normal(s)).to(DEV)
    x, res, gamma, Wr = bf(T, H), bf(T, H, sc=2.0), bf(H), bf(n, H, sc=H ** -0.5)
    W1, W2, b1 = bf(n, 2 * F, H, sc=H ** -0.5), bf(n, F, H, sc=F ** -0.5), bf(n, 2 * F, sc=0.1)
    prm, glu = L.router_params("softmax", renorm=True), L.glu_params("swiglu")
    whole = MoeServer(W1, W2, gamma, Wr, k, prm, glu, b1=b1)
    out = np_(whole.step(x, res)[0]).astype(np.float64)
    parts = []
    for lo, hi in zip(cuts, cuts[1:]):
        s = MoeServer(W1[lo:hi], W2[lo:hi], gamma, Wr, k, prm, glu, b1=b1[lo:hi], expert_begin=lo)
        parts.append(np_(s.step(x, res)[0]).astype(np.float64))
        assert ops.read_status(s.status) == 0
    mag = sum(np.abs(p) for p in parts) + np.abs(out)
    assert np.abs(out).max() > 0 and sum(bool(p.any()) for p in parts) >= 1
    assert np.all(np.abs(sum(parts) - out) <= (2.0 ** -8 + 2.0 ** -20) * mag + 1e-30)


def test_shard_outside_the_experts_is_refused():
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device=DEV)
    for begin in (-1, 8):
        with pytest.raises(ValueError):
            MoeServer(z(4, 64, 64), z(4, 32, 64), z(64), z(8, 64), 2, L.router_params(), L.glu_params("swiglu"),
                      expert_begin=begin)
