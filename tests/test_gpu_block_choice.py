"""The experts that MoeBlock and MoeServer choose are those of the float64
logits y . Wr^T (y as the norm wrote it): with 256 experts, logits rounded to
bf16 move the k-th place of a large part of the tokens.

The products of bf16 factors are exact in fp32; the tensor cores add at least
16 of them at a time into an fp32 accumulator, each addition good to 2^-22 of
the magnitudes it joins, so a logit is within (H / 16 + 8) 2^-22 sum |y w| of
the float64 one.  A token two of whose k + 1 largest logits are closer than
twice that is left out; there may be one and 5% of them."""
import numpy as np
import pytest
import torch

from grouped_gemm_glu_gb300 import block, ops, synth
from grouped_gemm_glu_gb300 import lib as L
from grouped_gemm_glu_gb300.layer import MoeLayer
from parity import np_

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
N, K, E, F = 256, 8, 4, 64


@pytest.mark.parametrize("T,H", [(1, 256), (16, 1024), (512, 256)])
@pytest.mark.parametrize("who", ["block", "server"])
def test_choice_is_that_of_unrounded_logits(T, H, who, monkeypatch):
    rng = np.random.default_rng(T + H)
    bf = lambda *s, sc=1.0: synth._bf16(sc * rng.standard_normal(s)).to(DEV)
    x, res, gamma, Wr = bf(T, H), bf(T, H), bf(H), bf(N, H, sc=H ** -0.5)
    W1, W2 = bf(E, 2 * F, H, sc=H ** -0.5), bf(E, F, H, sc=F ** -0.5)
    prm, glu = L.router_params("softmax", renorm=True), L.glu_params("swiglu")
    seen = {}
    router = ops.router

    def watch(logits, *a, **kw):
        seen["logits"], seen["idx"] = logits, (o := router(logits, *a, **kw))["idx"]
        return o

    monkeypatch.setattr(block.ops, "router", watch)
    if who == "block":
        ly = MoeLayer(W1, W2, T, K, (T * K + 31 * E + 127) // 128 * 128, glu)
        block.MoeBlock(ly, gamma, Wr, prm).forward(x, res)
    else:
        block.MoeServer(W1, W2, gamma, Wr, K, prm, glu).step(x, res)
    y = np_(ops.rmsnorm(x, gamma, residual=res)["y"]).astype(np.float64)
    w = np_(Wr).astype(np.float64)
    ref, err = y @ w.T, (H / 16 + 8) * 2.0 ** -22 * (np.abs(y) @ np.abs(w).T)
    assert seen["logits"].dtype == torch.float32
    assert np.all(np.abs(np_(seen["logits"]) - ref) <= err)
    best = -np.sort(-ref, axis=1)[:, : K + 1]
    close = np.any(best[:, :-1] - best[:, 1:] <= 2 * err.max(1, keepdims=True), axis=1)
    assert close.sum() <= 1 + 0.05 * T
    assert np.array_equal(np_(seen["idx"])[~close], np.argsort(-ref, axis=1, kind="stable")[~close, :K])
