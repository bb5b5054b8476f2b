"""Clipping of gradients far larger than max_norm: the clipped step is the
formula's as long as the norm is finite.

The clipping factor c is then far below 1 and its square below what fp32
holds, while c g is an ordinary number: the bounds are those of ordinary
steps (test_gpu_adamw.py)."""
import pytest
import torch

from test_gpu_adamw import BF, F32, Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("state", ["f32", "mxfp8"])
@pytest.mark.parametrize("gtype", [F32, BF])
@pytest.mark.parametrize("size,max_norm", [(1e15, 1e-2), (1e17, 1.0), (1e18, 1e-2), (1e18, 1e-6), (1e18, 1e-12)])
def test_spikes(state, gtype, size, max_norm):
    c = Case([1, 257, 5003, 40000], (BF, F32), (gtype,), seed=21, state=state, max_norm=max_norm, betas=(0.9, 0.999))
    for _ in range(2):
        was = c.before()
        # elements from size / 100 to size, the norm at least 0.5 size sqrt(45261) = 106 size and at most 213: the smallest v is
        # at least 0.001 (max_norm / 21300)^2, 2.2e-36 for 1e-12, where v below 2^-126 = 1.2e-38 would count as 0
        g = [(x.sign() * size * (0.01 + 0.99 * torch.rand_like(x, dtype=F32))).to(gtype) for x in c.grads()]
        norm = c.opt.step(g)
        assert bool(torch.isfinite(norm))
        c.check(g, was, norm)


def test_a_spike_after_ordinary_steps_moves_the_weights_no_further_than_its_clipped_size():
    c = Case([40000], (BF,), (F32,), seed=22, state="f32", max_norm=1e-2, betas=(0.9, 0.999))
    for k in range(3):
        was = c.before()
        g = c.grads()
        if k == 1:
            g = [x * 1e19 for x in g]
        c.check(g, was, c.opt.step(g))
