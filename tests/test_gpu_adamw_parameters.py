"""The optimizer on weights as models hold them: parameters that require
gradients, and weights whose tensor was given other memory."""
import copy

import pytest
import torch

from grouped_gemm_glu_gb300.optim import AdamW

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


def _parameters(seed=0):
    g = torch.Generator().manual_seed(seed)
    w = [torch.randn(*s, generator=g) for s in ((65, 40), (33,), (7, 3, 5))]
    return [torch.nn.Parameter(x.to(t).to(DEV)) for x, t in zip(w, (BF, F32, BF))]


def _grads(ws, seed):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(w.shape, generator=g).to(w.dtype).to(DEV) for w in ws]


@pytest.mark.parametrize("state", ["f32", "mxfp8"])
def test_parameters_that_require_gradients(state):
    kw = dict(lr=1e-2, weight_decay=0.1, state=state, seed=3)
    ws = _parameters()
    plain = [w.detach().clone() for w in ws]
    a, b = AdamW(ws, **kw), AdamW(plain, **kw)
    assert not a.master.requires_grad
    for k in range(2):
        a.step(_grads(ws, k))
        b.step(_grads(ws, k))
    keep = a.state_dict()
    assert all(v.grad_fn is None and not v.requires_grad for v in keep.values())
    copy.deepcopy(keep)
    at_two = [w.detach().clone() for w in ws]
    a.step(_grads(ws, 2))
    a.load_state_dict(keep)
    for w, p, old in zip(ws, plain, at_two):
        assert w.requires_grad and w.is_leaf
        if w.dtype == BF:  # (an f32 weight is not part of the state)
            assert torch.equal(w.detach(), old)
        else:
            w.data.copy_(old)
    a.step(_grads(ws, 3))
    b.step(_grads(ws, 3))
    assert all(torch.equal(w.detach(), p) for w, p in zip(ws, plain))
    assert all(torch.equal(v, b.state_dict()[k]) for k, v in a.state_dict().items())


def test_a_parameter_still_trains_behind_a_step():
    # the step changes the weight outside of what autograd records: a graph made afterwards sees the new values
    w = torch.nn.Parameter(torch.ones(64, dtype=BF, device=DEV))
    opt = AdamW([w], lr=0.5, weight_decay=0.0)
    for _ in range(2):
        (w.float() ** 2).sum().backward()
        assert torch.equal(w.grad.float(), (2 * w.detach().float()))
        opt.step([w.grad])
        w.grad = None
    assert bool((w.detach() < 0.1).all())


def test_a_load_writes_the_memory_that_the_step_writes():
    w = torch.ones(5000, dtype=BF, device=DEV)
    opt = AdamW([w], lr=0.5, weight_decay=0.0)
    keep = opt.state_dict()
    first = opt._memory[0]
    opt.step([torch.ones(5000, dtype=BF, device=DEV)])
    assert bool((first == 0.5).all())
    w.data = torch.full((5000,), 7.0, dtype=BF, device=DEV)
    opt.load_state_dict(keep)
    assert bool((first == 1).all()) and bool((w == 7).all())
    # ... and values of other sizes do not get in its way
    w.data = torch.full((3,), 7.0, dtype=BF, device=DEV)
    opt.load_state_dict(keep)
    assert bool((w == 7).all())
