"""Groups that have lost experts (logit or bias of -inf).  A group's score is
the sum of its group_top best keys as they are: with group_top = 2, a group
with fewer than two experts left scores -inf, ranks behind every group with
two, and ties by index with the other groups of that kind, empty ones among
them.  With group_top = 1 a group counts while one expert is left."""
import numpy as np
import pytest
import torch

from grouped_gemm_glu_gb300 import lib as L
from grouped_gemm_glu_gb300 import ops
from parity import np_
from test_gpu_router import _choose

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
NINF = float("-inf")


def _idx(x, k, top, keep, bias=None):
    prm = L.router_params("sigmoid", renorm=True, n_group=4, topk_group=keep, group_top=top)
    return np_(ops.router(torch.tensor(x, dtype=torch.float32, device=DEV), k, prm, bias=bias)["idx"]).tolist()


@pytest.mark.parametrize("with_bias", [False, True])
def test_one_expert_left(with_bias):
    b = torch.zeros(8, device=DEV) if with_bias else None
    x = [[0.0, 0.1, 5.0, NINF, 0.3, 0.2, NINF, NINF]]  # group 1's best expert has no neighbour, group 3 is empty
    assert _idx(x, 2, 2, 2, b) == [[4, 5]]             # groups 0 and 2 have two
    assert _idx(x, 2, 1, 2, b) == [[2, 4]]             # with one key a group, expert 2 is first
    # three groups kept: 0, 2 and the first of the two that score -inf
    assert _idx(x, 5, 2, 3, b) == [[2, 4, 5, 1, 0]]
    y = [[NINF, NINF, 5.0, NINF, NINF, NINF, 0.3, NINF]]  # no group has two: the first two groups are kept
    assert _idx(y, 2, 2, 2, b) == [[2, -1]]
    assert _idx(y, 2, 1, 2, b) == [[2, 6]]
    if with_bias:  # switched off by the bias instead of the logit
        off = torch.tensor([0, 0, 0, NINF, 0, 0, NINF, NINF], device=DEV)
        assert _idx([[0.0, 0.1, 5.0, 1.0, 0.3, 0.2, 1.0, 1.0]], 2, 2, 2, off) == [[4, 5]]


@pytest.mark.parametrize("T,n,G,keep,k", [(300, 16, 8, 3, 4), (200, 256, 32, 6, 8), (200, 96, 4, 2, 5), (100, 24, 12, 5, 3),
                                          (64, 1024, 32, 5, 12)])
@pytest.mark.parametrize("top", [1, 2])
@pytest.mark.parametrize("with_bias", [False, True])
def test_many_dead_experts(T, n, G, keep, k, top, with_bias):
    """Against the definition in float64, near-ties left out as in the router's
    other tests (keys closer than 2^-20 at a place that decides)."""
    rng = np.random.default_rng(T + n + top)
    x = (1.5 * rng.standard_normal((T, n))).astype(np.float32)
    gs = n // G
    live = rng.integers(0, 3, (T, G, 1))  # 0, 1 or 2 and more experts of each group
    order = rng.permuted(np.broadcast_to(np.arange(gs), (T, G, gs)), axis=2)
    x[(order >= np.where(live == 2, gs, live)).reshape(T, n)] = NINF
    b = (0.1 * rng.standard_normal(n)).astype(np.float32) if with_bias else None
    prm = L.router_params("sigmoid", renorm=True, n_group=G, topk_group=keep, group_top=top)
    o = ops.router(torch.from_numpy(x).to(DEV), k, prm, bias=None if b is None else torch.from_numpy(b).to(DEV))
    ref, unsafe = _choose(x.astype(np.float64), k, "sigmoid", b, G, keep, top, None)
    idx = np_(o["idx"])
    assert unsafe.mean() <= 0.02
    assert np.array_equal(idx[~unsafe], ref[~unsafe])
    assert np.all(np_(o["prob"])[idx < 0] == 0)
    assert np.array_equal(np_(o["load"]), np.bincount(idx[idx >= 0], minlength=n))
