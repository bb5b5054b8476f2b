"""GPU parity of the router (choice, weights, load) and of its backward
against the definition in float64.

The choice is exact where it is made on the logits themselves (no bias).  With
a bias the keys are fp32 sums of a score that is within 4 u (u = 2^-24) of the
formula's and a bias: a token whose float64 keys (or group scores) come closer
than 2^-20 at a place that decides, without being equal, is left out of the
comparison of indices; such tokens must stay below 2%.
Weights: a score is within 8 u of the formula's and a sum of at most 1024
positive terms within 64 u, so weights lie within 128 u of theirs.
Gradients: each is a few products and one warp sum: |err| <= 2^-19 scale
(|g| + sum |g w|) with w <= 1, plus 2^-8 of the value for bf16."""
import numpy as np
import pytest
import torch

from grouped_gemm_glu_gb300 import lib as L
from grouped_gemm_glu_gb300 import ops
from parity import np_

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
NINF = float("-inf")


def _scores(x, kind):
    with np.errstate(over="ignore", invalid="ignore"):
        if kind == "sigmoid":
            return 1.0 / (1.0 + np.exp(-x))
        m = np.where(np.isneginf(x.max(1, keepdims=True)), 0.0, x.max(1, keepdims=True))
        e = np.exp(x - m)
        return e / np.maximum(e.sum(1, keepdims=True), 1e-300)


def _choose(x, k, score, bias, G, keep, gtop, mask):
    """(idx [T, k], unsafe [T]) by the definition."""
    T, n = x.shape
    s = _scores(x, score)
    key = x if bias is None else np.where(np.isneginf(x), NINF, s + bias)
    exact = bias is None
    unsafe = np.zeros(T, bool)

    def close(v, m):  # some neighbours among the best m + 1 nearly tie
        v = -np.sort(-v, axis=1)[:, :m + 1]
        with np.errstate(invalid="ignore"):
            d = v[:, :-1] - v[:, 1:]
        return np.any((d > 0) & (d < 2.0 ** -20), axis=1)

    if G > 1:
        gk = key if (gtop == 1 or bias is not None) else np.where(np.isneginf(x), NINF, s)
        best = -np.sort(-gk.reshape(T, G, -1), axis=2)[:, :, :gtop]
        gs = best.sum(2)
        if not (exact and gtop == 1):
            unsafe |= close(gs, keep)
        order = np.argsort(-gs, axis=1, kind="stable")[:, :keep]
        on = np.zeros((T, G), bool)
        np.put_along_axis(on, order, True, 1)
        key = np.where(np.repeat(on, n // G, 1), key, NINF)
    if mask is not None:
        key = np.where(mask[:, None] != 0, key, NINF)
    if not exact:
        unsafe |= close(key, k)
    idx = np.argsort(-key, axis=1, kind="stable")[:, :k]
    val = np.take_along_axis(key, idx, 1)
    return np.where(np.isneginf(val), -1, idx), unsafe


def _weights(x, idx, score, renorm):
    s = _scores(x, score)
    on, at = idx >= 0, np.maximum(idx, 0)
    if renorm and score == "softmax":
        xs = np.where(on, np.take_along_axis(x, at, 1), NINF)
        return np.where(on, _scores(xs, "softmax"), 0.0)
    w = np.where(on, np.take_along_axis(s, at, 1), 0.0)
    return w / (w.sum(1, keepdims=True) + 1e-20) if renorm else w


CASES = [
    # T, n, k, score, bias, renorm, G, keep, gtop, dtype
    (1, 1, 1, "softmax", False, False, 1, 1, 1, "f32"),
    (1, 256, 8, "sigmoid", True, True, 8, 4, 2, "f32"),
    (777, 256, 8, "sigmoid", True, True, 8, 4, 2, "f32"),
    (300, 33, 5, "softmax", False, True, 1, 1, 1, "bf16"),
    (4099, 64, 6, "softmax", False, False, 1, 1, 1, "bf16"),
    (513, 160, 6, "softmax", False, False, 8, 3, 1, "f32"),
    (257, 1023, 32, "sigmoid", False, True, 1, 1, 1, "f32"),
    (65, 1024, 12, "softmax", False, True, 32, 5, 2, "f32"),
    (130, 96, 4, "softmax", True, True, 4, 2, 2, "f32"),
    (200, 40, 40 // 2, "sigmoid", True, False, 1, 1, 1, "bf16"),
    (90, 12, 3, "sigmoid", False, True, 12, 3, 2, "f32"),  # groups of one expert
    (64, 32, 32, "softmax", False, False, 1, 1, 1, "f32"),  # every expert
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(v) for v in c))
def test_choice_weights_load_and_gradient(case):
    T, n, k, score, with_bias, renorm, G, keep, gtop, dt = case
    rng = np.random.default_rng(T + n)
    x = (1.5 * rng.standard_normal((T, n))).astype(np.float32)
    if n > 8:
        x[:, rng.permutation(n)[: n // 8]] = NINF
    xt = torch.from_numpy(x).to(torch.bfloat16 if dt == "bf16" else torch.float32)
    x = np_(xt).astype(np.float64)
    bias = (0.1 * rng.standard_normal(n)).astype(np.float32) if with_bias else None
    mask = (rng.random(T) > 0.1).astype(np.uint8) if T > 50 else None
    prm = L.router_params(score, renorm=renorm, scale=1.75, n_group=G, topk_group=keep, group_top=gtop)
    xd = xt.to(DEV)
    o = ops.router(xd, k, prm, bias=None if bias is None else torch.from_numpy(bias).to(DEV),
                   token_mask=None if mask is None else torch.from_numpy(mask).to(DEV))
    idx = np_(o["idx"])
    ref, unsafe = _choose(x, k, score, bias, G, keep, gtop, mask)
    assert unsafe.mean() <= 0.02
    assert np.array_equal(idx[~unsafe], ref[~unsafe])
    assert np.array_equal(np_(o["load"]), np.bincount(idx[idx >= 0], minlength=n))
    if mask is not None:
        assert np.all(idx[mask == 0] == -1)
    w = 1.75 * _weights(x, idx, score, renorm)
    p = np_(o["prob"]).astype(np.float64)
    assert np.all(p[idx < 0] == 0) and np.all(np.abs(p - w) <= 128 * U * w)
    # gradient of sum(dprob * prob) for the choice made
    dprob = rng.standard_normal((T, k)).astype(np.float32)
    d = np_(ops.router_bwd(xd, o["idx"], torch.from_numpy(dprob).to(DEV), prm)).astype(np.float64)
    on, at = idx >= 0, np.maximum(idx, 0)
    g = np.where(on, 1.75 * dprob.astype(np.float64), 0.0)
    s = _scores(x, score)
    wv = w / 1.75
    refd = np.zeros((T, n + 1))
    rows = np.arange(T)[:, None]
    if renorm:
        inner = (g * wv).sum(1, keepdims=True)
        if score == "softmax":
            np.add.at(refd, (rows, idx + 1), np.where(on, wv * (g - inner), 0.0))
        else:
            se = np.where(on, np.take_along_axis(s, at, 1), 0.0)
            np.add.at(refd, (rows, idx + 1), np.where(on, wv * (g - inner) * (1.0 - se), 0.0))
        refd = refd[:, 1:]
    elif score == "softmax":
        np.add.at(refd, (rows, idx + 1), g * wv)
        refd = refd[:, 1:] - s * (g * wv).sum(1, keepdims=True)
    else:
        np.add.at(refd, (rows, idx + 1), g * wv * (1.0 - wv))
        refd = refd[:, 1:]
    lim = 2.0 ** -19 * (np.abs(g).max(1, keepdims=True) + np.abs(g * wv).sum(1, keepdims=True)) + 1e-30
    if dt == "bf16":
        lim = lim + 2.0 ** -8 * np.abs(refd)
    assert np.all(np.abs(d - refd) <= lim)
    assert np.all(d[np.isneginf(x)] == 0)


@pytest.mark.parametrize("score,renorm", [("softmax", False), ("softmax", True), ("sigmoid", False), ("sigmoid", True)])
def test_gradient_matches_differences(score, renorm):
    """dlogits against central differences (float64, step 1e-5, error ~1e-9)
    of the weights of the fixed choice; the fp32 gradient is within 2^-18."""
    rng = np.random.default_rng(9)
    T, n, k = 3, 20, 4
    x = rng.standard_normal((T, n)).astype(np.float32)
    prm = L.router_params(score, renorm=renorm, scale=2.0)
    xd = torch.from_numpy(x).to(DEV)
    o = ops.router(xd, k, prm)
    dprob = rng.standard_normal((T, k)).astype(np.float32)
    d = np_(ops.router_bwd(xd, o["idx"], torch.from_numpy(dprob).to(DEV), prm))
    idx = np_(o["idx"])

    def loss(z):
        return (2.0 * _weights(z, idx, score, renorm) * dprob).sum()

    for t in range(T):
        for e in range(n):
            h = np.zeros((T, n))
            h[t, e] = 1e-5
            num = (loss(x + h) - loss(x - h)) / 2e-5
            assert abs(num - d[t, e]) <= 2.0 ** -16


def test_ties_empty_rows_and_nonfinite():
    prm = L.router_params("softmax", renorm=True)
    x = torch.zeros(6, 70, device=DEV)
    x[1] = NINF                     # no expert at all
    x[2] = NINF
    x[2, 69] = 1.0                  # one expert for three slots
    x[3, 40] = float("nan")
    x[4, ::2] = -0.0                # equal to +0
    x[5] = torch.finfo(torch.float32).min
    o = ops.router(x, 3, prm)
    idx, p = np_(o["idx"]), np_(o["prob"])
    assert idx[0].tolist() == [0, 1, 2] and np.allclose(p[0], 1 / 3)
    assert idx[1].tolist() == [-1] * 3 and np.all(p[1] == 0)
    assert idx[2].tolist() == [69, -1, -1] and p[2].tolist() == [1, 0, 0]
    assert idx[3, 0] == 40 and np.all(np.isnan(p[3]))
    assert idx[4].tolist() == [0, 1, 2]
    assert idx[5].tolist() == [0, 1, 2] and np.allclose(p[5], 1 / 3)
    d = np_(ops.router_bwd(x, o["idx"], torch.ones(6, 3, device=DEV), prm))
    assert np.all(d[1] == 0) and np.all(d[2] == 0)
    # masked tokens may hold anything
    m = torch.ones(6, dtype=torch.bool, device=DEV)
    m[3] = False
    o = ops.router(x, 3, prm, token_mask=m)
    assert np_(o["idx"])[3].tolist() == [-1] * 3 and np.all(np_(o["prob"])[3] == 0)
    for kind, rn in (("softmax", False), ("softmax", True), ("sigmoid", False), ("sigmoid", True)):
        assert np.all(np_(ops.router_bwd(x, o["idx"], torch.ones(6, 3, device=DEV), L.router_params(kind, rn)))[3] == 0)
    assert int(o["load"].sum()) == 10  # three, one, three and three experts of rows 0, 2, 4, 5
    # sigmoids that underflow: the renormalised weights are 0, not NaN
    y = torch.full((1, 8), -200.0, device=DEV)
    assert np.all(np_(ops.router(y, 2, L.router_params("sigmoid", renorm=True))["prob"]) == 0)


def test_side_stream_empty_batch_and_route():
    rng = np.random.default_rng(1)
    x = torch.from_numpy(rng.standard_normal((64, 16)).astype(np.float32)).to(DEV)
    prm = L.router_params("softmax")
    want = ops.router(x, 2, prm)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = ops.router(x, 2, prm)
    s.synchronize()
    assert all(torch.equal(want[k], got[k]) for k in want)
    e = ops.router(x[:0], 2, prm)
    assert e["idx"].shape == (0, 2) and int(e["load"].sum()) == 0
    assert ops.router_bwd(x[:0], e["idx"], e["prob"], prm).shape == (0, 16)
    # the choice feeds the routing as it is; -1 slots are dropped there
    x[5] = NINF
    o = ops.router(x, 2, prm)
    h = torch.zeros(64, 64, dtype=torch.bfloat16, device=DEV)
    r = ops.route_permute(h, o["idx"], o["prob"], 16, 64 * 2 + 16 * 32)
    assert np_(r["counts"]).tolist() == np_(o["load"]).tolist()
    assert np.all(np_(r["row_of"]).reshape(64, 2)[5] == -1)


def test_refusals():
    x = torch.zeros(4, 16, device=DEV)
    ok = L.router_params()
    for bad in (lambda: ops.router(x.double(), 2, ok), lambda: ops.router(x.cpu(), 2, ok),
                lambda: ops.router(x.t(), 2, ok), lambda: ops.router(x, 2, ok, bias=torch.zeros(8, device=DEV)),
                lambda: ops.router(x, 2, ok, token_mask=torch.zeros(3, dtype=torch.uint8, device=DEV)),
                lambda: ops.router_bwd(x, torch.zeros(4, 2, dtype=torch.int64, device=DEV), x[:, :2].contiguous(), ok)):
        with pytest.raises(ValueError):
            bad()
    for k, prm in ((0, ok), (17, ok), (2, L.router_params(n_group=3)), (9, L.router_params(n_group=2, topk_group=1)),
                   (2, L.router_params(n_group=2, topk_group=3)), (2, L.router_params(group_top=3))):
        with pytest.raises(L.MoeError):
            ops.router(x, k, prm)
    with pytest.raises(L.MoeError):
        ops.router(torch.zeros(2, 1025, device=DEV), 2, ok)


@pytest.mark.parametrize("T,n,k,score,bias,renorm,dt", [
    (1, 5, 3, "softmax", False, True, "f32"), (3, 32, 8, "sigmoid", True, True, "bf16"),
    (1001, 8, 2, "softmax", False, False, "f32"), (4100, 61, 7, "softmax", False, False, "f32"),
    (259, 64, 8, "sigmoid", True, False, "bf16"), (515, 100, 16, "softmax", True, True, "f32"),
    (130, 128, 9, "sigmoid", False, True, "f32"), (33, 64, 9, "softmax", False, True, "f32"),
    (70, 33, 8, "softmax", False, True, "bf16"), (2, 24, 8, "sigmoid", True, True, "f32")])
def test_few_experts(T, n, k, score, bias, renorm, dt):
    """Sizes at which a token has part of a warp (and one, k = 9 of 64, that
    does not): rows past T in the last warp, masked tokens beside live ones,
    rows with fewer live experts than slots, coarse logits with many ties."""
    rng = np.random.default_rng(T * n)
    x = np.round(4 * rng.standard_normal((T, n))).astype(np.float32) / 4
    x[rng.random((T, n)) < 0.1] = NINF
    x[:: 7, k // 2:] = NINF
    xt = torch.from_numpy(x).to(torch.bfloat16 if dt == "bf16" else torch.float32)
    b = (np.round(64 * 0.1 * rng.standard_normal(n)) / 64).astype(np.float32) if bias else None
    mask = (rng.random(T) > 0.2).astype(np.uint8)
    prm = L.router_params(score, renorm=renorm, scale=0.5)
    o = ops.router(xt.to(DEV), k, prm, bias=None if b is None else torch.from_numpy(b).to(DEV),
                   token_mask=torch.from_numpy(mask).to(DEV))
    x = np_(xt).astype(np.float64)
    ref, unsafe = _choose(x, k, score, b, 1, 1, 1, mask)
    idx = np_(o["idx"])
    assert unsafe.mean() <= 0.02
    assert np.array_equal(idx[~unsafe], ref[~unsafe])
    w = 0.5 * _weights(x, idx, score, renorm)
    assert np.all(np.abs(np_(o["prob"]) - w) <= 128 * U * w)
    assert np.array_equal(np_(o["load"]), np.bincount(idx[idx >= 0], minlength=n))


@pytest.mark.parametrize("n", [64, 512])
def test_past_32_bits(n):
    """More than 2^31 logits: the last tokens are those of a small call."""
    T = (1 << 31) // n + 1000
    x = torch.full((T, n), -1.0, dtype=torch.bfloat16, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(1)
    x[-500:] = torch.randn(500, n, generator=g, device=DEV).to(torch.bfloat16)
    prm = L.router_params("softmax")
    o, w = ops.router(x, 3, prm), ops.router(x[-500:].contiguous(), 3, prm)
    assert torch.equal(o["idx"][-500:], w["idx"]) and torch.equal(o["prob"][-500:], w["prob"])
    assert int(o["load"].sum()) == 3 * T
    d = ops.router_bwd(x, o["idx"], o["prob"], prm)
    assert torch.equal(d[-500:], ops.router_bwd(x[-500:].contiguous(), w["idx"], w["prob"], prm))
