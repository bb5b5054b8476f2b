"""GPU tests of the low-rank adapters against their formulas in float64.

Tolerances (e = 2^-23, at most what one fp32 addition in the tensor cores
loses of its larger operand; b = 2^-8, half a bf16 step):
  * h = bf16(scale sum_k A x): |err| <= b |h| + (K + 2) e scale sum |A x|;
  * y = bf16(base + sum_j B h): what h is off by, times |B|, and its own
    rounding and sums: b |y| (1 + b) + sum |B| err(h) + (r + 2) e (sum |B h| + |base|);
  * dx likewise with u for h; dB = bf16(sum over n rows of h dy) from the h that
    the call gets: b |dB| + (n + 2) e sum |h dy|; dA from u: and sum |x| err(u).
Infinities and NaN are compared by where they are.
"""
import numpy as np
import pytest
import torch

from grouped_gemm_glu_gb300 import lib as L
from grouped_gemm_glu_gb300 import ops

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F64 = torch.bfloat16, torch.float64
E, B = 2.0 ** -23, 2.0 ** -8


def _idx(rng, T, G, order):
    if order == "rows":
        idx = rng.integers(-1, G, T)
    elif order == "runs":
        cuts = np.sort(rng.integers(0, T + 1, min(T, 6)))
        idx = np.repeat(rng.integers(-1, G, len(cuts) + 1), np.diff(np.concatenate([[0], cuts, [T]])))
    elif order == "one":
        idx = np.full(T, G - 1)
    else:  # nobody, in every way of saying so
        idx = rng.choice([-1, G, G + 7, -2 ** 31, 2 ** 31 - 1], T)
    return torch.from_numpy(idx.astype(np.int32))


class Case:
    def __init__(self, T, K, N, r, G, order, seed=0, base=True):
        rng = np.random.default_rng(seed)
        f = lambda *s, sc=1.0: (torch.from_numpy(rng.standard_normal(s).astype(np.float32)) * sc).to(BF)
        self.T, self.K, self.N, self.r, self.G = T, K, N, r, G
        self.x, self.dy = f(T, K), f(T, N)
        self.A, self.B = f(G, r, K, sc=K ** -0.5), f(G, r, N, sc=r ** -0.5)
        self.scale = torch.from_numpy(rng.uniform(0.25, 2.0, G).astype(np.float32))
        self.idx = _idx(rng, T, G, order)
        self.yb, self.xb = (f(T, N), f(T, K)) if base else (None, None)
        for k in ("x", "dy", "A", "B", "scale", "idx", "yb", "xb"):
            v = getattr(self, k)
            setattr(self, k + "_", v.to(DEV) if v is not None else None)

    def rows(self, a):
        return torch.nonzero(self.idx == a).view(-1)

    def half(self, X, P, Q, base, width, h_given=None):
        """(h, its error, out, its error) of one direction, float64."""
        X, P, Q = X.to(F64), P.to(F64), Q.to(F64)
        h, eh = torch.zeros(self.T, self.r, dtype=F64), torch.zeros(self.T, self.r, dtype=F64)
        y = torch.zeros(self.T, width, dtype=F64) if base is None else base.to(F64).clone()
        ey = 0 * y
        size = y.abs()
        for a in set(self.idx.tolist()):
            if not 0 <= a < self.G:
                continue
            t, s = self.rows(a), float(self.scale[a])
            h[t] = s * (X[t] @ P[a].T)
            eh[t] = B * h[t].abs() + (X.shape[1] + 2) * E * s * (X[t].abs() @ P[a].abs().T)
            y[t] += h[t] @ Q[a]
            size[t] += h[t].abs() @ Q[a].abs()
            ey[t] = eh[t] @ Q[a].abs()
        ey += B * (1 + B) * (y.abs() + ey) + (self.r + 2) * E * size
        return h, eh, y, ey

    def grad(self, z, ez, X):
        d = torch.zeros(self.G, self.r, X.shape[1], dtype=F64)
        e = 0 * d
        X = X.to(F64)
        for a in set(self.idx.tolist()):
            if 0 <= a < self.G:
                t = self.rows(a)
                d[a] = z[t].T @ X[t]
                e[a] = ez[t].T @ X[t].abs() + (len(t) + 2) * E * (z[t].abs().T @ X[t].abs())
        return d, e + B * (1 + B) * (d.abs() + e)


def _ok(got, want, lim, what):
    d = (got.cpu().to(F64) - want).abs()
    bad = ~(d <= lim + 1e-37)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst {float((d - lim).max()):.3g}, at {torch.nonzero(bad)[0].tolist()}"


def _forward(c):
    o = ops.lora(c.x_, c.A_, c.B_, c.idx_, c.scale_, base=c.yb_)
    h, eh, y, ey = c.half(c.x, c.A, c.B, c.yb, c.N)
    _ok(o["h"], h, eh, "h")
    _ok(o["y"], y, ey, "y")
    none = ~((c.idx >= 0) & (c.idx < c.G))
    assert torch.equal(o["y"].cpu()[none], c.yb[none] if c.yb is not None else torch.zeros(int(none.sum()), c.N, dtype=BF))
    return o


def _backward(c, h):
    dx, dA, dB = ops.lora_bwd(c.dy_, c.x_, h, c.A_, c.B_, c.idx_, c.scale_, base=c.xb_)
    u, eu, x, ex = c.half(c.dy, c.B, c.A, c.xb, c.K)
    _ok(dx, x, ex, "dx")
    _ok(dA, *c.grad(u, eu, c.x), "dA")
    hh = h.cpu().to(F64)
    _ok(dB, *c.grad(hh, 0 * hh, c.dy), "dB")
    return dx, dA, dB


# ranks around the operand widths (16, 64, 128), widths around the stages (64) and the column tiles (128), rows
# around the few-rows rule and the tiles
@pytest.mark.parametrize("order", ["runs", "rows", "one", "none"])
@pytest.mark.parametrize("T,K,N,r,G", [(1, 8, 8, 8, 1), (2, 2880, 1024, 16, 3), (63, 72, 136, 24, 5), (64, 264, 8, 128, 2),
                                       (65, 64, 128, 16, 40), (127, 1000, 136, 8, 3), (129, 8, 264, 64, 2),
                                       (300, 256, 512, 72, 4), (700, 520, 1048, 128, 3), (1030, 2048, 200, 32, 1),
                                       (513, 136, 72, 112, 70)])
def test_forward_and_backward(order, T, K, N, r, G):
    c = Case(T, K, N, r, G, order, seed=T + r, base=(T + r) % 3 != 0)
    o = _forward(c)
    _backward(c, o["h"])


def test_wide():
    c = Case(400, 7168, 7168, 16, 6, "runs", seed=1)
    _backward(c, _forward(c)["h"])
    c = Case(80, 7168, 2880, 64, 64, "rows", seed=2)
    _backward(c, _forward(c)["h"])


def test_many_adapters():
    # the largest count (the grouping runs on one warp), and one on either side of where a warp drops out
    for G in (32767, 1023, 1024):
        c = Case(500, 16, 24, 8, G, "rows", seed=G)
        o = _forward(c)
        dx, dA, dB = ops.lora_bwd(c.dy_, c.x_, o["h"], c.A_, c.B_, c.idx_, c.scale_)
        used = torch.zeros(G, dtype=torch.bool)
        used[c.idx[(c.idx >= 0)].long()] = True
        assert not bool(dA.cpu()[~used].any()) and not bool(dB.cpu()[~used].any())
        hh = o["h"].cpu().to(F64)
        _ok(dB, *c.grad(hh, 0 * hh, c.dy), "dB")


@pytest.mark.parametrize("T", [5, 200])
def test_in_place_and_neighbours(T):
    c = Case(T, 136, 264, 16, 3, "runs", seed=4)
    o = _forward(c)
    back = _backward(c, o["h"])

    def inside(like, fill):  # a buffer with 64 guard elements on either side
        full = torch.full((like.numel() + 128,), 3.0, dtype=BF, device=DEV)
        v = full[64:-64].view(like.shape)
        if fill is not None:
            v.copy_(fill)
        return full, v

    guards = lambda full: bool((full[:64] == 3).all()) and bool((full[-64:] == 3).all())
    full, v = inside(o["y"], c.yb_)
    if c.yb_ is not None:
        r = ops.lora(c.x_, c.A_, c.B_, c.idx_, c.scale_, base=v, out=v, with_h=False)
        assert r["y"].data_ptr() == v.data_ptr() and "h" not in r and torch.equal(v, o["y"]) and guards(full)
        full, v = inside(back[0], c.xb_)
        dx, dA, dB = ops.lora_bwd(c.dy_, c.x_, o["h"], c.A_, c.B_, c.idx_, c.scale_, base=v, out=v)
        assert torch.equal(v, back[0]) and torch.equal(dA, back[1]) and torch.equal(dB, back[2]) and guards(full)
    full, v = inside(o["y"], None)
    ops.lora(c.x_, c.A_, c.B_, c.idx_, c.scale_, base=c.yb_, out=v)
    assert torch.equal(v, o["y"]) and guards(full)


@pytest.mark.parametrize("T", [40, 333])
def test_nan_and_infinities_stay_with_their_adapter_and_row(T):
    c = Case(T, 72, 200, 16, 3, "rows", seed=6)
    clean = ops.lora(c.x_, c.A_, c.B_, c.idx_, c.scale_, base=c.yb_)
    A, Bm, x = c.A_.clone(), c.B_.clone(), c.x_.clone()
    A[1, 3, 70] = float("nan")
    Bm[2, 15, 199] = float("inf")
    x[7, 0] = float("-inf")
    got = ops.lora(x, A, Bm, c.idx_, c.scale_, base=c.yb_)
    keep = (c.idx != 1) & (c.idx != 2)
    keep[7] = False
    assert torch.equal(got["y"].cpu()[keep], clean["y"].cpu()[keep])
    assert bool(got["y"].cpu()[c.idx == 1].isnan().all())
    two = (c.idx == 2) & (torch.arange(T) != 7)
    assert torch.equal(got["y"].cpu()[two, :199], clean["y"].cpu()[two, :199])
    assert bool((~got["y"].cpu()[two, 199].isfinite()).all())
    if c.idx[7] == -1:
        assert torch.equal(got["y"].cpu()[7], clean["y"].cpu()[7])
    dx, dA, dB = ops.lora_bwd(c.dy_, x, clean["h"], c.A_, c.B_, c.idx_, c.scale_)
    ref = ops.lora_bwd(c.dy_, c.x_, clean["h"], c.A_, c.B_, c.idx_, c.scale_)
    assert torch.equal(dx, ref[0]) and torch.equal(dB, ref[2])
    others = [a for a in range(3) if a != int(c.idx[7])]
    assert torch.equal(dA[others], ref[1][others])


def test_few_rows_and_many_adapters():
    c = Case(20, 264, 520, 16, 2500, "rows", seed=15)
    o = _forward(c)
    dx, dA, dB = _backward(c, o["h"])
    unused = torch.ones(c.G, dtype=torch.bool)
    unused[c.idx[c.idx >= 0].long()] = False
    assert not bool(dA.cpu()[unused].any()) and not bool(dB.cpu()[unused].any())


def test_empty_batch():
    c = Case(4, 16, 24, 8, 2, "runs")
    z = lambda n: torch.empty(0, n, dtype=BF, device=DEV)
    i = torch.empty(0, dtype=torch.int32, device=DEV)
    o = ops.lora(z(16), c.A_, c.B_, i, c.scale_, base=z(24))
    assert o["y"].shape == (0, 24) and o["h"].shape == (0, 8)
    dx, dA, dB = ops.lora_bwd(z(24), z(16), z(8), c.A_, c.B_, i, c.scale_)
    assert dx.shape == (0, 16) and not bool(dA.any()) and not bool(dB.any())


@pytest.mark.parametrize("T", [30, 900])
def test_gradients_against_differences(T):
    # y is linear in x, in A and in B: a difference over a whole step of size 1 is the derivative.  Its error is that of
    # the two forwards' outputs times |dy|, the gradient's its own tolerance times the direction.
    c = Case(T, 64, 72, 16, 3, "runs", seed=9, base=False)
    o = ops.lora(c.x_, c.A_, c.B_, c.idx_, c.scale_)
    dx, dA, dB = ops.lora_bwd(c.dy_, c.x_, o["h"], c.A_, c.B_, c.idx_, c.scale_)
    g = torch.Generator().manual_seed(1)
    dy = c.dy.to(F64)
    err0 = c.half(c.x, c.A, c.B, None, c.N)[3]
    for name, grad in (("x", dx), ("A", dA), ("B", dB)):
        old = getattr(c, name)
        new = (old.float() + torch.randn(old.shape, generator=g) * float(old.float().std())).to(BF)
        direction = new.to(F64) - old.to(F64)
        args = {"x": c.x, "A": c.A, "B": c.B, name: new}
        y = ops.lora(*(args[k].to(DEV) for k in ("x", "A", "B")), c.idx_, c.scale_)["y"].cpu().to(F64)
        diff = ((y - o["y"].cpu().to(F64)) * dy).sum()
        lim = ((err0 + c.half(args["x"], args["A"], args["B"], None, c.N)[3]) * dy.abs()).sum()
        u, eu, x, ex = c.half(c.dy, c.B, c.A, None, c.K)
        hh, eh = c.half(c.x, c.A, c.B, None, c.N)[:2]
        e = {"x": ex, "A": c.grad(u, eu, c.x)[1], "B": c.grad(hh, eh, c.dy)[1]}[name]
        lim += (e * direction.abs()).sum()
        got = (grad.cpu().to(F64) * direction).sum()
        assert abs(float(got - diff)) <= float(lim), (name, float(got), float(diff), float(lim))


@pytest.mark.parametrize("T", [48, 400])
def test_captured_on_other_streams_and_the_same_bits(T):
    c = Case(T, 264, 136, 24, 5, "runs", seed=11)
    want = ops.lora(c.x_, c.A_, c.B_, c.idx_, c.scale_, base=c.yb_)
    grads = ops.lora_bwd(c.dy_, c.x_, want["h"], c.A_, c.B_, c.idx_, c.scale_, base=c.xb_)

    def both():
        o = ops.lora(c.x_, c.A_, c.B_, c.idx_, c.scale_, base=c.yb_)
        return [o["y"], o["h"], *ops.lora_bwd(c.dy_, c.x_, o["h"], c.A_, c.B_, c.idx_, c.scale_, base=c.xb_)]

    wanted = [want["y"], want["h"], *grads]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = both()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            cap = both()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, wanted))
    # new rows and another grouping in the captured buffers
    c2 = Case(T, 264, 136, 24, 5, "rows", seed=12)
    for k in ("x_", "dy_", "idx_", "yb_", "xb_"):
        if getattr(c, k) is not None:
            getattr(c, k).copy_(getattr(c2, k))
    g.replay()
    torch.cuda.synchronize()
    again = both()
    assert all(torch.equal(a, b) for a, b in zip(cap, again))
    # two calls at once, each with its own workspace
    s2 = torch.cuda.Stream()
    s2.wait_stream(torch.cuda.current_stream())
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        with torch.cuda.stream(s):
            a = both()
        with torch.cuda.stream(s2):
            b = both()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(a, again)) and all(torch.equal(x, y) for x, y in zip(b, again))


def test_offsets_past_32_bits():
    T, K = 600_000, 7168  # 4.3e9 elements
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("40 GB of free device memory are needed")
    c = Case(200, K, 64, 8, 2, "runs", seed=13, base=False)
    x = torch.zeros(T, K, dtype=BF, device=DEV)
    x[-200:] = c.x_
    idx = torch.full((T,), -1, dtype=torch.int32, device=DEV)
    idx[-200:] = c.idx_
    o = ops.lora(x, c.A_, c.B_, idx, c.scale_)
    h, eh, y, ey = c.half(c.x, c.A, c.B, None, c.N)
    _ok(o["h"][-200:], h, eh, "h")
    _ok(o["y"][-200:], y, ey, "y")
    assert not bool(o["y"][:-200].any()) and not bool(o["h"][:-200].any())
    dy = torch.zeros(T, 64, dtype=BF, device=DEV)
    dy[-200:] = c.dy_
    dx, dA, dB = ops.lora_bwd(dy, x, o["h"], c.A_, c.B_, idx, c.scale_)
    u, eu, xg, ex = c.half(c.dy, c.B, c.A, None, c.K)
    _ok(dx[-200:], xg, ex, "dx")
    _ok(dA, *c.grad(u, eu, c.x), "dA")
    assert not bool(dx[:1000].any())
    del x, dx
    torch.cuda.empty_cache()


@pytest.mark.parametrize("T,r", [(76, 16), (77, 16), (256, 16), (257, 16), (128, 32), (129, 32), (256, 8), (3, 128), (8, 8),
                                 (9, 16), (9, 24), (10, 72), (32, 128), (33, 64), (34, 40), (64, 64), (64, 72), (65, 16)])
def test_around_the_few_rows_rule(T, r):
    c = Case(T, 136, 264, r, 5, "rows", seed=T)
    _backward(c, _forward(c)["h"])


def test_whatever_the_workspace_held():
    c = Case(700, 264, 520, 40, 6, "runs", seed=14)
    want = _forward(c)
    back = ops.lora_bwd(c.dy_, c.x_, want["h"], c.A_, c.B_, c.idx_, c.scale_, base=c.xb_)
    lib, p = L.load(), lambda t: None if t is None else t.data_ptr()
    stream = torch.cuda.current_stream().cuda_stream
    n, nb = lib.moe_lora_fwd_workspace_size(700, 40, 6), lib.moe_lora_bwd_workspace_size(700, 40, 6)
    for fill in (0, 0x7F, 0xFF):
        y, h = torch.empty_like(want["y"]), torch.empty_like(want["h"])
        ws = torch.full((max(n, nb) + 512,), fill, dtype=torch.uint8, device=DEV)
        assert lib.moe_lora_fwd(p(c.x_), p(c.A_), p(c.B_), p(c.idx_), p(c.scale_), p(c.yb_), 700, 264, 520, 40, 6, p(y), p(h),
                                p(ws), n, None, stream) == L.MOE_OK
        assert torch.equal(y, want["y"]) and torch.equal(h, want["h"]) and bool((ws[n:] == fill).all())
        ws.fill_(fill)
        out = [torch.empty_like(t) for t in back]
        assert lib.moe_lora_bwd(p(c.dy_), p(c.x_), p(h), p(c.A_), p(c.B_), p(c.idx_), p(c.scale_), p(c.xb_), 700, 264, 520, 40, 6,
                                *map(p, out), p(ws), nb, None, stream) == L.MOE_OK
        assert all(torch.equal(a, b) for a, b in zip(out, back)) and bool((ws[nb:] == fill).all())


def test_refusals():
    c = Case(10, 16, 24, 8, 2, "runs")
    f = lambda **k: ops.lora(**{"x": c.x_, "A": c.A_, "B": c.B_, "idx": c.idx_, "scale": c.scale_, **k})
    f()
    for kw in (dict(x=c.x), dict(x=c.x_.float()), dict(x=c.x_[:, ::2]), dict(A=c.A_[0]), dict(A=c.A_[:1]), dict(A=c.A_[..., :8]),
               dict(idx=c.idx_.long()), dict(idx=c.idx_[:5]), dict(scale=c.scale_.to(BF)), dict(scale=c.scale_[:1]),
               dict(base=c.x_), dict(out=c.x_), dict(base=torch.zeros(10, 24, device=DEV))):
        with pytest.raises(ValueError):
            f(**kw)
    b = lambda **k: ops.lora_bwd(**{"dy": c.dy_, "x": c.x_, "h": torch.zeros(10, 8, dtype=BF, device=DEV), "A": c.A_,
                                    "B": c.B_, "idx": c.idx_, "scale": c.scale_, **k})
    b()
    for kw in (dict(dy=c.x_), dict(h=c.x_), dict(base=c.dy_), dict(out=c.dy_)):
        with pytest.raises(ValueError):
            b(**kw)
    # outputs over inputs
    buf = torch.zeros(10 * 24 + 64, dtype=BF, device=DEV)
    with pytest.raises(L.MoeError):
        f(base=buf[:240].view(10, 24), out=buf[8:248].view(10, 24))
    sq = Case(10, 16, 16, 8, 2, "runs")
    with pytest.raises(L.MoeError):
        ops.lora(sq.x_, sq.A_, sq.B_, sq.idx_, sq.scale_, out=sq.x_)
    with pytest.raises(L.MoeError):
        ops.lora_bwd(sq.dy_, sq.x_, torch.zeros(10, 8, dtype=BF, device=DEV), sq.A_, sq.B_, sq.idx_, sq.scale_, out=sq.dy_)
