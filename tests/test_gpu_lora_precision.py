"""The adapters' products from h and u in more bits than they are returned in:
what comes out is off by its own rounding and by sums in fp32, on both sides of
every rule that chooses a kernel.

Bounds (e = 2^-23, b = 2^-8 as in test_gpu_lora.py): h and u enter the products
behind them with at least 16 bits, off by 2^-17 at most, and by their own sums,
(K + 2) e scale sum |A x|.  Two parts of h double the terms of the sum over the
rank, (2 r + 2) e (sum |B h| + |base|), and of the sum over n rows.  The base
that is added cancels most of the product, so that an h rounded to bf16 shows.
"""
import pytest
import torch

from test_gpu_lora import B, BF, DEV, E, F64, Case, _ok

from grouped_gemm_glu_gb300 import ops

pytestmark = pytest.mark.gpu


def _product(X, P, Q, idx, scale, width):
    """(h, its error, h Q, its error) in float64, without a base."""
    X, P, Q = X.to(F64), P.to(F64), Q.to(F64)
    r = P.shape[1]
    h, eh = torch.zeros(X.shape[0], r, dtype=F64), torch.zeros(X.shape[0], r, dtype=F64)
    y, ey = torch.zeros(X.shape[0], width, dtype=F64), torch.zeros(X.shape[0], width, dtype=F64)
    for a in set(idx.tolist()):
        if 0 <= a < P.shape[0]:
            t, s = torch.nonzero(idx == a).view(-1), float(scale[a])
            h[t] = s * (X[t] @ P[a].T)
            eh[t] = 2.0 ** -17 * h[t].abs() + (X.shape[1] + 2) * E * s * (X[t].abs() @ P[a].abs().T)
            y[t] = h[t] @ Q[a]
            ey[t] = eh[t] @ Q[a].abs() + (2 * r + 2) * E * 2 * (h[t].abs() @ Q[a].abs())
    return h, eh, y, ey


SHAPES = [(40, 264, 520, 16, 5), (130, 136, 264, 64, 3), (300, 256, 512, 8, 4), (700, 520, 1048, 16, 3), (513, 136, 264, 32, 2),
          (520, 264, 136, 48, 3), (700, 264, 520, 64, 3), (600, 136, 264, 72, 2), (700, 520, 264, 128, 3)]


@pytest.mark.parametrize("order", ["rows", "runs"])
@pytest.mark.parametrize("T,K,N,r,G", SHAPES)
def test_outputs_next_to_a_base_that_cancels(T, K, N, r, G, order):
    c = Case(T, K, N, r, G, order, seed=T + r)
    for X, P, Q, width, call in (
            (c.x, c.A, c.B, N, lambda base: ops.lora(c.x_, c.A_, c.B_, c.idx_, c.scale_, base=base)["y"]),
            (c.dy, c.B, c.A, K, lambda base: ops.lora_bwd(c.dy_, c.x_, torch.zeros(T, r, dtype=BF, device=DEV), c.A_, c.B_, c.idx_,
                                                          c.scale_, base=base)[0])):
        h, _, y, ey = _product(X, P, Q, c.idx, c.scale, width)
        base = (-y).to(BF)
        want = base.to(F64) + y
        lim = ey + B * (1 + B) * (want.abs() + ey) + (2 * r + 2) * E * base.to(F64).abs()
        _ok(call(base.to(DEV)), want, lim, "y" if width == N else "dx")


# Whole numbers: every product and every sum below 2^24 is exact in fp32, so that each output is the exact value's one
# rounding.  h and u reach some 2000 (11 bits; bf16 holds 8), their sums over the rank or the rows stay below 2^22.
@pytest.mark.parametrize("order", ["rows", "runs", "one"])
@pytest.mark.parametrize("T,K,N,r,G", SHAPES + [(20, 264, 136, 24, 3), (64, 264, 264, 64, 40), (2000, 264, 264, 16, 3)])
def test_whole_numbers_are_rounded_once(T, K, N, r, G, order):
    c = Case(T, K, N, r, G, order)
    g = torch.Generator().manual_seed(T + r)
    ints = lambda *s, most=7: torch.randint(-most, most + 1, s, generator=g).to(BF)
    x, dy, A, Bm = ints(T, K), ints(T, N), ints(G, r, K), ints(G, r, N)
    yb, xb, scale = ints(T, N, most=256), ints(T, K, most=256), torch.tensor([1.0, 0.5, -2.0, 1.0])[torch.arange(G) % 4]
    x64, dy64, A64, B64 = (v.to(F64) for v in (x, dy, A, Bm))
    h, u = torch.zeros(T, r, dtype=F64), torch.zeros(T, r, dtype=F64)
    y, dx = yb.to(F64).clone(), xb.to(F64).clone()
    dA, dB = torch.zeros(G, r, K, dtype=F64), torch.zeros(G, r, N, dtype=F64)
    most = 0.0  # of any sum's terms, by size
    for a in range(G):
        t = c.rows(a)
        h[t], u[t] = float(scale[a]) * (x64[t] @ A64[a].T), float(scale[a]) * (dy64[t] @ B64[a].T)
        y[t] += h[t] @ B64[a]
        dx[t] += u[t] @ A64[a]
        dA[a] = u[t].T @ x64[t]
        dB[a] = h[t].to(BF).to(F64).T @ dy64[t]
        if len(t):
            most = max(most, float((h[t].abs() @ B64[a].abs()).max()) + 256, float((u[t].abs() @ A64[a].abs()).max()) + 256,
                       float((u[t].abs().T @ x64[t].abs()).max()), float((h[t].abs().T @ dy64[t].abs()).max()))
    assert most < 2 ** 23 and float(u.abs().max()) > 256  # (halves: one bit more)
    d = lambda *v: [t.to(DEV) for t in v]
    x_, A_, B_, s_, yb_, dy_, xb_ = d(x, A, Bm, scale, yb, dy, xb)
    o = ops.lora(x_, A_, B_, c.idx_, s_, base=yb_)
    assert torch.equal(o["h"].cpu(), h.to(BF)) and torch.equal(o["y"].cpu(), y.to(BF))
    got = ops.lora_bwd(dy_, x_, o["h"], A_, B_, c.idx_, s_, base=xb_)
    for name, v, want in zip(("dx", "dA", "dB"), got, (dx, dA, dB)):
        assert torch.equal(v.cpu(), want.to(BF)), name
