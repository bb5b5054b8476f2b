"""GPU parity of the residual RMS norm (forward, backward, MXFP8 rows) against
the formulas in float64.

Tolerances, from the arithmetic (u = 2^-24, fp32 unit roundoff; a bf16 result
is within 2^-8 of its magnitude of the value rounded):
  * h is one fp32 addition rounded to bf16: exact against the same two
    roundings;
  * the sum of squares adds H positive terms in chains of at most 32 plus 15
    tree levels: relative error below 64 u, so rstd (a square root and a
    division later) stays within 64 u;
  * y adds two products: |err| <= 2^-8 |y| (1 + 2^-9) for bf16; its MXFP8
    codes may land one step apart where y falls within 80 u of a rounding
    boundary;
  * dx: the dot product's error is below 64 u sum |t h|, and every other
    operation rounds once, so |err| <= 2^-8 |dx| + 96 u (r |t| + r |h| r^2
    mean|t h| + |dres|), taken as 2^-8 |dx| (1 + 2^-9) + 2^-17 (...);
  * dgamma sums T terms in fp32: |err| <= (T + 32) u sum |dy h r|.
"""
import numpy as np
import pytest
import torch

from grouped_gemm_glu_gb300 import lib as L
from grouped_gemm_glu_gb300 import ops
from oracle import moe_oracle as O
from parity import assert_mx_close, np_

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24


def _bf(rng, *shape, scale=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).to(torch.bfloat16)


def _bf16_ok(got, ref, extra=0.0):
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    lim = 2.0 ** -8 * np.abs(ref) * (1 + 2.0 ** -9) + extra + 1e-37
    bad = np.abs(got - ref) > lim
    assert not bad.any(), f"{bad.sum()} of {bad.size} outside, worst {np.max(np.abs(got - ref) - lim):.3g}"


# widths around a warp's 256 columns, odd multiples of 8, more than one vector
# a thread, the largest; tokens around the few-rows rule and the CTA's rows
@pytest.mark.parametrize("T,H", [(1, 8), (3, 248), (1, 2880), (257, 256), (300, 520), (9, 16384), (300, 8200),
                                 (513, 1032), (700, 2880), (1300, 96), (260, 7168)])
@pytest.mark.parametrize("residual", [True, False])
def test_forward(T, H, residual):
    rng = np.random.default_rng(T * 31 + H)
    x, g = _bf(rng, T, H, scale=0.7), _bf(rng, H)
    r = _bf(rng, T, H, scale=3.0) if residual else None
    x[0, :8] = 0
    if T > 2:
        x[2] = 0  # an all-zero row (with the residual: zeros too) has y = 0
        if residual:
            r[2] = 0
    mx = H % 32 == 0
    o = ops.rmsnorm(x.to(DEV), g.to(DEV), 1e-5, residual=None if r is None else r.to(DEV), mxfp8=mx)
    h = x if r is None else (x.float() + r.float()).to(torch.bfloat16)
    if residual:
        assert torch.equal(o["h"].cpu(), h)
    else:
        assert "h" not in o
    h = np_(h)
    rs = 1.0 / np.sqrt((h * h).mean(1) + np.float64(np.float32(1e-5)))
    assert np.all(np.abs(np_(o["rstd"]) - rs) <= 64 * U * rs)
    y = h * rs[:, None] * np_(g)
    _bf16_ok(np_(o["y"]), y)
    if mx:
        y32 = y.astype(np.float32)
        q, s = O.mx_quantize_rows(y32)
        assert_mx_close(np_(o["q"]), np_(o["s"]), q, s, y32, "MXFP8 rows", rel_band=1e-5)
        only = ops.rmsnorm(x.to(DEV), g.to(DEV), 1e-5, residual=None if r is None else r.to(DEV), bf16=False,
                           mxfp8=True, with_rstd=False)
        assert torch.equal(only["q"], o["q"]) and torch.equal(only["s"], o["s"]) and "y" not in only
        v = ops.dequantize_mxfp8(o["q"], o["s"])
        want = O.mx_dequantize(np_(o["q"]), np_(o["s"]))
        assert np.array_equal(np_(v), want.reshape(T, H))


@pytest.mark.parametrize("T,H", [(1, 8), (1, 2880), (2, 16384), (255, 248), (257, 264), (300, 520), (700, 2880),
                                 (1500, 96), (2600, 7168), (300, 8200)])
@pytest.mark.parametrize("dres", [True, False])
def test_backward(T, H, dres):
    rng = np.random.default_rng(T * 17 + H)
    h, dy, g = _bf(rng, T, H, scale=2.0), _bf(rng, T, H), _bf(rng, H)
    e = _bf(rng, T, H) if dres else None
    rstd = (1.0 / np.sqrt((np_(h) ** 2).mean(1) + 1e-5)).astype(np.float32)
    args = (dy.to(DEV), h.to(DEV), g.to(DEV), torch.from_numpy(rstd).to(DEV))
    ed = e.to(DEV) if dres else None
    dx, dg = ops.rmsnorm_bwd(*args, dres=ed)
    dy64, h64, g64, r = np_(dy), np_(h), np_(g), rstd.astype(np.float64)[:, None]
    t = dy64 * g64
    dot = (t * h64).mean(1, keepdims=True)
    ref = r * (t - h64 * r * r * dot)
    mag = r * (np.abs(t) + np.abs(h64) * r * r * np.abs(t * h64).mean(1, keepdims=True))
    if dres:
        ref = ref + np_(e)
        mag = mag + np.abs(np_(e))
    _bf16_ok(np_(dx), ref, 2.0 ** -17 * mag)
    term = dy64 * h64 * r
    assert np.all(np.abs(np_(dg) - term.sum(0)) <= (T + 32) * U * np.abs(term).sum(0) + 1e-37)
    # the same bits again, without dgamma, and written over dy
    dx2, dg2 = ops.rmsnorm_bwd(*args, dres=ed)
    assert torch.equal(dx, dx2) and torch.equal(dg, dg2)
    dx3, none = ops.rmsnorm_bwd(*args, dres=ed, with_dgamma=False)
    assert none is None and torch.equal(dx, dx3)


def test_backward_matches_differences():
    """<dx, v> and <dgamma, w> against central differences of the float64
    forward.  The difference's own error at step 1e-5 is ~1e-9 of the loss's
    scale; dx carries bf16 rounding, 2^-8 sum |dx v|."""
    rng = np.random.default_rng(3)
    T, H = 5, 96
    h, dy, g = _bf(rng, T, H), _bf(rng, T, H), _bf(rng, H)
    rstd = (1.0 / np.sqrt((np_(h) ** 2).mean(1) + 1e-5)).astype(np.float32)
    dx, dg = ops.rmsnorm_bwd(dy.to(DEV), h.to(DEV), g.to(DEV), torch.from_numpy(rstd).to(DEV))

    def loss(hh, gg):
        return float((np_(dy) * hh * gg / np.sqrt((hh * hh).mean(1, keepdims=True) + 1e-5)).sum())

    for k in range(4):
        v, w = rng.standard_normal((T, H)), rng.standard_normal(H)
        d = 1e-5
        num = (loss(np_(h) + d * v, np_(g)) - loss(np_(h) - d * v, np_(g))) / (2 * d)
        assert abs(num - float((np_(dx) * v).sum())) <= 2.0 ** -8 * float(np.abs(np_(dx) * v).sum()) + 1e-5
        num = (loss(np_(h), np_(g) + d * w) - loss(np_(h), np_(g) - d * w)) / (2 * d)
        assert abs(num - float((np_(dg) * w).sum())) <= 1e-5 * float(np.abs(np_(dg) * w).sum()) + 1e-5


def test_nonfinite_and_large_values():
    """A row with a NaN (or Inf) is NaN where the formula is, its MXFP8 blocks
    are NaN blocks, and no other row sees it; values near bf16's largest
    overflow the sum of squares to rstd = 0 as the fp32 formula does."""
    H = 320
    x = torch.ones(4, H, dtype=torch.bfloat16)
    x[1, 5] = float("nan")
    x[2, 7] = float("inf")
    x[3] = 1e30
    o = ops.rmsnorm(x.to(DEV), torch.ones(H, dtype=torch.bfloat16, device=DEV), 0.0, mxfp8=True)
    y = np_(o["y"])
    assert np.all(y[0] == 1.0) and np.all(np.isnan(y[1])) and np.all(y[3] == 0.0)
    assert np.isnan(y[2, 7]) and np.all(np.delete(y[2], 7) == 0.0)
    s = np_(o["s"])
    assert np.all(s[1] == 0xFF) and s[2, 0] == 0xFF and np.all(s[2, 1:] == 0) and np.all(s[0] == 119)
    assert np.all(np.isnan(np_(ops.dequantize_mxfp8(o["q"], o["s"]))[1]))


def test_side_stream_and_empty_batch():
    rng = np.random.default_rng(5)
    x, g = _bf(rng, 64, 256).to(DEV), _bf(rng, 256).to(DEV)
    want = ops.rmsnorm(x, g, mxfp8=True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = ops.rmsnorm(x, g, mxfp8=True)
    s.synchronize()
    for k in want:
        assert torch.equal(want[k], got[k])
    e = ops.rmsnorm(x[:0], g, residual=x[:0], mxfp8=True)
    assert e["y"].shape == (0, 256) and e["s"].shape == (0, 8)
    dx, dg = ops.rmsnorm_bwd(x[:0], x[:0], g, want["rstd"][:0])
    assert dx.shape == (0, 256) and torch.all(dg == 0)


def test_refusals():
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device=DEV)
    g = torch.ones(64, dtype=torch.bfloat16, device=DEV)
    for bad in (lambda: ops.rmsnorm(x.float(), g), lambda: ops.rmsnorm(x.cpu(), g), lambda: ops.rmsnorm(x, g[:32]),
                lambda: ops.rmsnorm(x.t(), g), lambda: ops.rmsnorm(x, g, residual=x[:2]),
                lambda: ops.rmsnorm_bwd(x, x, g, torch.zeros(4, device=DEV, dtype=torch.float64)),
                lambda: ops.dequantize_mxfp8(x, x)):
        with pytest.raises(ValueError):
            bad()
    y = torch.zeros(4, 40, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(L.MoeError):  # MXFP8 rows need whole blocks of 32
        ops.rmsnorm(y, g[:40].contiguous(), mxfp8=True)
    with pytest.raises(L.MoeError):  # neither output
        ops.rmsnorm(x, g, bf16=False)
    odd = torch.zeros(4 * 64 + 1, dtype=torch.bfloat16, device=DEV)[1:].view(4, 64)
    with pytest.raises(L.MoeError):  # not 16-byte aligned
        ops.rmsnorm(odd, g)
    with pytest.raises(L.MoeError):  # eps < 0
        ops.rmsnorm(x, g, -1.0)


def test_past_32_bits():
    """2.2 billion elements: the last rows are those of a small call."""
    T, H = 270_000, 8192
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.zeros(T, H, dtype=torch.bfloat16, device=DEV)
    x[-300:] = torch.randn(300, H, generator=g, device=DEV).to(torch.bfloat16)
    gm = torch.ones(H, dtype=torch.bfloat16, device=DEV)
    o, w = ops.rmsnorm(x, gm, residual=x, mxfp8=True), ops.rmsnorm(x[-300:], gm, residual=x[-300:], mxfp8=True)
    for k in w:
        assert torch.equal(o[k][-300:], w[k]), k
    v = ops.dequantize_mxfp8(o["q"], o["s"])
    assert torch.equal(v[-300:], ops.dequantize_mxfp8(w["q"], w["s"]))
    del v
    dx, dg = ops.rmsnorm_bwd(x, o["h"], gm, o["rstd"])
    wx, wg = ops.rmsnorm_bwd(x[-300:], w["h"], gm, w["rstd"])
    assert torch.equal(dx[-300:], wx)
    # the rows of zeros add nothing; the order of the sums differs
    assert torch.all((dg - wg).abs() <= 300 * U * (x[-300:].float() * w["h"].float() * w["rstd"][:, None]).abs().sum(0))


@pytest.mark.parametrize("T,H", [(152, 8192), (153, 8192), (173, 7168), (174, 7168), (405, 2880), (406, 2880),
                                 (512, 64), (513, 64)])
def test_both_sides_of_the_few_rows_rule(T, H):
    """The last size that gets a CTA per row and the first that does not: rstd
    within 64 u, y and dx as above, dgamma's sum over either split's lines."""
    rng = np.random.default_rng(T + H)
    x, res, g, dy = _bf(rng, T, H), _bf(rng, T, H), _bf(rng, H), _bf(rng, T, H)
    o = ops.rmsnorm(x.to(DEV), g.to(DEV), residual=res.to(DEV))
    h = (x.float() + res.float()).to(torch.bfloat16)
    assert torch.equal(o["h"].cpu(), h)
    h64, g64, dy64 = np_(h), np_(g), np_(dy)
    r = 1.0 / np.sqrt((h64 ** 2).mean(1) + 1e-5)
    assert np.all(np.abs(np_(o["rstd"]) - r) <= 64 * U * r)
    r = np_(o["rstd"]).astype(np.float64)[:, None]
    _bf16_ok(np_(o["y"]), h64 * r * g64, 128 * U * np.abs(h64 * r * g64))
    dx, dg = ops.rmsnorm_bwd(dy.to(DEV), o["h"], g.to(DEV), o["rstd"])
    t = dy64 * g64
    ref = r * (t - h64 * r * r * (t * h64).mean(1, keepdims=True))
    mag = r * (np.abs(t) + np.abs(h64) * r * r * np.abs(t * h64).mean(1, keepdims=True))
    _bf16_ok(np_(dx), ref, 2.0 ** -17 * mag)
    term = dy64 * h64 * r
    assert np.all(np.abs(np_(dg) - term.sum(0)) <= (T + 32) * U * np.abs(term).sum(0) + 1e-37)
