"""GPU parity of MXFP4 weights: the cast (exact), its read-back (exact) and
the grouped products of MXFP8 rows with MXFP4 weights.

Tolerance of a product, from the arithmetic: the factors and their products
are exact in fp32; the tensor cores add 32 products at a time into an fp32
accumulator, each addition good to 2^-22 of the magnitudes it joins, so the
sum is within (K / 32 + 8) 2^-22 sum |a w| of the exact one, and the bf16
result within 2^-8 of its magnitude of that.  Through the activation the
accumulator's error is multiplied by its slopes, which are below
16 (1 + max |pre-activation|) for every form here."""
import numpy as np
import pytest
import torch

from grouped_gemm_glu_gb300 import lib as L
from grouped_gemm_glu_gb300 import ops, synth
from oracle import moe_oracle as O
from parity import np_

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def mx4_reference(v):
    """(codes [..., K], scale bytes [..., K/32]) of float32 values along the last axis."""
    b = np.asarray(v, np.float32).reshape(*v.shape[:-1], -1, 32).astype(np.float64)
    with np.errstate(invalid="ignore", divide="ignore"):
        amax = np.abs(b).max(-1)
        e = np.where(amax > 0, np.floor(np.log2(np.where(amax > 0, amax, 1.0))) - 2 + 127, 0)
        bad = ~np.isfinite(amax)
        byte = np.where(bad, 255, np.clip(e, 0, 254)).astype(np.int64)
        x = np.where(bad[..., None], 0.0, b * np.exp2(127.0 - np.where(bad, 127, byte))[..., None])
    codes = O.e2m1_encode(x)
    codes = np.where(bad[..., None], 7, codes)
    return codes.reshape(v.shape).astype(np.uint8), byte.astype(np.uint8)


def unpack(q, K):
    q = np.asarray(q)[..., : K // 2]
    return np.stack([q & 15, q >> 4], -1).reshape(*q.shape[:-1], K)


def untile(s, G, N, K):
    nt, kb = (N + 255) // 256, (K + 127) // 128
    t = np.asarray(s).reshape(G, nt, kb, 2, 32, 4, 4).transpose(0, 1, 3, 5, 4, 2, 6).reshape(G, nt * 256, kb * 4)
    return t


@pytest.mark.parametrize("G,R,C", [(1, 32, 32), (2, 96, 160), (3, 128, 256), (1, 288, 2880), (2, 2880, 96), (5, 416, 352)])
@pytest.mark.parametrize("col", [False, True])
def test_cast_and_read_back(G, R, C, col):
    rng = np.random.default_rng(G * 7 + R + C)
    x = (rng.standard_normal((G, R, C)) * np.exp2(rng.integers(-6, 6, (G, R, 1)))).astype(np.float32)
    x[0, :, 1] = 0                      # zero elements, and (rows) whole zero blocks below
    x[0, 3, :32] = 0
    x[0, :32, 5] = 0
    src = torch.from_numpy(x).to(torch.bfloat16)
    v = np_(src)
    if col:
        v = v.transpose(0, 2, 1)
    N, K = v.shape[1:]
    q, s = ops.quantize_mxfp4(src.to(DEV), col=col)
    codes, byte = mx4_reference(v)
    got = unpack(np_(q), K)
    zero = (got & 7) == 0               # +0 and -0 stand for the same value
    assert np.array_equal(np.where(zero, 0, got), np.where((codes & 7) == 0, 0, codes))
    t = untile(np_(s), G, N, K)
    assert np.array_equal(t[:, :N, : K // 32], byte)
    assert not t[:, N:].any() and not t[:, :, K // 32:].any()
    assert not np_(q)[..., K // 2:].any()
    back = np_(ops.dequantize_mxfp4(q, s, K))
    want = O.e2m1_decode(codes).reshape(G, N, K // 32, 32) * np.exp2(byte.astype(np.float64) - 127)[..., None]
    assert np.array_equal(back, want.reshape(G, N, K))


def test_cast_extremes():
    """Ties, saturation, the smallest and largest scales, and blocks that hold
    NaN or Inf."""
    x = np.zeros((1, 32, 64), np.float32)
    x[0, 0, :8] = [4.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]      # ties at scale 1
    x[0, 1, :4] = [7.75, -7.75, 6.5, 1.0]                             # above 6: saturates
    x[0, 2, :2] = [2.0 ** -126, 2.0 ** -127]                          # clamped scale
    x[0, 3, :2] = [3.3e38, 1e38]
    x[0, 4, 3] = np.nan
    x[0, 5, 40] = np.inf
    x[0, 6, :2] = [-0.0, 2.0 ** -133]
    src = torch.from_numpy(x).to(torch.bfloat16)
    q, s = ops.quantize_mxfp4(src.to(DEV))
    codes, byte = mx4_reference(np_(src))
    got = unpack(np_(q), 64)
    assert np.array_equal(untile(np_(s), 1, 32, 64)[:, :32, :2], byte)
    zero = (got & 7) == 0
    assert np.array_equal(np.where(zero, 0, got), np.where((codes & 7) == 0, 0, codes))
    back = np_(ops.dequantize_mxfp4(q, s, 64))
    assert np.isnan(back[0, 4, :32]).all() and np.isnan(back[0, 5, 32:]).all() and not np.isnan(back[0, 5, :32]).any()


def _rows(rng, counts, K):
    """Rows of experts with these counts: (xq, xs, counts, offsets, values, R_cap)."""
    off = np.concatenate([[0], np.cumsum((np.asarray(counts) + 31) // 32 * 32)])
    cap = max(128, (int(off[-1]) + 127) // 128 * 128)
    x = np.zeros((cap, K), np.float32)
    for e, c in enumerate(counts):
        x[off[e]:off[e] + c] = rng.standard_normal((c, K))
    q, s = O.mx_quantize_rows(x)
    val = O.mx_dequantize(q, s)
    # whatever lies in rows past the counts must not matter: garbage codes there
    pad = np.ones(cap, bool)
    for e, c in enumerate(counts):
        pad[off[e]:off[e] + c] = False
    q[pad] = 0x7F
    s[pad] = 0xFF
    t = lambda a, dt=torch.uint8: torch.from_numpy(np.ascontiguousarray(a)).to(dt).to(DEV)
    return t(q), t(s), t(counts, torch.int32), t(off, torch.int32), val, cap


def _weight(rng, E, N, K):
    w = torch.from_numpy((rng.standard_normal((E, N, K)) * K ** -0.5).astype(np.float32)).to(torch.bfloat16)
    q, s = ops.quantize_mxfp4(w.to(DEV))
    codes, byte = mx4_reference(np_(w))
    val = O.e2m1_decode(codes).reshape(E, N, K // 32, 32) * np.exp2(byte.astype(np.float64) - 127)[..., None]
    return q, s, val.reshape(E, N, K)


SHAPES = [
    # counts, K, N
    ([1], 32, 32),
    ([0, 3, 0, 1], 256, 96),
    ([1, 0, 1, 1, 0, 1], 2880, 576),
    ([5, 33, 0, 64], 160, 288),
    ([130, 1, 300], 416, 544),
    ([0, 0], 128, 64),
    ([7, 8, 9, 15, 16, 17], 1024, 352),
    ([600, 20], 96, 1056),
]


@pytest.mark.parametrize("counts,K,N", SHAPES)
def test_product(counts, K, N):
    rng = np.random.default_rng(K + N)
    xq, xs, cnt, off, xv, cap = _rows(rng, counts, K)
    q, s, wv = _weight(rng, len(counts), N, K)
    out = torch.full((cap, N), 77.0, dtype=torch.bfloat16, device=DEV)
    st = ops.new_status(DEV)
    ops.fc2_fwd_mxfp4(xq, xs, q, s, cnt, off, status=st, out=out)
    assert ops.read_status(st) == 0
    y, o = np_(out), np_(off)
    for e, c in enumerate(counts):
        r0 = o[e]
        ref = xv[r0:r0 + c] @ wv[e].T
        mag = np.abs(xv[r0:r0 + c]) @ np.abs(wv[e]).T
        lim = 2.0 ** -8 * np.abs(ref) + (K / 32 + 8) * 2.0 ** -22 * mag + 1e-30
        assert np.all(np.abs(y[r0:r0 + c] - ref) <= lim), (e, np.abs(y[r0:r0 + c] - ref).max())
        assert np.all(y[r0 + c:o[e + 1]] == 0)          # pad rows
    assert np.all(y[o[-1]:] == 77.0)                      # rows past the segments untouched
    again = ops.fc2_fwd_mxfp4(xq, xs, q, s, cnt, off)
    assert torch.equal(again[:o[-1]], out[:o[-1]])


@pytest.mark.parametrize("counts,K,F", [([1], 32, 32), ([1, 0, 1, 1, 0, 1], 2880, 288), ([5, 33, 0, 64], 160, 160),
                                        ([130, 1, 300], 416, 544), ([9, 0, 17], 512, 96)])
@pytest.mark.parametrize("act", ["gptoss", "swiglu", "geglu", "srelu"])
def test_up_projection_with_activation(counts, K, F, act):
    rng = np.random.default_rng(K + F)
    E = len(counts)
    gated = act != "srelu"
    N = 2 * F if gated else F
    prm = L.glu_params("swiglu", alpha=1.702, up_offset=1.0, gate_lo=-7.0, gate_hi=7.0) if act == "gptoss" else \
        L.glu_params(act)
    op = {"gptoss": O.ActParams(O.ACT_SWIGLU, alpha=1.702, up_offset=1.0, gate_lo=-7.0, gate_hi=7.0),
          "swiglu": O.ActParams(O.ACT_SWIGLU), "geglu": O.ActParams(O.ACT_GEGLU),
          "srelu": O.ActParams(O.ACT_SRELU)}[act]
    xq, xs, cnt, off, xv, cap = _rows(rng, counts, K)
    q, s, wv = _weight(rng, E, N, K)
    bias = synth._bf16(0.3 * rng.standard_normal((E, N)))
    bd = bias.to(DEV) if act in ("gptoss", "srelu") else None
    scale = torch.from_numpy(rng.random(cap).astype(np.float32)).to(DEV) if act == "geglu" else None
    o = ops.fc1_fwd_mxfp4(xq, xs, q, s, cnt, off, F, prm, out_mode=L.OUT_BF16, b1p=bd, row_scale=scale)
    m = ops.fc1_fwd_mxfp4(xq, xs, q, s, cnt, off, F, prm, out_mode=L.OUT_MXFP8, b1p=bd, row_scale=scale,
                          save_pre=False)
    assert ops.read_status(o["status"]) == 0 and ops.read_status(m["status"]) == 0
    y, pre, of = np_(o["y"]), np_(o["pre"]), np_(off)
    for e, c in enumerate(counts):
        if not c:
            continue
        r = slice(of[e], of[e] + c)
        z = xv[r] @ wv[e].T + (np_(bias)[e] if bd is not None else 0.0)
        mag = np.abs(xv[r]) @ np.abs(wv[e]).T
        lim = 2.0 ** -8 * np.abs(z) + (K / 32 + 8) * 2.0 ** -22 * (mag + np.abs(z)) + 1e-30
        assert np.all(np.abs(pre[r] - z) <= lim)
        if gated:
            u, g = O.unpack_glu_cols(z)
            mu, mg = O.unpack_glu_cols(mag + np.abs(z))
            ref, slack = O.act_fwd(u, g, op), np.maximum(mu, mg)
        else:
            ref, slack = O.act_fwd(z, None, op), mag + np.abs(z)
        if scale is not None:
            ref = ref * np_(scale)[r, None]
        # 2^-20 of the output: the activation's own fp32 arithmetic
        lim = (2.0 ** -8 + 2.0 ** -18) * np.abs(ref) + 16 * (K / 32 + 8) * 2.0 ** -22 * slack * (1 + np.abs(z).max()) + 1e-30
        assert np.all(np.abs(y[r] - ref) <= lim), (e, np.max(np.abs(y[r] - ref) - lim))
        assert np.all(y[of[e] + c:of[e + 1]] == 0)
        d = O.mx_dequantize(np_(m["q_row"])[r], np_(m["s_row"])[r])
        blk = np.abs(ref).reshape(c, -1, 32).max(-1, keepdims=True)
        # a block's step is at most 2^-3 of its largest element (saturation included)
        assert np.all(np.abs(d - ref).reshape(c, -1, 32) <= 0.13 * blk + lim.reshape(c, -1, 32))


def test_side_stream_graph_and_capacity():
    rng = np.random.default_rng(2)
    counts, K, N = [3, 0, 40], 256, 320
    xq, xs, cnt, off, xv, cap = _rows(rng, counts, K)
    q, s, wv = _weight(rng, 3, N, K)
    want = ops.fc2_fwd_mxfp4(xq, xs, q, s, cnt, off)
    end = int(off[-1])
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    status = ops.new_status(DEV)
    with torch.cuda.stream(st):
        got = ops.fc2_fwd_mxfp4(xq, xs, q, s, cnt, off, status=status)
        st.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            cap_out = ops.fc2_fwd_mxfp4(xq, xs, q, s, cnt, off, status=status)
    assert torch.equal(got[:end], want[:end])
    # the captured call follows the counts in device memory
    cnt.copy_(torch.tensor([1, 0, 2], dtype=torch.int32))
    off.copy_(torch.tensor([0, 32, 32, 64], dtype=torch.int32))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(cap_out[:1], want[:1])
    assert not cap_out[1:32].any()
    # more rows than the buffers hold: reported, nothing computed
    off.copy_(torch.tensor([0, 32, 32, cap + 32], dtype=torch.int32))
    cnt.copy_(torch.tensor([1, 0, 2], dtype=torch.int32))
    ops.fc2_fwd_mxfp4(xq, xs, q, s, cnt, off, status=status)
    assert ops.read_status(status) == L.MOE_ERR_CAPACITY


def test_refusals():
    z = torch.zeros(128, 64, dtype=torch.uint8, device=DEV)
    s = torch.zeros(128, 2, dtype=torch.uint8, device=DEV)
    w = torch.zeros(2, 64, 64, dtype=torch.bfloat16, device=DEV)
    q4, s4 = ops.quantize_mxfp4(w)
    c, o = torch.zeros(2, dtype=torch.int32, device=DEV), torch.zeros(3, dtype=torch.int32, device=DEV)
    for bad in (lambda: ops.quantize_mxfp4(w.float()), lambda: ops.quantize_mxfp4(w[0]),
                lambda: ops.dequantize_mxfp4(q4, s4, 256), lambda: ops.dequantize_mxfp4(q4, s4[:-1], 64),
                lambda: ops.fc2_fwd_mxfp4(z, s[:, :1].contiguous(), q4, s4, c, o),
                lambda: ops.fc2_fwd_mxfp4(z, s, q4, s4, c.long(), o), lambda: ops.fc2_fwd_mxfp4(z, s, q4, s4, c, c),
                lambda: ops.fc1_fwd_mxfp4(z, s, q4, s4, c, o, 64, L.glu_params("swiglu"))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(L.MoeError):
        ops.quantize_mxfp4(torch.zeros(1, 48, 64, dtype=torch.bfloat16, device=DEV))
    with pytest.raises(L.MoeError):  # R_cap % 128
        ops.fc2_fwd_mxfp4(z[:64].contiguous(), s[:64].contiguous(), q4, s4, c, o)


@pytest.mark.parametrize("counts,K,N", [([0, 3, 0, 1], 256, 96), ([130, 1, 300], 416, 544), ([40] * 5, 96, 288)])
def test_product_output_forms(counts, K, N):
    """MXFP8 outputs are the fp32 accumulator's (as the bf16 output rounds it),
    row-wise and column-wise; NVFP4 mode is the bf16 output with its amax."""
    rng = np.random.default_rng(K)
    xq, xs, cnt, off, xv, cap = _rows(rng, counts, K)
    q, s, wv = _weight(rng, len(counts), N, K)
    y = np_(ops.fc2_fwd_mxfp4(xq, xs, q, s, cnt, off))
    n4 = ops.fc2_fwd_mxfp4(xq, xs, q, s, cnt, off, out_mode=L.OUT_NVFP4)
    m = ops.fc2_fwd_mxfp4(xq, xs, q, s, cnt, off, out_mode=L.OUT_MXFP8)
    r = ops.fc2_fwd_mxfp4(xq, xs, q, s, cnt, off, out_mode=L.OUT_MXFP8, with_col=False)
    o = np_(off)
    R = int(o[-1])
    assert np.array_equal(np_(n4["y"])[:R], y[:R])
    real = np.concatenate([np.arange(o[e], o[e] + c) for e, c in enumerate(counts)])
    ref = np.zeros((R, N))
    for e, c in enumerate(counts):
        ref[o[e]:o[e] + c] = xv[o[e]:o[e] + c] @ wv[e].T
    # the largest magnitude, within the accumulator's error and (nothing) of rounding
    a = float(n4["amax"])
    assert abs(a - np.abs(ref).max()) <= (K / 32 + 8) * 2.0 ** -22 * 8 * np.abs(ref).max()
    assert torch.equal(m["q_row"][:R], r["q_row"][:R]) and torch.equal(m["s_row"][:R], r["s_row"][:R])
    for d in (O.mx_dequantize(np_(m["q_row"])[:R], np_(m["s_row"])[:R]),
              O.mx_dequantize(np_(m["q_col"])[:, :R].copy(), np_(m["s_col"])[:, :R // 32].copy()).T):
        # a step of E4M3 at a value is 2^-3 of it, and a block's smallest steps are 2^-9 2^-8 of its largest element
        blk = np.abs(ref).max()
        assert np.all(np.abs(d - ref)[real] <= 0.13 * np.abs(ref)[real] + 2.0 ** -16 * blk + 0.13 * 2.0 ** -3 * blk * (np.abs(ref)[real] < 2.0 ** -6 * blk))
        assert np.all(np.delete(d, real, axis=0) == 0)


def test_many_experts():
    """E = 1000 experts with 0 to 3 rows each."""
    rng = np.random.default_rng(8)
    counts = rng.integers(0, 4, 1000).tolist()
    xq, xs, cnt, off, xv, cap = _rows(rng, counts, 64)
    q, s, wv = _weight(rng, 1000, 32, 64)
    y, o = np_(ops.fc2_fwd_mxfp4(xq, xs, q, s, cnt, off)), np_(off)
    for e, c in enumerate(counts):
        r = slice(o[e], o[e] + c)
        ref = xv[r] @ wv[e].T
        lim = 2.0 ** -8 * np.abs(ref) + 10 * 2.0 ** -22 * (np.abs(xv[r]) @ np.abs(wv[e]).T) + 1e-30
        assert np.all(np.abs(y[r] - ref) <= lim), e


def test_past_32_bits():
    """4.3 billion weights: cast, read-back and product of the last expert."""
    E, N, K = 66, 8192, 8192
    w = torch.zeros(E, N, K, dtype=torch.bfloat16, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(1)
    w[-1] = torch.randn(N, K, generator=g, device=DEV).to(torch.bfloat16)
    q, s = ops.quantize_mxfp4(w)
    q1, s1 = ops.quantize_mxfp4(w[-1:].contiguous())
    assert torch.equal(q[-1:], q1) and torch.equal(s[-s1.numel():], s1)
    del w
    v = ops.dequantize_mxfp4(q, s, K)
    assert torch.equal(v[-1:], ops.dequantize_mxfp4(q1, s1, K)) and not v[:-1].any()
    del v
    rng = np.random.default_rng(0)
    counts = [0] * (E - 1) + [2]
    xq, xs, cnt, off, xv, cap = _rows(rng, counts, K)
    y = ops.fc2_fwd_mxfp4(xq, xs, q, s, cnt, off)
    one = torch.tensor([2], dtype=torch.int32, device=DEV), torch.tensor([0, 32], dtype=torch.int32, device=DEV)
    assert torch.equal(y[:32], ops.fc2_fwd_mxfp4(xq, xs, q1, s1, *one)[:32]) and y[:2].any()


@pytest.mark.parametrize("counts,K,F", [([1], 32, 32), ([5, 33, 0, 64], 160, 160), ([130, 1, 300], 416, 544),
                                        ([700, 0, 450], 96, 96)])
@pytest.mark.parametrize("act", ["gptoss", "swiglu", "geglu", "srelu"])
def test_up_projection_column_copy(counts, K, F, act):
    """The column-wise MXFP8 copy of the activation's output: blocks of 32 rows
    of one column, the padding rows zeros.  Its values and the row-wise copy's
    come from one fp32 value v that is within lim of the formula's (fp32 sums of
    exact products, as for the product itself; the activation's slope is below
    4 (1 + max |z|) in its pre-activations); E4M3 steps are at most 2^-3 of a
    block's largest element, half a step of rounding and at most one of
    saturation (448 to 512) below 0.13 of it."""
    rng = np.random.default_rng(K + F + 1)
    E, gated = len(counts), act != "srelu"
    N = 2 * F if gated else F
    prm = L.glu_params("swiglu", alpha=1.702, up_offset=1.0, gate_lo=-7.0, gate_hi=7.0) if act == "gptoss" else \
        L.glu_params(act)
    op = {"gptoss": O.ActParams(O.ACT_SWIGLU, alpha=1.702, up_offset=1.0, gate_lo=-7.0, gate_hi=7.0),
          "swiglu": O.ActParams(O.ACT_SWIGLU), "geglu": O.ActParams(O.ACT_GEGLU), "srelu": O.ActParams(O.ACT_SRELU)}[act]
    xq, xs, cnt, off, xv, cap = _rows(rng, counts, K)
    q, s, wv = _weight(rng, E, N, K)
    m = ops.fc1_fwd_mxfp4(xq, xs, q, s, cnt, off, F, prm, out_mode=L.OUT_MXFP8, save_pre=False)
    r = ops.fc1_fwd_mxfp4(xq, xs, q, s, cnt, off, F, prm, out_mode=L.OUT_MXFP8, save_pre=False, with_col=False)
    assert ops.read_status(m["status"]) == 0
    of = np_(off)
    end = int(of[-1])
    assert torch.equal(m["q_row"][:end], r["q_row"][:end]) and torch.equal(m["s_row"][:end], r["s_row"][:end])
    col = O.mx_dequantize(np_(m["q_col"])[:, :end].copy(), np_(m["s_col"])[:, :end // 32].copy()).T
    for e, c in enumerate(counts):
        if not c:
            continue
        rows = slice(of[e], of[e] + c)
        z = xv[rows] @ wv[e].T
        mag = np.abs(xv[rows]) @ np.abs(wv[e]).T + np.abs(z)
        if gated:
            ref, slack = O.act_fwd(*O.unpack_glu_cols(z), op), np.maximum(*O.unpack_glu_cols(mag))
        else:
            ref, slack = O.act_fwd(z, None, op), mag
        lim = 2.0 ** -18 * np.abs(ref) + 16 * (K / 32 + 8) * 2.0 ** -22 * slack * (1 + np.abs(z).max()) + 1e-30
        pad = int(of[e + 1] - of[e]) - c
        full = np.pad(ref, ((0, pad), (0, 0)))
        lim = np.pad(lim, ((0, pad), (0, 0)))
        blk = np.abs(full).reshape(-1, 32, F).max(1, keepdims=True)
        d = col[of[e]:of[e + 1]]
        assert np.all(np.abs(d - full).reshape(-1, 32, F) <= 0.13 * blk + lim.reshape(-1, 32, F).max(1, keepdims=True))
        assert not d[c:].any()
