"""The up projection on MXFP4 weights with the activations that have no short
form (tanh GeGLU, sReGLU, GeGLU with clamps) and with clamps of the up half;
NVFP4 mode of a gated product.  Tolerances as for the other activations: the
fp32 sums are within (K / 32 + 8) 2^-22 sum |a w| of the exact ones, an
activation's slopes below 16 (1 + max |pre-activation|), its own arithmetic
within 2^-18 of the output, a bf16 output within 2^-8 of its magnitude."""
import numpy as np
import pytest
import torch

from grouped_gemm_glu_gb300 import lib as L
from grouped_gemm_glu_gb300 import ops, synth
from oracle import moe_oracle as O
from parity import np_
from test_gpu_mxfp4 import _rows, _weight

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
CLAMPS = dict(gate_lo=-1.5, gate_hi=1.0, up_lo=-1.0, up_hi=0.75)
ACTS = {
    "geglu_clamped": ("geglu", O.ACT_GEGLU, dict(up_offset=0.5, **CLAMPS)),
    "geglu_tanh": ("geglu_tanh", O.ACT_GEGLU_TANH, {}),
    "geglu_tanh_clamped": ("geglu_tanh", O.ACT_GEGLU_TANH, CLAMPS),
    "sreglu": ("sreglu", O.ACT_SREGLU, dict(up_offset=1.0)),
    "sreglu_clamped": ("sreglu", O.ACT_SREGLU, CLAMPS),
    "swiglu_up_clamp": ("swiglu", O.ACT_SWIGLU, dict(alpha=1.3, up_lo=-0.5, up_hi=1.0)),
}


@pytest.mark.parametrize("counts,K,F", [([5, 33, 0, 64], 160, 160), ([130, 1, 300], 416, 96)])
@pytest.mark.parametrize("act", ACTS)
def test_up_projection(counts, K, F, act):
    name, code, kw = ACTS[act]
    rng = np.random.default_rng(K + F)
    E = len(counts)
    prm, op = L.glu_params(name, **kw), O.ActParams(code, **kw)
    xq, xs, cnt, off, xv, cap = _rows(rng, counts, K)
    q, s, wv = _weight(rng, E, 2 * F, K)
    bias = synth._bf16(0.3 * rng.standard_normal((E, 2 * F)))
    args = (xq, xs, q, s, cnt, off, F, prm)
    o = ops.fc1_fwd_mxfp4(*args, out_mode=L.OUT_BF16, b1p=bias.to(DEV))
    n4 = ops.fc1_fwd_mxfp4(*args, out_mode=L.OUT_NVFP4, b1p=bias.to(DEV), save_pre=False)
    m = ops.fc1_fwd_mxfp4(*args, out_mode=L.OUT_MXFP8, b1p=bias.to(DEV), save_pre=False, with_col=False)
    for r in (o, n4, m):
        assert ops.read_status(r["status"]) == 0
    y, of = np_(o["y"]), np_(off)
    assert np.array_equal(np_(n4["y"])[:of[-1]], y[:of[-1]])
    top = slack_top = 0.0
    for e, c in enumerate(counts):
        if not c:
            continue
        r = slice(of[e], of[e] + c)
        z = xv[r] @ wv[e].T + np_(bias)[e]
        mag = np.abs(xv[r]) @ np.abs(wv[e]).T + np.abs(z)
        ref = O.act_fwd(*O.unpack_glu_cols(z), op)
        acc = 16 * (K / 32 + 8) * 2.0 ** -22 * np.maximum(*O.unpack_glu_cols(mag)) * (1 + np.abs(z).max()) + 1e-30
        lim = (2.0 ** -8 + 2.0 ** -18) * np.abs(ref) + acc
        assert np.all(np.abs(y[r] - ref) <= lim), (e, np.max(np.abs(y[r] - ref) - lim))
        assert not y[of[e] + c:of[e + 1]].any()
        top, slack_top = max(top, np.abs(ref).max()), max(slack_top, acc.max())
        d = O.mx_dequantize(np_(m["q_row"])[r], np_(m["s_row"])[r])
        blk = np.abs(ref).reshape(c, -1, 32).max(-1, keepdims=True)
        assert np.all(np.abs(d - ref).reshape(c, -1, 32) <= 0.13 * blk + lim.reshape(c, -1, 32))
    assert abs(float(n4["amax"]) - top) <= 2.0 ** -8 * top + slack_top
