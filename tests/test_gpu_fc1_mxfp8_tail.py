"""The MXFP8-input FC1 without a gate (sReLU) at F % 64 == 32: the last
32 columns are half of the 64-column block its epilogue drains, and nothing
past them is read or written.  Every output lies in a larger buffer of known
bytes, which must come back unchanged on both sides."""
import ctypes as C

import numpy as np
import pytest
import torch

from grouped_gemm_glu_gb300 import lib as L
from grouped_gemm_glu_gb300 import ops, synth
from oracle import moe_oracle as O
from parity import assert_bf16_close, assert_mx_close, np_

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
GUARD = 8192


def _guarded(nbytes):
    buf = torch.full((nbytes + 2 * GUARD,), 0xA5, dtype=torch.uint8, device=DEV)
    return buf, buf.data_ptr() + GUARD


def _inside(buf):
    b = buf.cpu().numpy()
    assert np.all(b[:GUARD] == 0xA5) and np.all(b[-GUARD:] == 0xA5), "written outside the output"
    return b[GUARD:-GUARD].copy()


@pytest.mark.parametrize("F", [32, 160, 288])
def test_srelu_half_block(F):
    rng = np.random.default_rng(F)
    H, E, counts = 96, 2, [40, 3]
    off = [0, 64, 96]
    R_cap = 128
    x = np.zeros((R_cap, H), np.float32)
    for e in range(E):
        x[off[e]:off[e] + counts[e]] = rng.standard_normal((counts[e], H))
    W = synth._bf16(rng.standard_normal((E, F, H)) * H ** -0.5)
    b = synth._bf16(0.3 * rng.standard_normal((E, F)))
    cnt = torch.tensor(counts, dtype=torch.int32, device=DEV)
    offs = torch.tensor(off, dtype=torch.int32, device=DEV)
    xq, xs = ops.quantize_mxfp8(synth._bf16(x).to(DEV))
    Wq, Ws = ops.quantize_mxfp8(W.to(DEV))
    bd = b.to(DEV)
    lib, prm, st = L.load(), L.glu_params("srelu"), ops.new_status(DEV)
    sizes = {"q_row": R_cap * F, "s_row": R_cap * F // 32, "q_col": R_cap * F, "s_col": R_cap * F // 32,
             "pre": 2 * R_cap * F}
    bufs = {k: _guarded(n) for k, n in sizes.items()}
    out = L.ActOut(q_row=bufs["q_row"][1], s_row=bufs["s_row"][1], q_col=bufs["q_col"][1], s_col=bufs["s_col"][1],
                   pre=bufs["pre"][1])
    n = lib.moe_grouped_fc2_workspace_size(E, H, F, R_cap)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    L.check(lib.moe_grouped_fc1_glu_quant_fwd_mxfp8(
        xq.data_ptr(), xs.data_ptr(), Wq.data_ptr(), Ws.data_ptr(), bd.data_ptr(), None, cnt.data_ptr(),
        offs.data_ptr(), E, H, F, R_cap, C.byref(prm), L.OUT_MXFP8, C.byref(out), ws.data_ptr(), n, 0, st.data_ptr(),
        torch.cuda.current_stream().cuda_stream), "fc1")
    torch.cuda.synchronize()
    got = {k: _inside(v[0]) for k, v in bufs.items()}
    assert ops.read_status(st) == 0
    xd = O.mx_dequantize(np_(xq), np_(xs))
    Wd = O.mx_dequantize(np_(Wq).reshape(E * F, H), np_(Ws).reshape(E * F, H // 32)).reshape(E, F, H)
    pre = torch.from_numpy(got["pre"]).view(torch.bfloat16).view(R_cap, F)
    q, s = got["q_row"].reshape(R_cap, F), got["s_row"].reshape(R_cap, F // 32)
    for e in range(E):
        r = slice(off[e], off[e] + counts[e])
        z = xd[r] @ Wd[e].T + np_(b)[e]
        assert_bf16_close(np_(pre)[r], z, "pre")
        y = np.maximum(z, 0.0) ** 2
        qr, sr = O.mx_quantize_rows(y)
        assert_mx_close(q[r], s[r], qr, sr, y, "rows")
