"""torch-facing wrappers of the C ABI: allocate outputs with torch (device
memory and streams only) and pass raw pointers to libmoeglu.  No step of the
method is computed here."""
from __future__ import annotations

import ctypes as C
import functools

import torch

from . import lib as L


def _p(t):
    return None if t is None else C.c_void_p(t.data_ptr())


def _s(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return C.c_void_p(s.cuda_stream)


def _dev(t):
    if not t.is_cuda:
        raise ValueError("tensors must live on a CUDA device")
    return t.device


def new_status(device) -> torch.Tensor:
    return torch.zeros(1, dtype=torch.int32, device=device)


def read_status(status: torch.Tensor) -> int:
    out = C.c_int32(0)
    L.check(L.load().moe_get_status(_p(status), C.byref(out), _s()), "moe_get_status")
    return out.value


def wait_selftest(arrive: bool, device="cuda") -> tuple[int, int]:
    """Runs the bounded-wait self-test; returns (status word, ns waited)."""
    status = new_status(device)
    waited = torch.zeros(1, dtype=torch.int64, device=device)
    L.check(L.load().moe_wait_selftest(1 if arrive else 0, _p(status), _p(waited), _s()), "moe_wait_selftest")
    return read_status(status), int(waited.item())


def repack_fc1(W1: torch.Tensor, inverse: bool = False) -> torch.Tensor:
    """[E, 2F, H] logical input|gate rows <-> packed rows (bf16)."""
    lib = L.load()
    E, N1, H = W1.shape
    out = torch.empty_like(W1)
    L.check(lib.moe_repack_fc1(_p(W1), _p(out), E, N1 // 2, H, int(inverse), _s()), "moe_repack_fc1")
    return out


def route_permute(x, topk_idx, topk_prob, E: int, R_cap: int, expert_begin: int = 0, status=None,
                  with_col: bool = False) -> dict:
    """Routing + gather; with_col also returns the column-wise MXFP8 copy of
    x_perm made during the gather (x_qc [H, R_cap], x_sc [H, R_cap/32])."""
    lib = L.load()
    dev = _dev(x)
    T, H = x.shape
    k = topk_idx.shape[1]
    o = {
        "x_perm": torch.empty(R_cap, H, dtype=torch.bfloat16, device=dev),
        "row_of": torch.empty(T * k, dtype=torch.int32, device=dev),
        "tok_of": torch.empty(R_cap, dtype=torch.int32, device=dev),
        "prob_perm": torch.empty(R_cap, dtype=torch.float32, device=dev),
        "counts": torch.empty(E, dtype=torch.int32, device=dev),
        "offsets": torch.empty(E + 1, dtype=torch.int32, device=dev),
    }
    if with_col:
        o["x_qc"] = torch.zeros(H, R_cap, dtype=torch.uint8, device=dev)
        o["x_sc"] = torch.zeros(H, R_cap // 32, dtype=torch.uint8, device=dev)
    ws_bytes = lib.moe_route_workspace_size(T, k, E)
    ws = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
    st = status if status is not None else new_status(dev)
    L.check(lib.moe_route_permute(_p(x), _p(topk_idx), _p(topk_prob), T, H, k, expert_begin, E, R_cap,
                                  _p(o["x_perm"]), _p(o["row_of"]), _p(o["tok_of"]), _p(o["prob_perm"]),
                                  _p(o["counts"]), _p(o["offsets"]), _p(o.get("x_qc")), _p(o.get("x_sc")), _p(ws),
                                  ws_bytes, _p(st), _s()),
            "moe_route_permute")
    o["status"] = st
    return o


def _act_out(q_row=None, s_row=None, q_col=None, s_col=None, y=None, amax=None, pre=None) -> L.ActOut:
    return L.ActOut(*(None if t is None else t.data_ptr() for t in (q_row, s_row, q_col, s_col, y, amax, pre)))


def fc1_fwd(x_perm, W1p, counts, offsets, F: int, params: L.GluParams, out_mode: int = L.OUT_MXFP8,
            b1p=None, row_scale=None, save_pre: bool = True, with_col: bool = True, sm_margin: int = 0,
            status=None, out: dict | None = None, dynamic: bool = True) -> dict:
    """GroupGemm + Activation + Quantize/Transpose.  Returns the output tensors
    ({q_row, s_row, q_col, s_col} | {y[, amax]}, and pre when saved).
    dynamic=False runs the static tile schedule (no workspace)."""
    lib = L.load()
    dev = _dev(x_perm)
    R_cap, H = x_perm.shape
    E = counts.shape[0]
    gated = params.act in (L.ACT["swiglu"], L.ACT["geglu"], L.ACT["geglu_tanh"], L.ACT["sreglu"])
    N1 = 2 * F if gated else F
    o = out if out is not None else {}
    if params.act == L.ACT["none"]:
        o.setdefault("pre", torch.empty(R_cap, F, dtype=torch.bfloat16, device=dev))
    else:
        if out_mode == L.OUT_MXFP8:
            o.setdefault("q_row", torch.empty(R_cap, F, dtype=torch.uint8, device=dev))
            o.setdefault("s_row", torch.empty(R_cap, F // 32, dtype=torch.uint8, device=dev))
            if with_col:
                o.setdefault("q_col", torch.empty(F, R_cap, dtype=torch.uint8, device=dev))
                o.setdefault("s_col", torch.empty(F, R_cap // 32, dtype=torch.uint8, device=dev))
        else:
            o.setdefault("y", torch.empty(R_cap, F, dtype=torch.bfloat16, device=dev))
            if out_mode == L.OUT_NVFP4:
                o.setdefault("amax", torch.zeros(1, dtype=torch.float32, device=dev))
        if save_pre:
            o.setdefault("pre", torch.empty(R_cap, N1, dtype=torch.bfloat16, device=dev))
    st = status if status is not None else new_status(dev)
    ao = _act_out(o.get("q_row"), o.get("s_row"), o.get("q_col"), o.get("s_col"), o.get("y"), o.get("amax"),
                  o.get("pre"))
    ws_bytes = lib.moe_grouped_fc1_workspace_size(E, N1, R_cap) if dynamic else 0
    ws = torch.empty(ws_bytes, dtype=torch.uint8, device=dev) if dynamic else None
    L.check(lib.moe_grouped_fc1_glu_quant_fwd(_p(x_perm), _p(W1p), _p(b1p), _p(row_scale), _p(counts),
                                              _p(offsets), E, H, F, R_cap, C.byref(params), out_mode,
                                              C.byref(ao), _p(ws), ws_bytes, sm_margin, _p(st), _s()),
            "moe_grouped_fc1_glu_quant_fwd")
    o["status"] = st
    return o


def fc1_fwd_mxfp8(xq, xs, W1q, W1s, counts, offsets, F: int, params: L.GluParams, out_mode: int = L.OUT_MXFP8,
                  b1p=None, row_scale=None, save_pre: bool = True, with_col: bool = True, sm_margin: int = 0,
                  status=None) -> dict:
    """GroupGemm + Activation + Quantize/Transpose on MXFP8 operands: xq/xs
    [R_cap, H] (+ /32) the row-wise MXFP8 of x_perm, W1q/W1s [E, N1, H]
    (+ /32) the row-wise MXFP8 of the packed W1p.  Same outputs as fc1_fwd."""
    lib = L.load()
    dev = _dev(xq)
    R_cap, H = xq.shape
    E, N1, _ = W1q.shape
    o = {}
    if out_mode == L.OUT_MXFP8:
        o["q_row"] = torch.empty(R_cap, F, dtype=torch.uint8, device=dev)
        o["s_row"] = torch.empty(R_cap, F // 32, dtype=torch.uint8, device=dev)
        if with_col:
            o["q_col"] = torch.empty(F, R_cap, dtype=torch.uint8, device=dev)
            o["s_col"] = torch.empty(F, R_cap // 32, dtype=torch.uint8, device=dev)
    else:
        o["y"] = torch.empty(R_cap, F, dtype=torch.bfloat16, device=dev)
        if out_mode == L.OUT_NVFP4:
            o["amax"] = torch.zeros(1, dtype=torch.float32, device=dev)
    if save_pre:
        o["pre"] = torch.empty(R_cap, N1, dtype=torch.bfloat16, device=dev)
    st = status if status is not None else new_status(dev)
    ws_bytes = lib.moe_grouped_fc2_workspace_size(E, H, N1, R_cap)
    ws = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
    ao = _act_out(o.get("q_row"), o.get("s_row"), o.get("q_col"), o.get("s_col"), o.get("y"), o.get("amax"),
                  o.get("pre"))
    L.check(lib.moe_grouped_fc1_glu_quant_fwd_mxfp8(_p(xq), _p(xs), _p(W1q), _p(W1s), _p(b1p), _p(row_scale),
                                                    _p(counts), _p(offsets), E, H, F, R_cap, C.byref(params),
                                                    out_mode, C.byref(ao), _p(ws), ws_bytes, sm_margin, _p(st),
                                                    _s()), "moe_grouped_fc1_glu_quant_fwd_mxfp8")
    o["status"] = st
    return o


def dglu_bwd(dY_perm, W2, pre, counts, offsets, F: int, params: L.GluParams, out_mode: int = L.OUT_MXFP8,
             row_scale=None, with_col: bool = True, sm_margin: int = 0, status=None,
             out: dict | None = None, row_dot: bool = False, rht_signs: int | None = None,
             dbias: bool = False, dynamic: bool = True) -> dict:
    """GroupGemm + dActivation + Quantize/Transpose.  dFC1 in packed order;
    row_dot=True also returns o["row_dot"], the per-row partials of the
    feature-scale gradient (reduce with feature_scale_grad).  NVFP4 mode
    returns y and amax (max |y|); with rht_signs (16-bit mask) also
    o["rht_amax"], the amax of y's transposed random Hadamard rotation.
    dbias=True also returns o["dbias"] [E, N1] f32, the FC1 bias gradient
    (packed column order)."""
    lib = L.load()
    dev = _dev(dY_perm)
    R_cap, H = dY_perm.shape
    E = counts.shape[0]
    N1 = pre.shape[1]
    o = out if out is not None else {}
    if out_mode == L.OUT_MXFP8:
        o.setdefault("q_row", torch.empty(R_cap, N1, dtype=torch.uint8, device=dev))
        o.setdefault("s_row", torch.empty(R_cap, N1 // 32, dtype=torch.uint8, device=dev))
        if with_col:
            o.setdefault("q_col", torch.empty(N1, R_cap, dtype=torch.uint8, device=dev))
            o.setdefault("s_col", torch.empty(N1, R_cap // 32, dtype=torch.uint8, device=dev))
    else:
        o.setdefault("y", torch.empty(R_cap, N1, dtype=torch.bfloat16, device=dev))
        if out_mode == L.OUT_NVFP4:
            o.setdefault("amax", torch.zeros(1, dtype=torch.float32, device=dev))
            if rht_signs is not None:
                o.setdefault("rht_amax", torch.zeros(1, dtype=torch.float32, device=dev))
    if row_dot:
        o.setdefault("row_dot", torch.empty(R_cap, lib.moe_dglu_row_dot_parts(F), dtype=torch.float32, device=dev))
    st = status if status is not None else new_status(dev)
    ao = _act_out(o.get("q_row"), o.get("s_row"), o.get("q_col"), o.get("s_col"), o.get("y"), o.get("amax"))
    ao.row_dot = o["row_dot"].data_ptr() if "row_dot" in o else None
    if "rht_amax" in o:
        ao.rht_amax, ao.rht_signs = o["rht_amax"].data_ptr(), int(rht_signs) & 0xFFFF
    ws_bytes, ws = 0, None
    if dbias:
        o.setdefault("dbias", torch.empty(E, N1, dtype=torch.float32, device=dev))
    if dbias or dynamic:
        ws_bytes = lib.moe_grouped_dglu_workspace_size(N1, R_cap) if dbias else lib.moe_grouped_dglu_workspace_size(0, 0)
        ws = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
    L.check(lib.moe_grouped_dglu_quant_bwd(_p(dY_perm), _p(W2), _p(pre), _p(row_scale), _p(counts), _p(offsets),
                                           E, H, F, R_cap, C.byref(params), out_mode, C.byref(ao), _p(o.get("dbias")),
                                           _p(ws), ws_bytes, sm_margin, _p(st), _s()),
            "moe_grouped_dglu_quant_bwd")
    o["status"] = st
    return o


def quantize_mxfp8(src, col: bool = False, counts=None, offsets=None, out=None, status=None, tiled: bool = False):
    """src [R, C] or [G, R, C] bf16 -> (q, s); col=True gives the transposed
    column-wise copy; tiled (with col) writes the scales in the tensor-core
    order of a GEMM weight operand (flat uint8 [moe_mxfp8_tiled_scale_bytes])."""
    lib = L.load()
    dev = _dev(src)
    s3 = src if src.dim() == 3 else src.unsqueeze(0)
    G, R, Cc = s3.shape
    if col and tiled:
        q = torch.empty(G, Cc, R, dtype=torch.uint8, device=dev) if out is None else out[0]
        s = (torch.empty(lib.moe_mxfp8_tiled_scale_bytes(G, R, Cc), dtype=torch.uint8, device=dev)
             if out is None else out[1])
        L.check(lib.moe_quantize_mxfp8(_p(s3), G, R, Cc, 2, None, None, 0, _p(q), _p(s), _p(status), _s()),
                "moe_quantize_mxfp8")
        return (q[0] if src.dim() == 2 and out is None else q), s
    if col:
        q = torch.empty(G, Cc, R, dtype=torch.uint8, device=dev) if out is None else out[0]
        s = torch.empty(G, Cc, R // 32, dtype=torch.uint8, device=dev) if out is None else out[1]
    else:
        q = torch.empty(G, R, Cc, dtype=torch.uint8, device=dev) if out is None else out[0]
        s = torch.empty(G, R, Cc // 32, dtype=torch.uint8, device=dev) if out is None else out[1]
    E = 0 if counts is None else counts.shape[0]
    L.check(lib.moe_quantize_mxfp8(_p(s3), G, R, Cc, int(col), _p(counts), _p(offsets), E, _p(q), _p(s),
                                   _p(status), _s()), "moe_quantize_mxfp8")
    if src.dim() == 2 and out is None:
        return q[0], s[0]
    return q, s


def quantize_mxfp8_dual(src, status=None):
    """src [G, R, C] (or [R, C]) bf16 read once -> (q_row [G, R, C],
    s_row [G, R, C/32], q_col [G, C, R], s_col [G, C, R/32])."""
    lib = L.load()
    dev = _dev(src)
    s3 = src if src.dim() == 3 else src.unsqueeze(0)
    G, R, Cc = s3.shape
    qr = torch.empty(G, R, Cc, dtype=torch.uint8, device=dev)
    sr = torch.empty(G, R, Cc // 32, dtype=torch.uint8, device=dev)
    qc = torch.empty(G, Cc, R, dtype=torch.uint8, device=dev)
    sc = torch.empty(G, Cc, R // 32, dtype=torch.uint8, device=dev)
    L.check(lib.moe_quantize_mxfp8_dual(_p(s3), G, R, Cc, _p(qr), _p(sr), _p(qc), _p(sc), _p(status), _s()),
            "moe_quantize_mxfp8_dual")
    return qr, sr, qc, sc


def fc2_fwd(Aq, As, Wq, Ws, counts, offsets, sm_margin: int = 0, status=None, out=None,
            out_mode: int = L.OUT_BF16, with_col: bool = True, w_tiled: bool = False):
    """GroupGemm (+ Quantize): y [R_cap, N] = A [R_cap, K] . W[e]^T per expert
    with W [E, N, K].  MXFP8 operands (codes Aq/Wq with E8M0 scales As/Ws),
    or bf16 operands when As and Ws are None.  out_mode OUT_BF16 returns the
    bf16 tensor y; OUT_MXFP8 returns {q_row, s_row[, q_col, s_col]};
    OUT_NVFP4 returns {y, amax}.  w_tiled: Ws is in the tensor-core order
    (quantize_mxfp8(..., col=True, tiled=True))."""
    lib = L.load()
    dev = _dev(Aq)
    R_cap, K = Aq.shape
    E, N, _ = Wq.shape
    if (As is None) != (Ws is None):
        raise ValueError("both operands bf16 (no scales) or both MXFP8")
    o = {}
    if out_mode == L.OUT_BF16:
        o["y"] = out if out is not None else torch.empty(R_cap, N, dtype=torch.bfloat16, device=dev)
    elif out_mode == L.OUT_MXFP8:
        o["q_row"] = torch.empty(R_cap, N, dtype=torch.uint8, device=dev)
        o["s_row"] = torch.empty(R_cap, N // 32, dtype=torch.uint8, device=dev)
        if with_col:
            o["q_col"] = torch.empty(N, R_cap, dtype=torch.uint8, device=dev)
            o["s_col"] = torch.empty(N, R_cap // 32, dtype=torch.uint8, device=dev)
    else:
        o["y"] = torch.empty(R_cap, N, dtype=torch.bfloat16, device=dev)
        o["amax"] = torch.zeros(1, dtype=torch.float32, device=dev)
    st = status if status is not None else new_status(dev)
    a_in = L.in_operand(Aq.data_ptr(), None if As is None else As.data_ptr())
    w_in = L.in_operand(Wq.data_ptr(), None if Ws is None else Ws.data_ptr(), tiled=w_tiled)
    ws_bytes = lib.moe_grouped_fc2_workspace_size(E, K, N, R_cap) if As is not None else 0
    ws = torch.empty(max(ws_bytes, 1), dtype=torch.uint8, device=dev)
    ao = _act_out(o.get("q_row"), o.get("s_row"), o.get("q_col"), o.get("s_col"), o.get("y"), o.get("amax"))
    L.check(lib.moe_grouped_fc2_fwd(C.byref(a_in), C.byref(w_in), _p(counts), _p(offsets), E, K, N, R_cap, out_mode,
                                    C.byref(ao), _p(ws), ws_bytes, sm_margin, _p(st), _s()), "moe_grouped_fc2_fwd")
    o["status"] = st
    return o["y"] if out_mode == L.OUT_BF16 else o


def fc2_fwd_nvfp4(Aq, As, sgA, Wq, Ws, sgW, counts, offsets, sm_margin: int = 0, status=None, out=None,
                  w_tiled: bool = False):
    """GroupGemm on NVFP4 operands: y [R_cap, N] bf16 = A . W[e]^T with
    A = packed E2M1 [R_cap, K/2] + E4M3 scales [R_cap, K/16] + per-tensor
    scale sgA (device float [1]), W [E, N, K/2] + [E, N, K/16] + sgW
    (w_tiled: Ws in the tensor-core order, nvfp4_cast_cols(..., tiled=True))."""
    lib = L.load()
    dev = _dev(Aq)
    R_cap, K2 = Aq.shape
    K = 2 * K2
    E, N, _ = Wq.shape
    y = out if out is not None else torch.empty(R_cap, N, dtype=torch.bfloat16, device=dev)
    st = status if status is not None else new_status(dev)
    a_in = L.in_operand(Aq.data_ptr(), As.data_ptr(), sgA.data_ptr())
    w_in = L.in_operand(Wq.data_ptr(), Ws.data_ptr(), sgW.data_ptr(), tiled=w_tiled)
    ws_bytes = lib.moe_grouped_fc2_workspace_size(E, K, N, R_cap)
    ws = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
    ao = _act_out(y=y)
    L.check(lib.moe_grouped_fc2_fwd(C.byref(a_in), C.byref(w_in), _p(counts), _p(offsets), E, K, N, R_cap,
                                    L.OUT_BF16, C.byref(ao), _p(ws), ws_bytes, sm_margin, _p(st), _s()),
            "moe_grouped_fc2_fwd (NVFP4)")
    return y


def amax_bf16(x):
    """max |x| of a bf16 tensor as a device float [1]."""
    lib = L.load()
    a = torch.empty(1, dtype=torch.float32, device=_dev(x))
    L.check(lib.moe_amax_bf16(_p(x), x.numel(), _p(a), _s()), "moe_amax_bf16")
    return a


def nvfp4_cast_cols(src, amax, status=None, tiled: bool = False, out=None):
    """Column-wise NVFP4 of src [G, R, C] (or [R, C]) bf16: (q [G, C, R/2],
    s [G, C, R/16], s_global [1]); tiled: s in the tensor-core order of a
    GEMM weight operand (flat uint8 [moe_nvfp4_tiled_scale_bytes]).  out:
    optional (q, s, s_global) to write into."""
    lib = L.load()
    dev = _dev(src)
    s3 = src if src.dim() == 3 else src.unsqueeze(0)
    G, R, Cc = s3.shape
    if out is not None:
        q, s, sg = out
    else:
        q = torch.empty(G, Cc, R // 2, dtype=torch.uint8, device=dev)
        s = (torch.empty(lib.moe_nvfp4_tiled_scale_bytes(G, R, Cc), dtype=torch.uint8, device=dev) if tiled
             else torch.empty(G, Cc, R // 16, dtype=torch.uint8, device=dev))
        sg = torch.empty(1, dtype=torch.float32, device=dev)
    fn = lib.moe_nvfp4_cast_cols_tiled if tiled else lib.moe_nvfp4_cast_cols
    L.check(fn(_p(s3), G, R, Cc, _p(amax), _p(q), _p(s), _p(sg), _p(status), _s()),
            "moe_nvfp4_cast_cols_tiled" if tiled else "moe_nvfp4_cast_cols")
    return q, s, sg


def wgrad(Aq_col, As_col, Bq_col, Bs_col, counts, offsets, out_f32: bool = False, sm_margin: int = 0,
          status=None, out=None):
    """D [E, M, N] = per-expert contraction over the expert's rows of the
    column-wise MXFP8 copies A [M, R_cap] and B [N, R_cap]."""
    lib = L.load()
    dev = _dev(Aq_col)
    M, R_cap = Aq_col.shape
    N = Bq_col.shape[0]
    E = counts.shape[0]
    D = out if out is not None else torch.empty(E, M, N, dtype=torch.float32 if out_f32 else torch.bfloat16,
                                                device=dev)
    st = status if status is not None else new_status(dev)
    ws_bytes = lib.moe_grouped_wgrad_workspace_size(E, M, N, R_cap)
    ws = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
    L.check(lib.moe_grouped_wgrad(_p(Aq_col), _p(As_col), _p(Bq_col), _p(Bs_col), _p(counts), _p(offsets), E, M,
                                  N, R_cap, _p(D), int(out_f32), _p(ws), ws_bytes, sm_margin, _p(st), _s()),
            "moe_grouped_wgrad")
    return D


def rht_amax_cols(src, offsets, signs: int, status=None):
    """max |rotated value| of src [R_cap, C] (16-row Hadamard blocks below
    offsets[E]) as a device float [1]."""
    lib = L.load()
    R_cap, Cc = src.shape
    a = torch.empty(1, dtype=torch.float32, device=_dev(src))
    L.check(lib.moe_rht_amax_cols(_p(src), R_cap, Cc, _p(offsets), offsets.shape[0] - 1, int(signs) & 0xFFFF, _p(a),
                                  _p(status), _s()), "moe_rht_amax_cols")
    return a


def nvfp4_rht_cast_cols(src, offsets, amax, signs: int, status=None):
    """Rotated column-wise NVFP4 of src [R_cap, C]: (q [C, R_cap/2],
    s [C, R_cap/16], s_global [1])."""
    lib = L.load()
    dev = _dev(src)
    R_cap, Cc = src.shape
    q = torch.empty(Cc, R_cap // 2, dtype=torch.uint8, device=dev)
    s = torch.empty(Cc, R_cap // 16, dtype=torch.uint8, device=dev)
    sg = torch.empty(1, dtype=torch.float32, device=dev)
    L.check(lib.moe_nvfp4_rht_cast_cols(_p(src), R_cap, Cc, _p(offsets), offsets.shape[0] - 1, _p(amax),
                                        int(signs) & 0xFFFF, _p(q), _p(s), _p(sg), _p(status), _s()),
            "moe_nvfp4_rht_cast_cols")
    return q, s, sg


def wgrad_nvfp4(Aq, As, sgA, Bq, Bs, sgB, counts, offsets, out_f32: bool = False, sm_margin: int = 0, status=None):
    """D [E, M, N] = per-expert contraction over the expert's rows of the
    column-wise NVFP4 operands A [M, R_cap/2] and B [N, R_cap/2]."""
    lib = L.load()
    dev = _dev(Aq)
    M, R2 = Aq.shape
    R_cap = 2 * R2
    N = Bq.shape[0]
    E = counts.shape[0]
    D = torch.empty(E, M, N, dtype=torch.float32 if out_f32 else torch.bfloat16, device=dev)
    st = status if status is not None else new_status(dev)
    ws_bytes = lib.moe_grouped_wgrad_workspace_size(E, M, N, R_cap)
    ws = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
    L.check(lib.moe_grouped_wgrad_nvfp4(_p(Aq), _p(As), _p(sgA), _p(Bq), _p(Bs), _p(sgB), _p(counts), _p(offsets), E,
                                        M, N, R_cap, _p(D), int(out_f32), _p(ws), ws_bytes, sm_margin, _p(st), _s()),
            "moe_grouped_wgrad_nvfp4")
    return D


def unpermute_combine(y_perm, row_of, topk_prob, status=None, out=None):
    lib = L.load()
    dev = _dev(y_perm)
    T, k = topk_prob.shape
    H = y_perm.shape[1]
    o = out if out is not None else torch.empty(T, H, dtype=torch.bfloat16, device=dev)
    L.check(lib.moe_unpermute_combine(_p(y_perm), _p(row_of), _p(topk_prob), T, H, k, _p(o), _p(status), _s()),
            "moe_unpermute_combine")
    return o


def combine_bwd(dout, y_perm, route: dict, k: int, status=None, out=None, col=None):
    """Gradient of the combine for dout [T, H]: (dY_perm [R_cap, H] bf16,
    dprob [T, k] f32); route = the dict of route_permute.  col = (q [H, R_cap],
    s [H, R_cap/32]) uint8 tensors: also the column-wise MXFP8 of dY_perm."""
    lib = L.load()
    dev = _dev(dout)
    T, H = dout.shape
    R_cap = y_perm.shape[0]
    E = route["counts"].shape[0]
    dY = out[0] if out is not None else torch.empty(R_cap, H, dtype=torch.bfloat16, device=dev)
    dprob = out[1] if out is not None else torch.empty(T, k, dtype=torch.float32, device=dev)
    st = status if status is not None else route.get("status")
    L.check(lib.moe_combine_bwd(_p(dout), _p(y_perm), _p(route["row_of"]), _p(route["tok_of"]),
                                _p(route["prob_perm"]), _p(route["offsets"]), T, H, k, E, R_cap, _p(dY),
                                _p(dprob), _p(col[0] if col else None), _p(col[1] if col else None), _p(st),
                                _s()), "moe_combine_bwd")
    return dY, dprob


def feature_scale_grad(row_dot, row_of, T: int, k: int, out=None):
    """dprob [T, k] f32 from the dGLU epilogue's per-row partials."""
    lib = L.load()
    o = out if out is not None else torch.empty(T, k, dtype=torch.float32, device=row_dot.device)
    L.check(lib.moe_feature_scale_grad(_p(row_dot), row_dot.shape[1], _p(row_of), T, k, _p(o), _s()),
            "moe_feature_scale_grad")
    return o


def permute_bwd(dx_perm, row_of, T: int, k: int, status=None, out=None):
    """Gradient of the permute: dx [T, H] bf16 from dx_perm [R_cap, H]."""
    lib = L.load()
    dev = _dev(dx_perm)
    H = dx_perm.shape[1]
    o = out if out is not None else torch.empty(T, H, dtype=torch.bfloat16, device=dev)
    L.check(lib.moe_permute_bwd(_p(dx_perm), _p(row_of), T, H, k, _p(o), _p(status), _s()), "moe_permute_bwd")
    return o


def nvfp4_cast(y, amax, counts, offsets):
    lib = L.load()
    dev = _dev(y)
    R_cap, N = y.shape
    q = torch.empty(R_cap, N // 2, dtype=torch.uint8, device=dev)
    s = torch.empty(R_cap, N // 16, dtype=torch.uint8, device=dev)
    sg = torch.empty(1, dtype=torch.float32, device=dev)
    L.check(lib.moe_nvfp4_cast(_p(y), _p(amax), _p(counts), _p(offsets), counts.shape[0], N, R_cap, _p(q), _p(s),
                               _p(sg), _s()), "moe_nvfp4_cast")
    return q, s, sg


def glu_act(pre, counts, offsets, F: int, params: L.GluParams):
    lib = L.load()
    dev = _dev(pre)
    R_cap = pre.shape[0]
    y = torch.empty(R_cap, F, dtype=torch.bfloat16, device=dev)
    L.check(lib.moe_glu_act(_p(pre), _p(counts), _p(offsets), counts.shape[0], F, R_cap, C.byref(params), _p(y),
                            _s()), "moe_glu_act")
    return y


def dglu_act(da, pre, counts, offsets, F: int, params: L.GluParams):
    """Unfused backward activation: da [R, F] and pre [R, N1] -> dFC1 [R, N1]."""
    lib = L.load()
    dev = _dev(da)
    R_cap, N1 = pre.shape
    d = torch.empty(R_cap, N1, dtype=torch.bfloat16, device=dev)
    L.check(lib.moe_dglu_act(_p(da), _p(pre), _p(counts), _p(offsets), counts.shape[0], F, R_cap, C.byref(params),
                             _p(d), _s()), "moe_dglu_act")
    return d


def _need(t, dtype, shape, what):
    """A dense CUDA tensor of this type and shape (None: any shape), or ValueError."""
    if isinstance(t, torch.Tensor) and t.is_cuda and t.dtype == dtype and t.is_contiguous() and (
            shape is None or t.shape == shape):
        return t
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{what}: a CUDA tensor is needed")
    if t.dtype != dtype:
        raise ValueError(f"{what}: {dtype} is needed, got {t.dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{what}: shape {tuple(shape)} is needed, got {tuple(t.shape)}")
    raise ValueError(f"{what}: a contiguous tensor is needed")


def _need2(t, dtype, what):
    """_need for a matrix of any size; returns its two extents."""
    _need(t, dtype, None, what)
    if t.dim() != 2:
        raise ValueError(f"{what}: two dimensions are needed, got {tuple(t.shape)}")
    return t.shape


def _cur(t) -> int:
    """The current stream's handle on t's device."""
    return torch._C._cuda_getCurrentRawStream(t.get_device())


def _ptr(t):
    return None if t is None else t.data_ptr()


def rmsnorm(x, gamma, eps: float = 1e-5, residual=None, bf16: bool = True, mxfp8: bool = False,
            with_rstd: bool = True) -> dict:
    """Residual addition and RMS norm of x [T, H] bf16 with the weight gamma
    [H]: y = h * rstd * gamma with h = bf16(x + residual).  Returns h (with a
    residual), y (bf16=True), q [T, H] and s [T, H/32] (mxfp8=True: the
    row-wise MXFP8 of y, what an MXFP8 FC1 reads) and rstd [T]."""
    bf = torch.bfloat16
    T, H = _need2(x, bf, "x")
    _need(gamma, bf, (H,), "gamma")
    o = {}
    new, dev = torch.empty, x.device
    h = y = q = s = r = None
    if residual is not None:
        _need(residual, bf, (T, H), "residual")
        h = o["h"] = torch.empty_like(x)
    if bf16:
        y = o["y"] = torch.empty_like(x)
    if mxfp8:
        q = o["q"] = new(T, H, dtype=torch.uint8, device=dev)
        s = o["s"] = new(T, H // 32, dtype=torch.uint8, device=dev)
    if with_rstd:
        r = o["rstd"] = new(T, dtype=torch.float32, device=dev)
    L.check(L.load().moe_rmsnorm_fwd(x.data_ptr(), _ptr(residual), gamma.data_ptr(), eps, T, H, _ptr(h), _ptr(y),
                                     _ptr(q), _ptr(s), _ptr(r), _cur(x)), "moe_rmsnorm_fwd")
    return o


def rmsnorm_bwd(dy, h, gamma, rstd, dres=None, with_dgamma: bool = True):
    """Backward of rmsnorm: (dx [T, H] bf16, dgamma [H] f32 or None).  h is the
    forward's h (its x where there was no residual), dres the gradient that
    arrives at h from the rest of the residual stream; dx is the gradient of x
    and of the residual alike."""
    bf = torch.bfloat16
    T, H = _need2(dy, bf, "dy")
    _need(h, bf, (T, H), "h")
    _need(gamma, bf, (H,), "gamma")
    _need(rstd, torch.float32, (T,), "rstd")
    if dres is not None:
        _need(dres, bf, (T, H), "dres")
    lib = L.load()
    dx = torch.empty_like(dy)
    dgamma = ws = None
    nbytes = 0
    if with_dgamma:
        dgamma = torch.empty(H, dtype=torch.float32, device=dy.device)
        nbytes = _size("moe_rmsnorm_bwd_workspace_size", T, H)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=dy.device)
    L.check(lib.moe_rmsnorm_bwd(dy.data_ptr(), _ptr(dres), h.data_ptr(), gamma.data_ptr(), rstd.data_ptr(), T, H,
                                dx.data_ptr(), _ptr(dgamma), _ptr(ws), nbytes, _cur(dy)), "moe_rmsnorm_bwd")
    return dx, dgamma


def dequantize_mxfp8(q, s, out=None):
    """The bf16 values of MXFP8 codes q [..., C] with scales s [..., C/32]."""
    _need(q, torch.uint8, None, "q")
    if q.shape[-1] % 32:
        raise ValueError("q: the last dimension must be a multiple of 32")
    _need(s, torch.uint8, (*q.shape[:-1], q.shape[-1] // 32), "s")
    o = _need(out, torch.bfloat16, q.shape, "out") if out is not None else torch.empty(
        q.shape, dtype=torch.bfloat16, device=q.device)
    L.check(L.load().moe_dequantize_mxfp8(q.data_ptr(), s.data_ptr(), s.numel(), o.data_ptr(), _cur(q)),
            "moe_dequantize_mxfp8")
    return o


def _logits(logits):
    dt = logits.dtype
    if dt != torch.float32 and dt != torch.bfloat16:
        raise ValueError(f"logits: float32 or bfloat16 is needed, got {dt}")
    _need2(logits, dt, "logits")
    return 1 if dt == torch.bfloat16 else 0


def router(logits, k: int, params: L.RouterParams, bias=None, token_mask=None, with_load: bool = True) -> dict:
    """Expert choice from logits [T, n] (f32 or bf16): idx [T, k] int32 and
    prob [T, k] f32 (route_permute's topk_idx and topk_prob; slots without an
    expert hold -1 and 0) and load [n] int32, the tokens of each expert.
    bias [n] f32 takes part in the choice only; token_mask [T] uint8 or bool:
    tokens with 0 choose nothing.  With group_top = 2 a group that has fewer
    than two experts left (logit or bias not -inf) ranks behind all others."""
    b16 = _logits(logits)
    T, n = logits.shape
    if bias is not None:
        _need(bias, torch.float32, (n,), "bias")
    if token_mask is not None:
        if token_mask.dtype == torch.bool:
            token_mask = token_mask.view(torch.uint8)
        _need(token_mask, torch.uint8, (T,), "token_mask")
    dev = logits.device
    o = {"idx": torch.empty(T, k, dtype=torch.int32, device=dev),
         "prob": torch.empty(T, k, dtype=torch.float32, device=dev)}
    load = None
    if with_load:
        load = o["load"] = torch.empty(n, dtype=torch.int32, device=dev)
    L.check(L.load().moe_router_fwd(logits.data_ptr(), b16, _ptr(bias), _ptr(token_mask), T, n, k, C.byref(params),
                                    o["idx"].data_ptr(), o["prob"].data_ptr(), _ptr(load), _cur(logits)), "moe_router_fwd")
    return o


def router_bwd(logits, idx, dprob, params: L.RouterParams):
    """dlogits [T, n] (in the logits' type) from dprob [T, k] f32, the gradient
    of the weights that router returned with idx [T, k]."""
    b16 = _logits(logits)
    T, n = logits.shape
    k = _need2(idx, torch.int32, "idx")[1]
    _need(idx, torch.int32, (T, k), "idx")
    _need(dprob, torch.float32, (T, k), "dprob")
    d = torch.empty_like(logits)
    L.check(L.load().moe_router_bwd(logits.data_ptr(), b16, idx.data_ptr(), dprob.data_ptr(), T, n, k,
                                    C.byref(params), d.data_ptr(), _cur(logits)), "moe_router_bwd")
    return d


def quantize_mxfp4(src, col: bool = False, status=None):
    """MXFP4 form of a weight src [G, R, C] bf16: (q, s) with q [G, N, Kp/2]
    uint8 (packed codes, Kp = K rounded up to 128) and s the E8M0 scales in the
    tensor-core order (flat uint8).  Blocks run along C (N = R, K = C), or with
    col=True along R (N = C, K = R; the transposed form)."""
    lib = L.load()
    _need(src, torch.bfloat16, None, "src")
    if src.dim() != 3:
        raise ValueError(f"src: [G, R, C] is needed, got {tuple(src.shape)}")
    G, R, Cc = src.shape
    N, K = (Cc, R) if col else (R, Cc)
    q = torch.empty(G, N, (K + 127) // 128 * 64, dtype=torch.uint8, device=src.device)
    s = torch.empty(_size("moe_mxfp4_scale_bytes", G, N, K), dtype=torch.uint8, device=src.device)
    L.check(lib.moe_quantize_mxfp4(src.data_ptr(), G, R, Cc, int(col), q.data_ptr(), s.data_ptr(), _ptr(status),
                                   _cur(src)), "moe_quantize_mxfp4")
    return q, s


@functools.lru_cache(maxsize=1024)
def _size(name: str, *dims) -> int:
    """A *_bytes / *_workspace_size entry point: host arithmetic on the shape, asked once per shape."""
    return getattr(L.load(), name)(*dims)


def _mxfp4(q, s, K, what):
    """Checks an MXFP4 weight of contraction length K; returns (G, N)."""
    _need(q, torch.uint8, None, what)
    shape = q.shape
    if len(shape) != 3 or shape[2] != (K + 127) // 128 * 64:
        raise ValueError(f"{what}: [G, N, {(K + 127) // 128 * 64}] codes are needed, got {tuple(shape)}")
    G, N = shape[0], shape[1]
    _need(s, torch.uint8, (_size("moe_mxfp4_scale_bytes", G, N, K),), what)
    return G, N


def dequantize_mxfp4(q, s, K: int):
    """The bf16 values [G, N, K] of an MXFP4 weight (q, s)."""
    G, N = _mxfp4(q, s, K, "q")
    o = torch.empty(G, N, K, dtype=torch.bfloat16, device=q.device)
    L.check(L.load().moe_dequantize_mxfp4(q.data_ptr(), s.data_ptr(), G, N, K, o.data_ptr(), _cur(q)),
            "moe_dequantize_mxfp4")
    return o


def _rows_mxfp8(xq, xs, what):
    R, K = _need2(xq, torch.uint8, what)
    _need(xs, torch.uint8, (R, K // 32), what)
    return R, K


def _groups(counts, offsets, E):
    _need(counts, torch.int32, (E,), "counts")
    _need(offsets, torch.int32, (E + 1,), "offsets")


def _outputs(out_mode, R_cap, N, dev, with_col):
    """Output tensors of a fused epilogue and the moe_act_out_t that names them."""
    o, ao, new, u8 = {}, L.ActOut(), torch.empty, torch.uint8
    if out_mode == L.OUT_MXFP8:
        o["q_row"] = new(R_cap, N, dtype=u8, device=dev)
        o["s_row"] = new(R_cap, N // 32, dtype=u8, device=dev)
        if with_col:
            o["q_col"] = new(N, R_cap, dtype=u8, device=dev)
            o["s_col"] = new(N, R_cap // 32, dtype=u8, device=dev)
    else:
        o["y"] = new(R_cap, N, dtype=torch.bfloat16, device=dev)
        if out_mode == L.OUT_NVFP4:
            o["amax"] = torch.empty(1, dtype=torch.float32, device=dev)
    for k, v in o.items():
        setattr(ao, k, v.data_ptr())
    return o, ao


def fc2_fwd_mxfp4(Aq, As, Wq, Ws, counts, offsets, sm_margin: int = 0, status=None, out=None,
                  out_mode: int = L.OUT_BF16, with_col: bool = True):
    """GroupGemm on MXFP8 rows and an MXFP4 weight: y [R_cap, N] =
    A [R_cap, K] . W[e]^T per expert, A as codes and scales [R_cap, K/32], W
    [E, N, K] as quantize_mxfp4 writes it.  Returns the bf16 tensor y, or (out_mode) the
    dict of MXFP8 or NVFP4-mode outputs as fc2_fwd does."""
    R_cap, K = _rows_mxfp8(Aq, As, "A")
    E, N = _mxfp4(Wq, Ws, K, "W")
    _groups(counts, offsets, E)
    dev = Aq.device
    if out is not None:
        o, ao = {"y": _need(out, torch.bfloat16, (R_cap, N), "out")}, L.ActOut(y=out.data_ptr())
    else:
        o, ao = _outputs(out_mode, R_cap, N, dev, with_col)
    st = status if status is not None else new_status(dev)
    a_in = L.InT(L.IN_MXFP8, Aq.data_ptr(), As.data_ptr(), None)
    w_in = L.InT(L.IN_MXFP4, Wq.data_ptr(), Ws.data_ptr(), None)
    nbytes = _size("moe_grouped_mxfp4_workspace_size", E, K, R_cap)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    L.check(L.load().moe_grouped_fc2_fwd(C.byref(a_in), C.byref(w_in), counts.data_ptr(), offsets.data_ptr(), E, K, N,
                                         R_cap, out_mode, C.byref(ao), ws.data_ptr(), nbytes, sm_margin,
                                         st.data_ptr(), _cur(Aq)), "moe_grouped_fc2_fwd (MXFP4)")
    o["status"] = st
    return o["y"] if out_mode == L.OUT_BF16 else o


def fc1_fwd_mxfp4(xq, xs, W1q, W1s, counts, offsets, F: int, params: L.GluParams, out_mode: int = L.OUT_MXFP8,
                  b1p=None, row_scale=None, save_pre: bool = True, with_col: bool = True, sm_margin: int = 0,
                  status=None) -> dict:
    """fc1_fwd_mxfp8 with an MXFP4 weight: W1q, W1s the MXFP4 form of the
    packed W1p [E, N1, H] (quantize_mxfp4)."""
    R_cap, H = _rows_mxfp8(xq, xs, "x")
    E, N1 = _mxfp4(W1q, W1s, H, "W1")
    _groups(counts, offsets, E)
    if N1 != (F if params.act == L.ACT["srelu"] else 2 * F):
        raise ValueError(f"W1: {N1} rows do not match F = {F}")
    if b1p is not None:
        _need(b1p, torch.bfloat16, (E, N1), "b1p")
    if row_scale is not None:
        _need(row_scale, torch.float32, (R_cap,), "row_scale")
    dev = xq.device
    o, ao = _outputs(out_mode, R_cap, F, dev, with_col)
    if save_pre:
        o["pre"] = torch.empty(R_cap, N1, dtype=torch.bfloat16, device=dev)
        ao.pre = o["pre"].data_ptr()
    st = status if status is not None else new_status(dev)
    nbytes = _size("moe_grouped_mxfp4_workspace_size", E, H, R_cap)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    L.check(L.load().moe_grouped_fc1_glu_quant_fwd_mxfp4(
        xq.data_ptr(), xs.data_ptr(), W1q.data_ptr(), W1s.data_ptr(), _ptr(b1p), _ptr(row_scale), counts.data_ptr(),
        offsets.data_ptr(), E, H, F, R_cap, C.byref(params), out_mode, C.byref(ao), ws.data_ptr(), nbytes, sm_margin,
        st.data_ptr(), _cur(xq)), "moe_grouped_fc1_glu_quant_fwd_mxfp4")
    o["status"] = st
    return o


def route_permute_mxfp8(xq, xs, topk_idx, topk_prob, E: int, R_cap: int, expert_begin: int = 0, status=None) -> dict:
    """route_permute for MXFP8 rows xq [T, H], xs [T, H/32]: the routing tensors
    and xq_perm [R_cap, H], xs_perm [R_cap, H/32]."""
    T, H = _rows_mxfp8(xq, xs, "x")
    k = _need2(topk_idx, torch.int32, "topk_idx")[1]
    _need(topk_idx, torch.int32, (T, k), "topk_idx")
    _need(topk_prob, torch.float32, (T, k), "topk_prob")
    dev, i32, u8 = xq.device, torch.int32, torch.uint8
    o = {
        "xq_perm": torch.empty(R_cap, H, dtype=u8, device=dev),
        "xs_perm": torch.empty(R_cap, H // 32, dtype=u8, device=dev),
        "row_of": torch.empty(T * k, dtype=i32, device=dev),
        "tok_of": torch.empty(R_cap, dtype=i32, device=dev),
        "prob_perm": torch.empty(R_cap, dtype=torch.float32, device=dev),
        "counts": torch.empty(E, dtype=i32, device=dev),
        "offsets": torch.empty(E + 1, dtype=i32, device=dev),
    }
    n = _size("moe_route_workspace_size", T, k, E)
    ws = torch.empty(n, dtype=u8, device=dev)
    st = status if status is not None else new_status(dev)
    L.check(L.load().moe_route_permute_mxfp8(
        xq.data_ptr(), xs.data_ptr(), topk_idx.data_ptr(), topk_prob.data_ptr(), T, H, k, expert_begin, E, R_cap,
        o["xq_perm"].data_ptr(), o["xs_perm"].data_ptr(), o["row_of"].data_ptr(), o["tok_of"].data_ptr(),
        o["prob_perm"].data_ptr(), o["counts"].data_ptr(), o["offsets"].data_ptr(), ws.data_ptr(), n, st.data_ptr(),
        _cur(xq)), "moe_route_permute_mxfp8")
    o["status"] = st
    return o
