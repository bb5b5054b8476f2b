"""The norm, the router and the experts together: a training step (MoeBlock)
against float64 autograd of the same block with the choice made on the GPU,
and the serving forward (MoeServer) against float64 on the values its MXFP4
weights stand for; the gather of MXFP8 rows against the cast of gathered rows.

Tolerances: rounding to E4M3 under a block scale has a relative error of at
most 2^-4, 2^-4 / sqrt(3) = 3.6% in the root mean square.  The training step's
output passes one product of two such operands (the activation and W2: 5.1%),
its dx and weight gradients two in a row at most (dFC1 with W1, dFC1 with x;
7.2%), and the router's gradients come from dprob, a product with that output
(5.1%).  Errors are compared in the 2-norm with 1.25 times these bounds.  In
the serving forward only the activation is rounded again (3.6%), and x itself
is rounded as the reference rounds it."""
import numpy as np
import pytest
import torch

from grouped_gemm_glu_gb300 import lib as L
from grouped_gemm_glu_gb300 import ops, synth
from grouped_gemm_glu_gb300.block import MoeBlock, MoeServer
from grouped_gemm_glu_gb300.layer import MoeLayer
from parity import np_

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _rel(a, b):
    a, b = a.detach().double().cpu(), b.detach().double().cpu()
    return float((a - b).norm() / b.norm())


def _unpack(g):
    """Packed FC1 rows (32 input, 32 gate per block of 64) -> input rows, gate rows."""
    E, N1, H = g.shape
    v = g.view(E, N1 // 64, 2, 32, H)
    return torch.cat([v[:, :, 0].reshape(E, N1 // 2, H), v[:, :, 1].reshape(E, N1 // 2, H)], 1)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid_groups"])
def test_training_step_matches_autograd(kind):
    T, H, E, k, F = 160, 256, 8, 2, 128
    rng = np.random.default_rng(4)
    bf = lambda *s, sc=1.0: synth._bf16(sc * rng.standard_normal(s)).to(DEV)
    x, res, gamma = bf(T, H), bf(T, H, sc=2.0), synth._bf16(1 + 0.1 * rng.standard_normal(H)).to(DEV)
    Wr, W1, W2 = bf(E, H, sc=H ** -0.5 * 2), bf(E, 2 * F, H, sc=H ** -0.5), bf(E, F, H, sc=F ** -0.5)
    dout, dh = bf(T, H), bf(T, H)
    bias = None
    if kind == "softmax":
        prm = L.router_params("softmax", renorm=True)
    else:
        prm = L.router_params("sigmoid", renorm=True, scale=2.5, n_group=4, topk_group=2, group_top=2)
        bias = torch.from_numpy((0.05 * rng.standard_normal(E)).astype(np.float32)).to(DEV)
    mask = torch.ones(T, dtype=torch.bool, device=DEV)
    mask[7] = mask[100] = False
    layer = MoeLayer(W1, W2, T, k, (T * k + 31 * E + 127) // 128 * 128, L.glu_params("swiglu"))
    blk = MoeBlock(layer, gamma, Wr, prm, bias=bias)
    out, h = blk.forward(x, res, mask)
    out, h = out.clone(), h.clone()
    g = blk.backward(dout, dh)
    torch.cuda.synchronize()
    assert ops.read_status(layer.status) == 0
    idx = blk.idx.cpu().long()
    assert bool((idx[7] == -1).all()) and int(blk.load.sum()) == (T - 2) * k

    D = torch.float64
    leaf = lambda t: t.detach().cpu().to(D).requires_grad_(True)
    xs, gm, wr, w1, w2 = leaf(x), leaf(gamma), leaf(Wr), leaf(W1), leaf(W2)
    hh = xs + res.cpu().to(D)
    y = hh / torch.sqrt((hh * hh).mean(1, keepdim=True) + 1e-5) * gm
    lg = y @ wr.t()
    on, at = idx >= 0, idx.clamp(min=0)
    if kind == "softmax":
        w = torch.softmax(torch.where(on, lg.gather(1, at), torch.tensor(-1e300, dtype=D)), 1)
    else:
        s = torch.sigmoid(lg).gather(1, at)
        w = 2.5 * s / s.sum(1, keepdim=True)
    w = torch.where(on, w, torch.zeros((), dtype=D))
    u = torch.einsum("th,efh->tef", y, w1)
    a = torch.nn.functional.silu(u[..., F:]) * u[..., :F]
    ye = torch.einsum("tef,efh->teh", a, w2)
    o = (w[..., None] * torch.take_along_dim(ye, at[..., None].expand(-1, -1, H), 1)).sum(1)
    ((o * dout.cpu().to(D)).sum() + (hh * dh.cpu().to(D)).sum()).backward()
    assert _rel(h, hh) < 2.0 ** -8
    assert _rel(out, o) < 1.25 * 0.051
    assert _rel(g["dx"], xs.grad) < 1.25 * 0.072
    assert _rel(g["dgamma"], gm.grad) < 1.25 * 0.072
    assert _rel(g["dWr"], wr.grad) < 1.25 * 0.072
    assert _rel(g["dW2"], w2.grad) < 1.25 * 0.072
    assert _rel(_unpack(g["dW1"].cpu().double()), w1.grad) < 1.25 * 0.072
    assert not out[7].any()  # a masked token gets nothing from the experts ...
    assert torch.equal(g["dx"][7], ops.rmsnorm_bwd(torch.zeros_like(x), blk.h, gamma, blk.rstd, dres=dh)[0][7])


@pytest.mark.parametrize("T", [1, 5, 200])
def test_server_matches_values(T):
    H, E, k, F = 320, 8, 3, 192
    rng = np.random.default_rng(T)
    bf = lambda *s, sc=1.0: synth._bf16(sc * rng.standard_normal(s)).to(DEV)
    x, res, gamma = bf(T, H), bf(T, H, sc=2.0), synth._bf16(1 + 0.1 * rng.standard_normal(H)).to(DEV)
    Wr, W1, W2, b1 = bf(E, H, sc=H ** -0.5 * 2), bf(E, 2 * F, H, sc=H ** -0.5), bf(E, F, H, sc=F ** -0.5), bf(E, 2 * F, sc=0.1)
    glu = L.glu_params("swiglu", alpha=1.702, up_offset=1.0, gate_lo=-7.0, gate_hi=7.0)
    s = MoeServer(W1, W2, gamma, Wr, k, L.router_params("softmax", renorm=True), glu, b1=b1)
    out, h = s.step(x, res)
    torch.cuda.synchronize()
    assert ops.read_status(s.status) == 0
    n = ops.rmsnorm(x, gamma, residual=res, mxfp8=True)
    assert torch.equal(h, n["h"])
    r = ops.router(n["y"] @ Wr.t(), k, L.router_params("softmax", renorm=True))
    D = torch.float64
    y = ops.dequantize_mxfp8(n["q"], n["s"]).cpu().to(D)
    w1 = _unpack(ops.dequantize_mxfp4(s.W1q, s.W1s, H).cpu().to(D))
    w2 = ops.dequantize_mxfp4(s.W2q, s.W2s, F).cpu().to(D)  # [E, H, F]
    idx, w = r["idx"].cpu().long(), r["prob"].cpu().to(D)
    u = torch.einsum("th,efh->tef", y, w1) + b1.cpu().to(D)[None]
    gt = u[..., F:].clamp(-7, 7)
    a = (u[..., :F] + 1) * gt * torch.sigmoid(1.702 * gt)
    ye = torch.einsum("tef,ehf->teh", a, w2)
    ref = (w[..., None] * torch.take_along_dim(ye, idx[..., None].expand(-1, -1, H), 1)).sum(1)
    assert _rel(out, ref) < 1.25 * 0.036


def test_server_step_replays_from_a_graph():
    T, H, E, k, F = 4, 256, 8, 2, 128
    rng = np.random.default_rng(11)
    bf = lambda *s, sc=1.0: synth._bf16(sc * rng.standard_normal(s)).to(DEV)
    s = MoeServer(bf(E, 2 * F, H, sc=H ** -0.5), bf(E, F, H, sc=F ** -0.5), bf(H), bf(E, H, sc=0.1), k,
                  L.router_params("softmax", renorm=True), L.glu_params("swiglu"))
    x, res = bf(T, H), bf(T, H)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        s.step(x, res)
        st.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            out, h = s.step(x, res)
    torch.cuda.synchronize()
    x.copy_(bf(T, H))
    res.copy_(bf(T, H))
    g.replay()
    torch.cuda.synchronize()
    want, wh = s.step(x, res)
    assert torch.equal(out, want) and torch.equal(h, wh) and ops.read_status(s.status) == 0


@pytest.mark.parametrize("T,H,k,E,begin", [(1, 32, 1, 4, 0), (77, 544, 4, 6, 3), (300, 256, 8, 16, 0)])
def test_gather_of_mxfp8_rows(T, H, k, E, begin):
    rng = np.random.default_rng(T)
    x = synth._bf16(rng.standard_normal((T, H))).to(DEV)
    idx = torch.from_numpy(np.stack([rng.choice(16, size=k, replace=False) for _ in range(T)]).astype(np.int32)).to(DEV)
    prob = torch.from_numpy(rng.random((T, k)).astype(np.float32)).to(DEV)
    R_cap = (T * k + 31 * E + 127) // 128 * 128
    q, s = ops.quantize_mxfp8(x)
    m = ops.route_permute_mxfp8(q, s, idx, prob, E, R_cap, expert_begin=begin)
    r = ops.route_permute(x, idx, prob, E, R_cap, expert_begin=begin)
    for key in ("counts", "offsets", "row_of"):
        assert torch.equal(m[key], r[key]), key
    R = int(r["offsets"][-1])
    for key in ("tok_of", "prob_perm"):
        assert torch.equal(m[key][:R], r[key][:R]), key
    wq, ws = ops.quantize_mxfp8(r["x_perm"])
    assert torch.equal(m["xq_perm"][:R], wq[:R]) and torch.equal(m["xs_perm"][:R], ws[:R])
    assert ops.read_status(m["status"]) == 0
    small = ops.route_permute_mxfp8(q, s, idx, prob, E, 32, expert_begin=begin)
    assert (ops.read_status(small["status"]) == L.MOE_ERR_CAPACITY) == (R > 32)
    with pytest.raises(ValueError):
        ops.route_permute_mxfp8(q, s, idx.long(), prob, E, R_cap)
    with pytest.raises(L.MoeError):
        ops.route_permute_mxfp8(q, s, idx, prob, E, R_cap + 1)
