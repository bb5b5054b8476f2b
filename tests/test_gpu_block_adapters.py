"""Adapters and the optimizer in the block: a training step with adapters
against the step without them plus the adapters' formulas in float64, the
update against the AdamW formula, the whole of it in a captured graph, and the
adapted serving forward.

Tolerances: b = 2^-8 is half a bf16 step.  The adapters' part is added to the
experts' bf16 output and rounded again, its h = bf16(s A y): with u = h B,
|out - (base + u)| <= b |base + u| (1 + b) + 2 b sum |h B| (fp32 sums of at
most 256 terms are below b / 2 of their size and taken in).  dy gets the
adapters' part in the same way; the norm's backward is linear in dy, so the
two steps' dx and dgamma differ by its image of that part (computed by the same
backward from its float64 value, rounded to bf16: another b of it), plus the
roundings of both dx: compared in the 2-norm, 4 b of the larger one."""
import numpy as np
import pytest
import torch

from adamw_ref import step as adamw_step
from grouped_gemm_glu_gb300 import lib as L
from grouped_gemm_glu_gb300 import ops, synth
from grouped_gemm_glu_gb300.block import Adapters, MoeBlock, MoeServer
from grouped_gemm_glu_gb300.layer import MoeLayer

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
T, H, E, K, F, G, R = 192, 256, 8, 2, 128, 3, 16
B8 = 2.0 ** -8
F64 = torch.float64


class Setup:
    def __init__(self, seed=4, bias=False, **kw):
        rng = np.random.default_rng(seed)
        bf = lambda *s, sc=1.0: synth._bf16(sc * rng.standard_normal(s)).to(DEV)
        self.x, self.res, self.dout, self.dh = bf(T, H), bf(T, H, sc=2.0), bf(T, H), bf(T, H)
        self.gamma = synth._bf16(1 + 0.1 * rng.standard_normal(H)).to(DEV)
        self.Wr, self.W1, self.W2 = bf(E, H, sc=H ** -0.5 * 2), bf(E, 2 * F, H, sc=H ** -0.5), bf(E, F, H, sc=F ** -0.5)
        self.b1 = bf(E, 2 * F, sc=0.02) if bias else None
        self.ad = Adapters(bf(G, R, H, sc=H ** -0.5), bf(G, R, H, sc=R ** -0.5),
                           torch.tensor([0.5, 1.0, 2.0], device=DEV))
        self.prm = L.router_params("softmax", renorm=True)
        self.layer = MoeLayer(self.W1, self.W2, T, K, (T * K + 31 * E + 127) // 128 * 128, L.glu_params("swiglu"), b1=self.b1)
        self.block = MoeBlock(self.layer, self.gamma, self.Wr, self.prm, adapters=self.ad, **kw)
        idx = rng.integers(-1, G, T)
        idx[60:150] = 2  # a prompt among single tokens
        self.idx = torch.from_numpy(idx.astype(np.int32)).to(DEV)


def _low(y, ad, idx):
    """(h, u, sum |h B|) of the adapters' part, float64 on the CPU."""
    y, A, B, s = y.cpu().to(F64), ad.A.cpu().to(F64), ad.B.cpu().to(F64), ad.scale.cpu().to(F64)
    h, u, size = torch.zeros(T, R, dtype=F64), torch.zeros(T, H, dtype=F64), torch.zeros(T, H, dtype=F64)
    for a in range(G):
        t = torch.nonzero(idx.cpu() == a).view(-1)
        h[t] = s[a] * (y[t] @ A[a].T)
        u[t] = h[t] @ B[a]
        size[t] = h[t].abs() @ B[a].abs()
    return h, u, size


def _rel(a, b):
    a, b = a.detach().cpu().to(F64), b.detach().cpu().to(F64)
    return float((a - b).norm() / b.norm())


def test_training_step_with_adapters():
    s = Setup()
    blk = s.block
    out0, _ = blk.forward(s.x, s.res)
    out0 = out0.clone()
    g0 = blk.backward(s.dout, s.dh)
    g0 = {k: v.clone() for k, v in g0.items() if v is not None}
    assert "dA" not in g0
    out, _ = blk.forward(s.x, s.res, adapter=s.idx)
    out = out.clone()
    g = blk.backward(s.dout, s.dh)
    assert ops.read_status(s.layer.status) == 0
    h, u, size = _low(blk.y, s.ad, s.idx)
    want = out0.cpu().to(F64) + u
    assert bool(((out.cpu().to(F64) - want).abs() <= B8 * (1 + B8) * want.abs() + 2 * B8 * size).all())
    none = s.idx == -1
    assert torch.equal(out[none], out0[none])
    for k in ("dWr", "dW1", "dW2"):  # the experts' own gradients do not know of the adapters
        assert torch.equal(g[k], g0[k]), k
    # dA and dB from their formulas; the adapters' part of dy through the norm's backward
    dy, A, B, sc = (v.cpu().to(F64) for v in (s.dout, s.ad.A, s.ad.B, s.ad.scale))
    part = torch.zeros(T, H, dtype=F64)
    dA, dB = torch.zeros(G, R, H, dtype=F64), torch.zeros(G, R, H, dtype=F64)
    for a in range(G):
        t = torch.nonzero(s.idx.cpu() == a).view(-1)
        w = sc[a] * (dy[t] @ B[a].T)
        part[t] = w @ A[a]
        dA[a] = w.T @ blk.y.cpu().to(F64)[t]
        dB[a] = h[t].T @ dy[t]
    assert _rel(g["dA"], dA) < 2 * B8 and _rel(g["dB"], dB) < 2 * B8
    more, dgamma = ops.rmsnorm_bwd(part.to(torch.bfloat16).to(DEV), blk.h, s.gamma, blk.rstd)
    for got, base, add in ((g["dx"], g0["dx"], more), (g["dgamma"], g0["dgamma"], dgamma)):
        want = base.cpu().to(F64) + add.cpu().to(F64)
        assert float((got.cpu().to(F64) - want).norm()) <= 4 * B8 * float(max(want.norm(), base.cpu().to(F64).norm()))


@pytest.mark.parametrize("train,state,bias", [("all", "f32", True), ("block", "mxfp8", False), ("adapters", "f32", False)])
def test_update_is_adamw(train, state, bias):
    s = Setup(seed=5, bias=bias)
    blk = s.block
    opt = blk.optimizer(1e-2, train=train, weight_decay=0.1, betas=(0.9, 0.95), state=state, max_norm=1e3)
    names = ["dgamma", "dWr", "dW1", "dW2"] + (["db1"] if bias else [])
    low = ["dA", "dB"]
    assert blk.trained == {"all": names + low, "block": names, "adapters": low}[train]
    every = {"dgamma": s.gamma, "dWr": s.Wr, "dW1": s.layer.W1p, "dW2": s.W2, "dA": s.ad.A, "dB": s.ad.B}
    still = {k: v.clone() for k, v in every.items() if k not in blk.trained}
    for t in range(2):
        blk.forward(s.x, s.res, adapter=s.idx)
        g = blk.backward(s.dout, s.dh)
        master = [opt.master[at:at + w.numel()].clone() for w, at in zip(opt.weights, opt._at)]
        mom = [tuple(v.clone() for v in opt.moments(i)) for i in range(len(opt.weights))]
        norm = blk.update(g)
        total = sum(float(g[k].double().square().sum()) for k in blk.trained) ** 0.5
        assert abs(float(norm) - total) <= 1e-6 * total
        c = min(1.0, 1e3 / (total + 1e-6))
        for i, k in enumerate(blk.trained):
            wd = 0.0 if k in ("dgamma", "db1") else float(torch.tensor(0.1))
            w, m, v = adamw_step(master[i].cpu(), mom[i][0].cpu().view(-1), mom[i][1].cpu().view(-1), g[k].cpu().view(-1), t + 1,
                                 float(torch.tensor(1e-2)), (0.9, 0.95), 1e-8, wd, c)
            now = opt.master[opt._at[i]:opt._at[i] + w.numel()].cpu()
            # (5 fp32 roundings of w and 2^-18 of the step, which is at most lr / sqrt(1 - b2) large here)
            assert float((now.to(F64) - w).abs().max()) <= 5 * 2.0 ** -24 * float(w.abs().max()) + 2.0 ** -18 * 1e-2 * 5
            assert torch.equal(opt.weights[i].cpu().view(-1), now.to(torch.bfloat16))
    assert all(torch.equal(v, every[k]) for k, v in still.items())
    assert ops.read_status(s.layer.status) == 0


def test_captured_training_steps_equal_eager_ones():
    a, b = Setup(seed=6), Setup(seed=6)
    kw = dict(lr=1e-3, state="mxfp8", max_norm=1.0, seed=9)
    a.block.optimizer(**kw), b.block.optimizer(**kw)

    def train(s):
        s.block.forward(s.x, s.res, adapter=s.idx)
        return s.block.update(s.block.backward(s.dout, s.dh))

    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        train(a)  # the first step, outside the capture
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            norm = train(a)
    torch.cuda.synchronize()
    train(b)
    for i in range(3):
        new = torch.roll(b.x, i + 1, 0)
        a.x.copy_(new)
        b.x.copy_(new)
        a.idx.copy_(torch.roll(b.idx, 7, 0))
        b.idx.copy_(a.idx)
        g.replay()
        want = train(b)
        torch.cuda.synchronize()
        assert torch.equal(norm, want)
        assert all(torch.equal(x, y) for x, y in zip(a.block.opt.weights, b.block.opt.weights))
        assert all(torch.equal(v, b.block.opt.state_dict()[k]) for k, v in a.block.opt.state_dict().items())
    assert int(a.block.opt.t) == 4


@pytest.mark.parametrize("n", [1, 33, T])
def test_serving_with_adapters(n):
    s = Setup(seed=7)
    kw = dict(W1=s.W1, W2=s.W2, gamma=s.gamma, Wr=s.Wr, k=K, router=s.prm, params=L.glu_params("swiglu"))
    plain, adapted = MoeServer(**kw), MoeServer(**kw, adapters=s.ad)
    x, res, idx = s.x[:n].contiguous(), s.res[:n].contiguous(), s.idx[:n].contiguous()
    out0, h0 = plain.step(x, res)
    out, h = adapted.step(x, res, adapter=idx)
    assert torch.equal(h, h0) and ops.read_status(adapted.status) == 0
    y = ops.rmsnorm(x, s.gamma, residual=res)["y"]
    pad = lambda v, fill: torch.cat([v, torch.full((T - n, *v.shape[1:]), fill, dtype=v.dtype, device=DEV)])
    _, u, size = _low(pad(y, 0.0), s.ad, pad(idx, -1))
    want = out0.cpu().to(F64) + u[:n]
    assert bool(((out.cpu().to(F64) - want).abs() <= B8 * (1 + B8) * want.abs() + 2 * B8 * size[:n]).all())
    again, _ = adapted.step(x, res)
    assert torch.equal(again, out0)
    e, _ = adapted.step(x[:0], res[:0], adapter=idx[:0])
    assert e.shape == (0, H)


def test_refusals():
    s = Setup()
    b = s.block
    bf = torch.bfloat16
    z = lambda *sh, dt=bf: torch.zeros(*sh, dtype=dt, device=DEV)
    for args in ((z(G, R, H), z(G, R, 128), z(G, dt=torch.float32)), (z(R, H), z(R, H), z(G, dt=torch.float32)),
                 (z(G, R, H), z(G, R, H), z(G)), (z(G, R, H), z(G, R, H), z(2, dt=torch.float32))):
        with pytest.raises(ValueError):
            Adapters(*args)
    narrow = Adapters(z(G, R, 128), z(G, R, 128), z(G, dt=torch.float32))
    with pytest.raises(ValueError):
        MoeBlock(s.layer, s.gamma, s.Wr, s.prm, adapters=narrow)
    for bad in (s.idx.long(), s.idx[:5], s.idx.cpu()):
        with pytest.raises(ValueError):
            b.forward(s.x, s.res, adapter=bad)
    without = MoeBlock(s.layer, s.gamma, s.Wr, s.prm)
    with pytest.raises(ValueError):
        without.forward(s.x, s.res, adapter=s.idx)
    with pytest.raises(ValueError):
        without.optimizer(1e-3, train="adapters")
    with pytest.raises(ValueError):
        without.optimizer(1e-3, train="experts")
    with pytest.raises(ValueError):
        b.update({})
    b.optimizer(1e-3)
    b.forward(s.x, s.res)  # without adapters: no gradients for them
    with pytest.raises(ValueError):
        b.update(b.backward(s.dout))
    kw = dict(W1=s.W1, W2=s.W2, gamma=s.gamma, Wr=s.Wr, k=K, router=s.prm, params=L.glu_params("swiglu"))
    with pytest.raises(ValueError):
        MoeServer(**kw, adapters=narrow)
    with pytest.raises(ValueError):
        MoeServer(**kw).step(s.x, s.res, adapter=s.idx)
