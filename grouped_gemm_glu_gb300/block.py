"""The expert MLP with what stands in front of it: residual addition and RMS
norm, the router's product and choice, then the experts.

  MoeBlock   one training step of the block around a MoeLayer:
             norm -> router -> expert MLP, and the backward of all three
  MoeServer  the block's forward for serving, with the experts' weights in
             MXFP4: norm (bf16 and MXFP8 rows) -> router -> gather of the
             MXFP8 rows -> up projection with the activation -> down
             projection -> combine

Either may have low-rank adapters beside its experts, one per request
(Adapters): out = experts(y) + s_a B_a^T A_a y for the normed row y of each
token with an adapter a, the same for every expert.  MoeBlock.optimizer and
MoeBlock.update take the gradients of a step to the block's weights, the
adapters' or all.

Both issue library calls on the current stream and read nothing back, so a
step can be captured in a CUDA graph.  The router's product (logits =
y . Wr^T and its gradients) is a plain matrix product of a small weight and is
left to torch.  The logits keep the product's 32 bits: rounded to bf16,
neighbouring logits of hundreds of experts become equal and the lower index
wins.  (8192 x 7168 with 256 experts: 25.9 us against 25.6 with bf16 logits.)
"""
from __future__ import annotations

import torch

from . import lib as L
from . import ops
from .optim import AdamW


class Adapters:
    """G low-rank adapters of rank r beside the experts: A and B [G, r, H] bf16,
    scale [G] f32 (alpha / r, often).  Adapters of lower ranks are padded with
    zero rows.  A freshly made adapter has a zero B.  Forward and backward keep
    them apart; an optimizer over them does not: A and B are one tensor each, so
    that adapters without rows in a batch decay and move by their momentum as well,
    and max_norm scales all by one norm."""

    def __init__(self, A, B, scale):
        bf = torch.bfloat16
        for w, what in ((A, "A"), (B, "B")):
            if ops._need(w, bf, None, what).dim() != 3:
                raise ValueError(f"{what}: three dimensions are needed, got {tuple(w.shape)}")
        G, r, H = A.shape
        ops._need(B, bf, (G, r, H), "B")
        ops._need(scale, torch.float32, (G,), "scale")
        self.A, self.B, self.scale, self.H = A, B, scale, H

    def _beside(self, H: int):
        if self.H != H:
            raise ValueError(f"adapters of width {self.H} do not fit a block of width {H}")


def _need_adapter(adapter, adapters, T: int):
    if adapters is None:
        raise ValueError("adapter: this block has no adapters")
    ops._need(adapter, torch.int32, (T,), "adapter")


def _need_router(gamma, Wr, H: int):
    ops._need(gamma, torch.bfloat16, (H,), "gamma")
    if not Wr.is_cuda or Wr.dtype != torch.bfloat16 or Wr.dim() != 2 or Wr.shape[1] != H:  # (strides are torch's to follow)
        raise ValueError(f"Wr: [n, {H}] bf16 on a CUDA device is needed, got {tuple(Wr.shape)} {Wr.dtype}")


def _logits(y, Wr):
    """y . Wr^T, f32: the factors are bf16, their products exact, the sums f32."""
    return torch.mm(y, Wr.t(), out_dtype=torch.float32)


class MoeBlock:
    def __init__(self, layer, gamma, Wr, router: L.RouterParams, bias=None, eps: float = 1e-5, adapters=None):
        """layer: a MoeLayer; gamma [H] and Wr [n, H] bf16; router: how experts
        are chosen; bias [n] f32: the balance bias of the choice; adapters: an
        Adapters of the layer's width."""
        _need_router(gamma, Wr, layer.H)
        if adapters is not None:
            adapters._beside(layer.H)
        self.adapters, self.adapter, self.opt = adapters, None, None
        self.layer, self.gamma, self.Wr, self.router, self.bias, self.eps = layer, gamma, Wr, router, bias, eps

    def forward(self, x, residual=None, token_mask=None, adapter=None):
        """x [T, H] bf16 (the previous sublayer's output), residual [T, H] the
        stream it is added to; T is the layer's, other sizes are refused.
        adapter [T] int32: each token's adapter (-1: none; a token that
        token_mask takes from the experts keeps its adapter); the backward
        reads it again.
        Returns (out [T, H], h [T, H]): the experts' output and the new stream,
        the next sublayer's x and residual.  out is the layer's own buffer: the
        next forward overwrites it."""
        ly = self.layer
        ops._need(x, torch.bfloat16, (ly.T, ly.H), "x")
        if adapter is not None:
            _need_adapter(adapter, self.adapters, ly.T)
        n = ops.rmsnorm(x, self.gamma, self.eps, residual=residual)
        self.h = n["h"] if residual is not None else x
        self.y, self.rstd = n["y"], n["rstd"]
        self.logits = _logits(self.y, self.Wr)
        r = ops.router(self.logits, ly.k, self.router, bias=self.bias, token_mask=token_mask)
        self.idx, self.prob, self.load = r["idx"], r["prob"], r["load"]
        ly.run(ly.forward_calls(self.y, self.idx, self.prob))
        self.adapter = adapter
        if adapter is not None:
            ad = self.adapters
            self.low = ops.lora(self.y, ad.A, ad.B, adapter, ad.scale, base=ly.out, out=ly.out, status=ly.status)["h"]
        return ly.out, self.h

    def backward(self, dout, dh=None) -> dict:
        """dout, dh: the gradients arriving at forward's two outputs.  Returns
        dx (the gradient of x and of the residual alike), dgamma, dWr, dW1
        (packed rows), dW2 and, with an FC1 bias, db1 (packed), with adapters in
        the forward dA and dB.  dW1, dW2 and db1 are the layer's own buffers: the
        next backward overwrites them."""
        ly = self.layer
        ops._need(dout, torch.bfloat16, (ly.T, ly.H), "dout")
        if dh is not None:
            ops._need(dh, torch.bfloat16, (ly.T, ly.H), "dh")
        ly.run(ly.backward_calls(dout))
        # f32 up to its products, there an operand in bf16 like y and Wr: an error of 2^-9 of each element,
        # independent from one to the next, beside the 3.6% of the experts' MXFP8 operands behind dprob
        dlogits = ops.router_bwd(self.logits, self.idx, ly.dprob, self.router).to(torch.bfloat16)
        dy = torch.addmm(ly.dx, dlogits, self.Wr)  # the two uses of y: the experts' rows and the logits
        dA = dB = None
        if self.adapter is not None:  # (a third use of y)
            ad = self.adapters
            _, dA, dB = ops.lora_bwd(dout, self.y, self.low, ad.A, ad.B, self.adapter, ad.scale, base=dy, out=dy,
                                     status=ly.status)
        dx, dgamma = ops.rmsnorm_bwd(dy, self.h, self.gamma, self.rstd, dres=dh)
        g = {"dx": dx, "dgamma": dgamma, "dWr": dlogits.t() @ self.y, "dW1": ly.dW1, "dW2": ly.dW2, "db1": ly.db1}
        return {**g, "dA": dA, "dB": dB} if dA is not None else g

    def _weights(self, train: str):
        """(gradient's key, weight, its gradient's type, whether it decays)"""
        ly, f32, bf = self.layer, torch.float32, torch.bfloat16
        own = [("dgamma", self.gamma, f32, False), ("dWr", self.Wr, bf, True), ("dW1", ly.W1p, bf, True),
               ("dW2", ly.W2, bf, True)] + ([("db1", ly.b1p, f32, False)] if ly.b1p is not None else [])
        low = [("dA", self.adapters.A, bf, True), ("dB", self.adapters.B, bf, True)] if self.adapters is not None else []
        return {"all": own + low, "block": own, "adapters": low}[train]

    def optimizer(self, lr: float, train: str = "all", weight_decay: float = 0.01, **kw) -> AdamW:
        """An AdamW over the block's weights (train="block"), its adapters'
        ("adapters") or both ("all"), which update then steps; gamma and the
        bias do not decay.  The weights are updated where they are: gamma, Wr, W2,
        the adapters, and the layer's packed copies of W1 and b1 (layer.W1p,
        layer.b1p; ops.repack_fc1(..., inverse=True) gives the plain rows).
        max_norm: by the norm over this block's tensors, in a shard of the experts
        over that shard's alone: gamma and Wr, which every shard has, would then
        part.  Shards leave max_norm out."""
        if train not in ("all", "block", "adapters"):
            raise ValueError(f'train: "all", "block" or "adapters" is needed, got {train!r}')
        if train == "adapters" and self.adapters is None:
            raise ValueError("train: this block has no adapters")
        w = self._weights(train)
        self.trained = [k for k, *_ in w]
        self.opt = AdamW([t for _, t, *_ in w], lr=lr, weight_decay=[weight_decay if d else 0.0 for *_, d in w],
                         grad_dtype=[k for _, _, k, _ in w], **kw)
        return self.opt

    def update(self, grads: dict):
        """One step of optimizer()'s AdamW with what backward returned; returns
        the gradients' norm if the optimizer clips."""
        if self.opt is None:
            raise ValueError("update: optimizer() comes first")
        missing = [k for k in self.trained if grads.get(k) is None]
        if missing:
            raise ValueError(f"update: the gradients lack {missing} (a forward without adapters has none for them)")
        return self.opt.step([grads[k] for k in self.trained])


class MoeServer:
    def __init__(self, W1, W2, gamma, Wr, k: int, router: L.RouterParams, params: L.GluParams, b1=None, bias=None,
                 eps: float = 1e-5, expert_begin: int = 0, adapters=None):
        """W1 [E, 2F, H] (rows: input | gate) and W2 [E, F, H] bf16 are cast to
        MXFP4 here, once; b1 [E, 2F] bf16; gamma, Wr, router, bias and eps as
        for MoeBlock.  A shard: W1, W2 and b1 hold E of Wr's n experts, from
        expert_begin on; the others' part of the output is left to their shards.
        adapters: an Adapters of this width (of one shard only: their part of the
        output is not split)."""
        bf = torch.bfloat16
        for w, what in ((W1, "W1"), (W2, "W2")):
            if ops._need(w, bf, None, what).dim() != 3:
                raise ValueError(f"{what}: three dimensions are needed, got {tuple(w.shape)}")
        self.E, N1, self.H = W1.shape
        self.F, self.k = W2.shape[1], k
        ops._need(W2, bf, (self.E, self.F, self.H), "W2")
        if b1 is not None:
            ops._need(b1, bf, (self.E, N1), "b1")
        _need_router(gamma, Wr, self.H)
        if N1 != 2 * self.F or params.act in (L.ACT["srelu"], L.ACT["none"]):
            raise ValueError("a gated activation and W1 [E, 2F, H] are needed")
        if not 0 <= expert_begin < Wr.shape[0]:
            raise ValueError(f"expert_begin: one of the {Wr.shape[0]} experts is needed, got {expert_begin}")
        self.gamma, self.Wr, self.router, self.params, self.bias, self.eps = gamma, Wr, router, params, bias, eps
        self.expert_begin = expert_begin
        if adapters is not None:
            adapters._beside(self.H)
        self.adapters = adapters
        self.b1p = ops.repack_fc1(b1.unsqueeze(2)).squeeze(2).contiguous() if b1 is not None else None
        self.status = ops.new_status(W1.device)
        self.W1q, self.W1s = ops.quantize_mxfp4(ops.repack_fc1(W1), status=self.status)
        self.W2q, self.W2s = ops.quantize_mxfp4(W2, col=True, status=self.status)

    def rows(self, T: int) -> int:
        """Rows the permuted buffers of T tokens need: every assignment and up
        to 31 pad rows per expert that has one, rounded up to 128."""
        n = T * min(self.k, self.E)
        return (n + 31 * min(self.E, n) + 127) // 128 * 128

    def step(self, x, residual=None, token_mask=None, adapter=None):
        """(out [T, H], h [T, H]) as MoeBlock.forward, for one decoded token per
        sequence or a whole prompt; an empty batch gives empty results."""
        T = x.shape[0]
        if adapter is not None:
            _need_adapter(adapter, self.adapters, T)
        n = ops.rmsnorm(x, self.gamma, self.eps, residual=residual, mxfp8=True, with_rstd=False)
        h = n["h"] if residual is not None else x
        if T == 0:
            return torch.empty_like(x), h  # (the routing takes no empty batch)
        r = ops.router(_logits(n["y"], self.Wr), self.k, self.router, bias=self.bias, token_mask=token_mask,
                       with_load=False)
        p = ops.route_permute_mxfp8(n["q"], n["s"], r["idx"], r["prob"], self.E, self.rows(T),
                                    expert_begin=self.expert_begin, status=self.status)
        a = ops.fc1_fwd_mxfp4(p["xq_perm"], p["xs_perm"], self.W1q, self.W1s, p["counts"], p["offsets"], self.F,
                              self.params, b1p=self.b1p, save_pre=False, with_col=False, status=self.status)
        y = ops.fc2_fwd_mxfp4(a["q_row"], a["s_row"], self.W2q, self.W2s, p["counts"], p["offsets"],
                              status=self.status)
        out = ops.unpermute_combine(y, p["row_of"], r["prob"])
        if adapter is not None:
            ad = self.adapters
            ops.lora(n["y"], ad.A, ad.B, adapter, ad.scale, base=out, out=out, with_h=False, status=self.status)
        return out, h
