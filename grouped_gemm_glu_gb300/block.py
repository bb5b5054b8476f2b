"""The expert MLP with what stands in front of it: residual addition and RMS
norm, the router's product and choice, then the experts.

  MoeBlock   one training step of the block around a MoeLayer:
             norm -> router -> expert MLP, and the backward of all three
  MoeServer  the block's forward for serving, with the experts' weights in
             MXFP4: norm (bf16 and MXFP8 rows) -> router -> gather of the
             MXFP8 rows -> up projection with the activation -> down
             projection -> combine

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


def _need_router(gamma, Wr, H: int):
    ops._need(gamma, torch.bfloat16, (H,), "gamma")
    if not Wr.is_cuda or Wr.dtype != torch.bfloat16 or Wr.dim() != 2 or Wr.shape[1] != H:  # (strides are torch's to follow)
        raise ValueError(f"Wr: [n, {H}] bf16 on a CUDA device is needed, got {tuple(Wr.shape)} {Wr.dtype}")


def _logits(y, Wr):
    """y . Wr^T, f32: the factors are bf16, their products exact, the sums f32."""
    return torch.mm(y, Wr.t(), out_dtype=torch.float32)


class MoeBlock:
    def __init__(self, layer, gamma, Wr, router: L.RouterParams, bias=None, eps: float = 1e-5):
        """layer: a MoeLayer; gamma [H] and Wr [n, H] bf16; router: how experts
        are chosen; bias [n] f32: the balance bias of the choice."""
        _need_router(gamma, Wr, layer.H)
        self.layer, self.gamma, self.Wr, self.router, self.bias, self.eps = layer, gamma, Wr, router, bias, eps

    def forward(self, x, residual=None, token_mask=None):
        """x [T, H] bf16 (the previous sublayer's output), residual [T, H] the
        stream it is added to; T is the layer's, other sizes are refused.
        Returns (out [T, H], h [T, H]): the experts' output and the new stream,
        the next sublayer's x and residual.  out is the layer's own buffer: the
        next forward overwrites it."""
        ly = self.layer
        ops._need(x, torch.bfloat16, (ly.T, ly.H), "x")
        n = ops.rmsnorm(x, self.gamma, self.eps, residual=residual)
        self.h = n["h"] if residual is not None else x
        self.y, self.rstd = n["y"], n["rstd"]
        self.logits = _logits(self.y, self.Wr)
        r = ops.router(self.logits, ly.k, self.router, bias=self.bias, token_mask=token_mask)
        self.idx, self.prob, self.load = r["idx"], r["prob"], r["load"]
        ly.run(ly.forward_calls(self.y, self.idx, self.prob))
        return ly.out, self.h

    def backward(self, dout, dh=None) -> dict:
        """dout, dh: the gradients arriving at forward's two outputs.  Returns
        dx (the gradient of x and of the residual alike), dgamma, dWr, dW1
        (packed rows), dW2 and, with an FC1 bias, db1 (packed).  dW1, dW2 and db1
        are the layer's own buffers: the next backward overwrites them."""
        ly = self.layer
        ops._need(dout, torch.bfloat16, (ly.T, ly.H), "dout")
        if dh is not None:
            ops._need(dh, torch.bfloat16, (ly.T, ly.H), "dh")
        ly.run(ly.backward_calls(dout))
        # f32 up to its products, there an operand in bf16 like y and Wr: an error of 2^-9 of each element,
        # independent from one to the next, beside the 3.6% of the experts' MXFP8 operands behind dprob
        dlogits = ops.router_bwd(self.logits, self.idx, ly.dprob, self.router).to(torch.bfloat16)
        dy = torch.addmm(ly.dx, dlogits, self.Wr)  # the two uses of y: the experts' rows and the logits
        dx, dgamma = ops.rmsnorm_bwd(dy, self.h, self.gamma, self.rstd, dres=dh)
        return {"dx": dx, "dgamma": dgamma, "dWr": dlogits.t() @ self.y, "dW1": ly.dW1, "dW2": ly.dW2, "db1": ly.db1}


class MoeServer:
    def __init__(self, W1, W2, gamma, Wr, k: int, router: L.RouterParams, params: L.GluParams, b1=None, bias=None,
                 eps: float = 1e-5, expert_begin: int = 0):
        """W1 [E, 2F, H] (rows: input | gate) and W2 [E, F, H] bf16 are cast to
        MXFP4 here, once; b1 [E, 2F] bf16; gamma, Wr, router, bias and eps as
        for MoeBlock.  A shard: W1, W2 and b1 hold E of Wr's n experts, from
        expert_begin on; the others' part of the output is left to their shards."""
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
        self.b1p = ops.repack_fc1(b1.unsqueeze(2)).squeeze(2).contiguous() if b1 is not None else None
        self.status = ops.new_status(W1.device)
        self.W1q, self.W1s = ops.quantize_mxfp4(ops.repack_fc1(W1), status=self.status)
        self.W2q, self.W2s = ops.quantize_mxfp4(W2, col=True, status=self.status)

    def rows(self, T: int) -> int:
        """Rows the permuted buffers of T tokens need: every assignment and up
        to 31 pad rows per expert that has one, rounded up to 128."""
        n = T * min(self.k, self.E)
        return (n + 31 * min(self.E, n) + 127) // 128 * 128

    def step(self, x, residual=None, token_mask=None):
        """(out [T, H], h [T, H]) as MoeBlock.forward, for one decoded token per
        sequence or a whole prompt; an empty batch gives empty results."""
        T = x.shape[0]
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
        return ops.unpermute_combine(y, p["row_of"], r["prob"]), h
