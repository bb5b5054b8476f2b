"""The weights' update: AdamW over many tensors at once, with moments in 32 or
in 8 bits and optional clipping by the gradients' global norm: two launches a
step, three with clipping, for up to 4000 tensors.

  opt = AdamW(weights, lr=3e-4, weight_decay=0.1, max_norm=1.0, state="mxfp8")
  norm = opt.step(grads)

The step reads nothing back; count and learning rate live on the device, so it
can be captured in a CUDA graph and follows ``set_lr`` when it is replayed (the
gradients of a captured step keep their addresses).
"""
from __future__ import annotations

import array
import ctypes as C

import torch

from . import lib as L

_BLOCK = 32  # elements per scale; every tensor's state starts at a whole block of the flat buffers


class AdamW:
    def __init__(self, weights, lr: float, betas=(0.9, 0.999), eps: float = 1e-8, weight_decay=0.01, max_norm=None,
                 state: str = "f32", grad_dtype=None, seed: int = 0):
        """weights: contiguous CUDA tensors of one device, float32 or bfloat16,
        updated in place (parameters that require gradients too: the step is no
        part of what autograd records); a bfloat16 weight gets an f32 master here,
        which the step updates and rounds.  weight_decay: one number, or one per
        tensor.  max_norm: the gradients of a step are scaled down together to this
        2-norm, which is taken over this object's tensors alone: shards of one
        model that clip by max_norm each clip by their own norm, and what they hold
        copies of drifts apart; a step whose norm is not finite changes nothing.
        state: "f32" keeps m and v, "mxfp8" keeps m and sqrt(v) as E4M3 codes with a
        scale per 32 elements, rounded up or down by random bits that seed starts:
        right on average, but under normal gradients of a steady size the held
        sqrt(v) spreads by 12% (b2 = 0.95) to 15% (0.999) around the 32-bit one, the
        farthest of 65,536 elements to 0.55 and 1.8 of it.  grad_dtype: one type or one per tensor (default: the
        weight's).
        Every weight takes part in every step: zero gradients still decay it and
        move it by its momentum.
        A weight keeps its memory for as long as this object lives: one that is
        given another (w.data = ...) is no longer updated, by a step or a load.
        Steps of one object share their state and workspace and follow one another.
        Made once per set of weights: masters and addresses of a few hundred
        tensors take some milliseconds.

        Flat state, one stretch per tensor from a multiple of 32 on: m and v
        (float32, or uint8 codes with scales ms and vs), master (float32, where
        there are bfloat16 weights), t (int64, steps taken), lr (float32)."""
        ws = list(weights)
        for i, w in enumerate(ws):
            if not isinstance(w, torch.Tensor) or not w.is_cuda:
                raise ValueError(f"weights[{i}]: a CUDA tensor is needed")
            if w.dtype not in (torch.float32, torch.bfloat16):
                raise ValueError(f"weights[{i}]: float32 or bfloat16 is needed, got {w.dtype}")
            if not w.is_contiguous():
                raise ValueError(f"weights[{i}]: a contiguous tensor is needed")
            if w.device != ws[0].device:
                raise ValueError(f"weights[{i}]: lies on {w.device}, weights[0] on {ws[0].device}")
        spans = sorted((w.data_ptr(), w.data_ptr() + w.numel() * w.element_size(), i) for i, w in enumerate(ws) if w.numel())
        for (_, end, i), (begin, _, j) in zip(spans, spans[1:]):
            if begin < end:
                raise ValueError(f"weights[{i}] and weights[{j}] overlap")
        if state not in ("f32", "mxfp8"):
            raise ValueError(f'state: "f32" or "mxfp8" is needed, got {state!r}')
        if not (0.0 <= betas[0] < 1.0 and 0.0 <= betas[1] < 1.0):
            raise ValueError(f"betas: numbers in [0, 1) are needed, got {betas}")
        if not eps >= 0.0:
            raise ValueError(f"eps: a number >= 0 is needed, got {eps}")
        if max_norm is not None and not 0.0 < max_norm < float("inf"):
            raise ValueError(f"max_norm: a positive number is needed, got {max_norm}")
        n = len(ws)
        decay = list(weight_decay) if isinstance(weight_decay, (list, tuple)) else [weight_decay] * n
        kinds = list(grad_dtype) if isinstance(grad_dtype, (list, tuple)) else [
            w.dtype if grad_dtype is None else grad_dtype for w in ws]
        if len(decay) != n or len(kinds) != n:
            raise ValueError(f"weight_decay, grad_dtype: one value or {n} are needed")
        if any(not 0.0 <= d < float("inf") for d in decay):
            raise ValueError("weight_decay: numbers >= 0 are needed")
        if any(k not in (torch.float32, torch.bfloat16) for k in kinds):
            raise ValueError("grad_dtype: float32 or bfloat16 is needed")
        self.weights, self.state, self.max_norm = ws, state, max_norm
        self._memory = [w.detach() for w in ws]  # what the plan's addresses point at stays allocated
        self.device = dev = ws[0].device if ws else torch.device("cuda", torch.cuda.current_device())
        self._dtypes, self._shapes = kinds, [w.shape for w in ws]
        self._at = []
        total = 0
        for w in ws:
            self._at.append(total)
            total += (w.numel() + _BLOCK - 1) // _BLOCK * _BLOCK
        z = lambda k, dt: torch.zeros(k, dtype=dt, device=dev)
        f32, u8 = torch.float32, torch.uint8
        self.m, self.v = (z(total, f32), z(total, f32)) if state == "f32" else (z(total, u8), z(total, u8))
        self.ms, self.vs = (None, None) if state == "f32" else (z(total // _BLOCK, u8), z(total // _BLOCK, u8))
        self.master = z(total, f32) if any(w.dtype == torch.bfloat16 for w in ws) else None
        self.t, self.lr, self.norm = z(1, torch.int64), z(1, f32), z((), f32)
        self.set_lr(lr)
        size = self.m.element_size()
        self._rows = (L.AdamwTensor * max(n, 1))()
        for row, w, at, d, k in zip(self._rows, self._memory, self._at, decay, kinds):
            narrow = w.dtype == torch.bfloat16
            if narrow:
                self.master[at:at + w.numel()].copy_(w.view(-1))
            row.w, row.n = w.data_ptr(), w.numel()
            row.master = self.master.data_ptr() + 4 * at if narrow else None
            row.m, row.v = self.m.data_ptr() + size * at, self.v.data_ptr() + size * at
            if state == "mxfp8":
                row.m_scale, row.v_scale = self.ms.data_ptr() + at // _BLOCK, self.vs.data_ptr() + at // _BLOCK
            row.weight_decay, row.w_bf16, row.grad_bf16 = d, int(narrow), int(k == torch.bfloat16)
        lib = L.load()
        kind = L.MOMENTS[state]
        self._p = L.AdamwParams(betas[0], betas[1], eps, max_norm or 0.0, kind, seed & 0xFFFFFFFF)
        self._pref = C.byref(self._p)
        host = torch.zeros(max(lib.moe_adamw_plan_size(self._rows, n), 8), dtype=u8)
        L.check(lib.moe_adamw_plan(self._rows, n, kind, host.data_ptr(), host.numel()), "moe_adamw_plan")
        self._plan = host.to(dev)
        self._ws = torch.empty(lib.moe_adamw_workspace_size(n), dtype=u8, device=dev)

    def set_lr(self, lr: float):
        """The learning rate of the steps issued (or replayed) from here on."""
        if not 0.0 <= lr < float("inf"):
            raise ValueError(f"lr: a number >= 0 is needed, got {lr}")
        self.lr.fill_(lr)

    def step(self, grads):
        """One step with grads, one per weight in the weights' order, of their
        shapes and of grad_dtype, contiguous.  Returns the gradients' 2-norm before
        clipping (a float32 scalar, this object's own buffer) with max_norm, else None."""
        tensor, n, index = torch.Tensor, len(self._shapes), self.device.index
        try:  # (whole lists at a time: a few hundred tensors are checked in some tens of microseconds)
            fine = (len(grads) == n and [g.dtype for g in grads] == self._dtypes and [g.shape for g in grads] == self._shapes
                    and all(map(tensor.is_contiguous, grads)) and set(map(tensor.get_device, grads)) <= {index})
        except (AttributeError, TypeError):
            fine = False
        if not fine:
            self._refuse(grads)
        if index != torch._C._cuda_getDevice():
            raise ValueError(f"step: the weights lie on {self.device}, which is not the current device")
        at = array.array("Q", map(tensor.data_ptr, grads))
        L.check(L.load().moe_adamw_step(self._rows, at.buffer_info()[0] if n else None, n, self._plan.data_ptr(), self._pref,
                                        self.lr.data_ptr(), self.t.data_ptr(), self.norm.data_ptr(), self._ws.data_ptr(),
                                        self._ws.numel(), torch._C._cuda_getCurrentRawStream(index)), "moe_adamw_step")
        return self.norm if self.max_norm is not None else None

    def _refuse(self, grads):
        """What is wrong with these gradients."""
        if len(grads) != len(self._shapes):
            raise ValueError(f"grads: {len(self._shapes)} tensors are needed, got {len(grads)}")
        for i, (g, dtype, shape) in enumerate(zip(grads, self._dtypes, self._shapes)):
            want = f"grads[{i}]: a contiguous {dtype} tensor {tuple(shape)} on {self.device} is needed"
            if not isinstance(g, torch.Tensor):
                raise ValueError(want)
            if g.dtype != dtype or g.shape != shape or not g.is_contiguous() or g.get_device() != self.device.index:
                raise ValueError(f"{want}, got {g.dtype} {tuple(g.shape)} on {g.device}")
        raise ValueError("grads: tensors are needed")

    def moments(self, i: int):
        """(m, v) of weight i in its shape, float32; 8-bit states as the values they hold."""
        w, at = self._memory[i], self._at[i]
        n = w.numel()
        if self.state == "f32":
            return self.m[at:at + n].view(w.shape), self.v[at:at + n].view(w.shape)
        up = (n + _BLOCK - 1) // _BLOCK * _BLOCK

        def values(q, s):  # (a scale byte is a float's exponent field; 0 stands for 2^-127, a subnormal, 255 for NaN)
            e = s[at // _BLOCK:(at + up) // _BLOCK].to(torch.int32) << 23
            e = torch.where(e == 0, 0x00400000, torch.where(e == 0x7F800000, 0x7FC00000, e))
            return q[at:at + up].view(torch.float8_e4m3fn).float().view(-1, _BLOCK) * e.view(torch.float32).view(-1, 1)

        m, r = values(self.m, self.ms), values(self.v, self.vs)
        return m.view(-1)[:n].view(w.shape), r.view(-1)[:n].square().view(w.shape)

    def _state(self):
        return {k: getattr(self, k) for k in ("t", "m", "v", "ms", "vs", "master") if getattr(self, k) is not None}

    def state_dict(self) -> dict:
        """Copies of the flat state (without the weights and the learning rate)."""
        return {k: v.clone() for k, v in self._state().items()}

    def load_state_dict(self, d: dict):
        """Copies in a state that state_dict gave for the same weights and state
        kind; bfloat16 weights get the rounding of their masters."""
        mine = self._state()
        if set(d) != set(mine):
            raise ValueError(f"a state with {sorted(mine)} is needed, got {sorted(d)}")
        for k, v in mine.items():
            if d[k].shape != v.shape or d[k].dtype != v.dtype:
                raise ValueError(f"{k}: {v.dtype} {tuple(v.shape)} is needed, got {d[k].dtype} {tuple(d[k].shape)}")
        for k, v in mine.items():
            v.copy_(d[k])
        for w, at in zip(self._memory, self._at):
            if w.dtype == torch.bfloat16:
                w.view(-1).copy_(self.master[at:at + w.numel()])
