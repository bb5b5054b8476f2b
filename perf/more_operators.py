"""Workloads of what trains and adapts the block's weights: the AdamW step over
many tensors, and low-rank adapters of many requests beside a projection that
they share, forward and backward.

``listed()`` names fixed cases, ``draw(rng)`` makes one more from the same
ranges, ``prepare`` makes the inputs, ``run`` makes one pass (in plain torch
operations, or with the framework's calls when ``own`` is set), ``work``
counts the bytes and operations a pass cannot do without and ``exact`` gives
the operator's definition in 64 bits.

Definitions:
  adamw      t += 1; g' = c g with c = min(1, max_norm / (|g| + 1e-6)), |g| the
             2-norm over all tensors (c = 1 without max_norm);
             m = b1 m + (1 - b1) g', v = b2 v + (1 - b2) g'^2;
             w = w (1 - lr wd) - lr (m / (1 - b1^t)) / (sqrt(v / (1 - b2^t)) + eps).
             w is the f32 weight, or the f32 master of a bf16 weight, which gets
             its rounding.  States of 32 bits hold m and v.  States of 8 bits
             hold m and sqrt(v) as E4M3 codes with one scale 2^e per 32
             consecutive elements of a tensor, e the smallest with max <= 448 *
             2^e (at least -127); a value between two codes goes up when its
             distance above the lower one, as a fraction of theirs, and 16
             random bits over 65536 reach 1 together; a sqrt(v) that is not
             zero keeps at least the smallest code.  The random bits are a
             hash of a seed, t, the tensor and the element: the high half
             serves m, the low half sqrt(v).
  lora       h = s_a (A_a x), y = base + B_a^T h for the adapter a of each row
             (A [G, r, K], B [G, r, N], s [G]; rows without an adapter, index
             -1: h = 0, y = base)
  lora bwd   u = s_a (B_a dy), dx = base + A_a^T u,
             dA_a = sum over the adapter's rows of u x^T, dB_a = sum of h dy^T
"""
import math
import random

import torch

own = False
DEV = "cuda"
BLOCK = 32  # a tensor's slot in the flat buffers starts at a whole block
B1, B2, EPS, LR, WD, MAX_NORM = 0.9, 0.95, 1e-8, 3e-4, 0.1, 1.0


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # the norm's weight and the router of the GPT-OSS-shaped block, trained alone: latency
        {"name": "adamw_router", "op": "adamw", "layout": "layer", "E": 0, "H": 2880, "F": 0, "n": 32, "types": "bf16",
         "state": "f32", "clip": False},
        # the weights of that block with four of its experts: bf16 weights and gradients, f32 masters, clipped
        {"name": "adamw_layer", "op": "adamw", "layout": "layer", "E": 4, "H": 2880, "F": 2880, "n": 32,
         "types": "bf16", "state": "f32", "clip": True},
        # the same weights with both moments in 8 bits
        {"name": "adamw8_layer", "op": "adamw", "layout": "layer", "E": 4, "H": 2880, "F": 2880, "n": 32,
         "types": "bf16", "state": "mxfp8", "clip": True},
        # hundreds of f32 tensors of uneven, odd sizes (biases, norms, adapters, small matrices), clipped
        {"name": "adamw_many", "op": "adamw", "layout": "ragged", "tensors": 300, "elements": 30000000, "types": "f32",
         "state": "f32", "clip": True},
        # such a list of bf16 weights with moments in 8 bits, not clipped
        {"name": "adamw8_many", "op": "adamw", "layout": "ragged", "tensors": 120, "elements": 6000000, "types": "bf16",
         "state": "mxfp8", "clip": False},
        # one decoded token with an adapter beside the GPT-OSS-shaped block
        {"name": "lora_decode", "op": "lora", "T": 1, "K": 2880, "N": 2880, "r": 16, "G": 8, "order": "rows",
         "without": 0.0, "base": True},
        # one token of each of 64 requests, any of 64 adapters, DeepSeek-V3-shaped width
        {"name": "lora_batch", "op": "lora", "T": 64, "K": 7168, "N": 7168, "r": 16, "G": 64, "order": "rows",
         "without": 0.1, "base": True},
        # prompts of many requests in one batch of that width
        {"name": "lora_prompt", "op": "lora", "T": 8192, "K": 7168, "N": 7168, "r": 16, "G": 32, "order": "runs",
         "without": 0.1, "base": True},
        # decoded tokens and prompts together, higher rank, an output wider than the input, some requests without
        {"name": "lora_mixed", "op": "lora", "T": 4500, "K": 2880, "N": 5760, "r": 64, "G": 8, "order": "mixed",
         "without": 0.2, "base": True},
        # a small training batch of the tiny layer, two or three requests
        {"name": "lora_bwd_small", "op": "lora_bwd", "T": 300, "K": 256, "N": 512, "r": 8, "G": 4, "order": "runs",
         "without": 0.0, "base": True},
        # training eight adapters at once on one batch of the DeepSeek-V3-shaped width
        {"name": "lora_bwd_train", "op": "lora_bwd", "T": 8192, "K": 7168, "N": 7168, "r": 32, "G": 8, "order": "runs",
         "without": 0.0, "base": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["adamw", "adamw", "lora", "lora_bwd"])
    if op == "adamw":
        elements = _log(rng, 1000, 90_000_000)
        return {"op": op, "layout": "ragged", "tensors": min(_log(rng, 1, 300), elements // 100), "elements": elements,
                "types": rng.choice(["bf16", "f32"]), "state": rng.choice(["f32", "mxfp8"]), "clip": rng.random() < 0.5}
    order = rng.choice(["rows", "runs", "mixed"])
    K, N = 8 * _log(rng, 16, 896), 8 * _log(rng, 16, 896)
    r = rng.choice([8, 16, 24, 32, 64, 128])
    G = _log(rng, 1, 64)
    T = _log(rng, 1, 512 if order == "rows" else 8192)  # (rows: one decoded token per request)
    while T * G * r > 8192 * 32 * 16 and G > 1:
        G //= 2
    while T * r > 8192 * 64:
        T //= 2
    return {"op": op, "T": T, "K": K, "N": N, "r": r, "G": G, "order": order, "without": rng.choice([0.0, 0.1, 0.5]),
            "base": rng.random() < 0.7}


def _sizes(case):
    """Element counts of a case's tensors."""
    if case["layout"] == "layer":  # up projection, down projection, router, norm
        E, H, F = case["E"], case["H"], case["F"]
        return ([E * 2 * F * H, E * F * H] if E else []) + [case["n"] * H, H]
    n, total = case["tensors"], case["elements"]
    r = random.Random(n * 1_000_003 + total)
    part = [math.exp(r.uniform(0.0, 5.0)) for _ in range(n)]
    return [max(1, int(total * p / sum(part))) for p in part]


def work(case):
    if case["op"] == "adamw":
        n = sum(_sizes(case))
        narrow = case["types"] == "bf16"
        weights = 4 + 4 + 2 if narrow else 4 + 4  # master read and written, the bf16 weight written
        moments = 16 if case["state"] == "f32" else 2 * 2 * (1 + 1 / BLOCK) + 2 * 2  # (8 bits: also as values)
        return {"bytes": n * (weights + (2 if narrow else 4) + moments), "flops": 16 * n}
    T, K, N, r, G = (case[k] for k in ("T", "K", "N", "r", "G"))
    with_a = int(round(T * (1 - case["without"])))
    used = min(G, with_a)
    rows = with_a * K + (T * N if case["base"] else 0) + T * N + with_a * r  # x, base, y, h
    if case["op"] == "lora":
        return {"bytes": 2 * (rows + used * r * (K + N)) + 4 * T, "flops": 2 * with_a * r * (K + N)}
    rows = with_a * (N + K + r) + (T * K if case["base"] else 0) + T * K
    return {"bytes": 2 * (rows + used * r * (K + N) + G * r * (K + N)) + 4 * T, "flops": 4 * with_a * r * (K + N)}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _slots(sizes):
    return [(n + BLOCK - 1) // BLOCK * BLOCK for n in sizes]


def _views(flat, sizes):
    return [v[:n] for v, n in zip(flat.split(_slots(sizes)), sizes)]


def _codes(v):
    """E4M3 codes and scale bytes that hold f32 values (a state in mid-training)."""
    b = v.view(-1, BLOCK)
    top = b.abs().amax(1, keepdim=True)
    e = torch.where(top > 0, torch.ceil(torch.log2(top.clamp_min(1e-30) / 448)), torch.full_like(top, -127.0))
    return (b * torch.exp2(-e)).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).view(-1), (
        e.view(-1) + 127).to(torch.uint8)


def _prepare_adamw(case, seed):
    g = _gen(seed)
    sizes = _sizes(case)
    slots = torch.tensor(_slots(sizes), device=DEV)
    n = int(slots.sum())
    real = torch.zeros(n, device=DEV)
    for v in _views(real, sizes):
        v.fill_(1.0)
    # gradients of one tensor are alike in size, tensors differ; a few stretches have none (an expert without tokens)
    size = torch.repeat_interleave(torch.exp(_randn(g, len(sizes)) - 7.0), slots, output_size=n)
    alive = torch.repeat_interleave((torch.rand((n + 8191) // 8192, generator=g, device=DEV) > 0.02).float(), 8192)[:n]
    dt = torch.bfloat16 if case["types"] == "bf16" else torch.float32
    grad = (_randn(g, n) * size * alive * real).to(dt)
    w = _randn(g, n) * 0.02 * real
    m = _randn(g, n) * 0.3 * size * real
    v = (size * real) ** 2 * torch.exp(0.5 * _randn(g, n))
    s = {"sizes": sizes, "grad": grad, "t": torch.full((1,), 900 + seed % 200, dtype=torch.int64, device=DEV),
         "seed": seed % 1_000_003, "decay": [WD if k >= 2880 * 8 else 0.0 for k in sizes], "state": case["state"],
         "clip": MAX_NORM if case["clip"] else None}
    if dt == torch.bfloat16:
        s["master"], s["w"] = w, w.to(dt)
    else:
        s["w"] = w
    if case["state"] == "f32":
        s["m"], s["v"] = m, v
    else:
        s["m"], s["ms"] = _codes(m)
        s["v"], s["vs"] = _codes(v.sqrt())
    del m, v, w, size, alive
    if own:
        from grouped_gemm_glu_gb300.optim import AdamW
        s["grads"] = _views(grad, sizes)
        s["opt"] = AdamW(_views(s["w"], sizes), lr=LR, betas=(B1, B2), eps=EPS, weight_decay=s["decay"],
                         max_norm=s["clip"], state=s["state"], grad_dtype=dt, seed=s["seed"])
        s["opt"].load_state_dict({k: s[k] for k in ("t", "m", "v", "ms", "vs", "master") if k in s})
    return s


def _adapters_of_rows(case, g, seed):
    T, G, order = case["T"], case["G"], case["order"]
    rows = torch.randint(0, G, (T,), generator=g, device=DEV)
    rows = torch.where(torch.rand(T, generator=g, device=DEV) < case["without"], -1, rows)
    if order != "rows":
        r = random.Random(seed)
        at, starts = (T // 12 if order == "mixed" else 0), []
        while at < T:  # requests of some tens to a few thousand tokens, in the order they came
            starts.append(at)
            at += max(1, min(T - at, _log(r, 40, 3000)))
        if starts:
            length = torch.tensor([b - a for a, b in zip(starts, starts[1:] + [T])], device=DEV)
            one = torch.tensor([-1 if r.random() < case["without"] else r.randrange(G) for _ in starts], device=DEV)
            rows[starts[0]:] = torch.repeat_interleave(one, length)
    return rows.to(torch.int32)


def _prepare_lora(case, seed):
    g = _gen(seed)
    T, K, N, r, G = (case[k] for k in ("T", "K", "N", "r", "G"))
    bf = torch.bfloat16
    s = {"T": T, "K": K, "N": N, "r": r, "G": G, "x": _randn(g, T, K).to(bf),
         "A": (_randn(g, G, r, K) * K ** -0.5).to(bf), "B": (_randn(g, G, r, N) * 0.5 * r ** -0.5).to(bf),
         "scale": torch.rand(G, generator=g, device=DEV) * 1.5 + 0.5, "idx": _adapters_of_rows(case, g, seed)}
    if case["op"] == "lora":
        s["base"] = _randn(g, T, N).to(bf) if case["base"] else None
    else:
        s["dy"] = _randn(g, T, N).to(bf)
        s["base"] = _randn(g, T, K).to(bf) if case["base"] else None
        s["h"] = _hidden(s["x"], s["A"], s["scale"], s["idx"]).sum(1).to(bf)
    return s


def prepare(case, seed):
    s = _prepare_adamw(case, seed) if case["op"] == "adamw" else _prepare_lora(case, seed)
    s["op"] = case["op"]
    return s


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------
def _mul32(a, b):
    return (a * b) & 0xFFFFFFFF


def _mix(x):
    """A 32-bit hash of 32-bit values (held in int64)."""
    x = x ^ (x >> 16)
    x = _mul32(x, 0x7FEB352D)
    x = x ^ (x >> 15)
    x = _mul32(x, 0x846CA68B)
    return x ^ (x >> 16)


def _random_bits(s, slots):
    """32 random bits per element of the flat buffers (int64)."""
    n = s["grad"].numel()
    key = _mix((_mix(s["t"] & 0xFFFFFFFF) ^ s["seed"]) & 0xFFFFFFFF)
    keys = _mix((key + torch.arange(slots.numel(), device=DEV)) & 0xFFFFFFFF)
    first = torch.repeat_interleave(slots.cumsum(0) - slots, slots, output_size=n)
    i = torch.arange(n, device=DEV) - first
    return _mix((_mix((torch.repeat_interleave(keys, slots, output_size=n) + (i >> 32)) & 0xFFFFFFFF)
                 + (i & 0xFFFFFFFF)) & 0xFFFFFFFF)


def _pow2(e):
    """2^e of whole numbers, in 64 bits, to the bit."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _values(codes, scales, dt):
    return (codes.view(torch.float8_e4m3fn).to(dt).view(-1, BLOCK)
            * _pow2(scales.to(torch.int64) - 127).to(dt).view(-1, 1)).view(-1)


def _to_codes(x, bits16, at_least_one):
    """Codes and scale bytes of x (64 bits: the values lie next to the codes'
    borders), rounded up or down by 16 random bits."""
    b = x.view(-1, BLOCK)
    top = b.abs().amax(1, keepdim=True)
    f, k = torch.frexp(top)  # top = f 2^k, f in [1/2, 1): 448 = 0.875 * 2^9
    e = torch.where(top > 0, (k - 9 + (f > 0.875).to(k.dtype)).clamp_min(-127), -127)
    a = b.abs() * _pow2(-e)
    step = torch.frexp(a.clamp_min(2.0 ** -6))[1] - 4  # codes of a's size lie 2^step apart
    a = a * _pow2(-step)
    low = torch.floor(a)
    q = (low + ((a - low) + bits16.view(-1, BLOCK) / 65536.0 >= 1)) * _pow2(step)
    if at_least_one:
        q = torch.where((b > 0) & (q == 0), 2.0 ** -9, q)
    codes = torch.where(b < 0, -q, q).float().to(torch.float8_e4m3fn).view(torch.uint8)
    return codes.view(-1), (e.view(-1) + 127).to(torch.uint8)


def _adamw_plain(s):
    slots = torch.tensor(_slots(s["sizes"]), device=DEV)
    s["t"] += 1
    wide = s["state"] == "mxfp8"
    dt = torch.float64 if wide else torch.float32
    g = s["grad"].to(dt)
    norm = s["grad"].double().square().sum().sqrt()
    if s["clip"] is not None:
        c = (s["clip"] / (norm + 1e-6)).clamp_max(1.0)
        g = g * c.to(dt)
    m = _values(s["m"], s["ms"], dt) if wide else s["m"]
    v = _values(s["v"], s["vs"], dt).square() if wide else s["v"]
    m = m * B1 + g * (1 - B1)
    v = v * B2 + g * g * (1 - B2)
    t = s["t"].double()
    away1, away2 = (1 - B1 ** t).to(dt), (1 - B2 ** t).to(dt)
    decay = torch.repeat_interleave(torch.tensor(s["decay"], device=DEV), slots, output_size=g.numel())
    w = s["master"] if "master" in s else s["w"]
    w -= (w * (decay * LR) + LR * (m / away1) / ((v / away2).sqrt() + EPS)).float()
    out = {"w": s["w"]}
    if "master" in s:
        s["w"].copy_(w)
        out["master"] = w
    if s["clip"] is not None:
        out["norm"] = norm.float()
    if wide:
        bits = _random_bits(s, slots)
        codes, scales = _to_codes(m, bits >> 16, False)
        s["m"].copy_(codes)
        s["ms"].copy_(scales)
        codes, scales = _to_codes(v.sqrt(), bits & 0xFFFF, True)
        s["v"].copy_(codes)
        s["vs"].copy_(scales)
        out["m"] = _values(s["m"], s["ms"], torch.float32).bfloat16()
        out["root_v"] = _values(s["v"], s["vs"], torch.float32).bfloat16()
    else:
        out["m"], out["v"] = s["m"].copy_(m), s["v"].copy_(v)
    return out


def _spread(rows, idx, G):
    """[T, G, r]: the rows in their adapter's place, zero in the others'."""
    mine = idx.view(-1, 1).long() == torch.arange(G, device=DEV)
    return torch.where(mine.unsqueeze(2), rows, 0.0)


def _hidden(x, A, scale, idx):
    """s_a (A_a x) of every row in its adapter's place, [T, G, r] f32."""
    G, r, K = A.shape
    h = (x.float() @ A.float().view(G * r, K).t()).view(-1, G, r)
    return _spread(h * scale.view(1, G, 1), idx, G)


def _lora_plain(s):
    h = _hidden(s["x"], s["A"], s["scale"], s["idx"])
    y = h.view(-1, s["G"] * s["r"]) @ s["B"].float().view(-1, s["N"])
    if s["base"] is not None:
        y += s["base"].float()
    return {"y": y.bfloat16(), "h": h.sum(1).bfloat16()}


def _lora_bwd_plain(s):
    G, r, K, N = s["G"], s["r"], s["K"], s["N"]
    u = _hidden(s["dy"], s["B"], s["scale"], s["idx"]).view(-1, G * r)
    dx = u @ s["A"].float().view(-1, K)
    if s["base"] is not None:
        dx += s["base"].float()
    h = _spread(s["h"].float().unsqueeze(1), s["idx"], G).view(-1, G * r)
    dA, dB = u.t() @ s["x"].float(), h.t() @ s["dy"].float()
    return {"dx": dx.bfloat16(), "dA": dA.view(G, r, K).bfloat16(), "dB": dB.view(G, r, N).bfloat16()}


def run(state):
    s = state
    if not own:
        return {"adamw": _adamw_plain, "lora": _lora_plain, "lora_bwd": _lora_bwd_plain}[s["op"]](s)
    from grouped_gemm_glu_gb300 import ops
    if s["op"] == "lora":
        return ops.lora(s["x"], s["A"], s["B"], s["idx"], s["scale"], base=s["base"])
    if s["op"] == "lora_bwd":
        dx, dA, dB = ops.lora_bwd(s["dy"], s["x"], s["h"], s["A"], s["B"], s["idx"], s["scale"], base=s["base"])
        return {"dx": dx, "dA": dA, "dB": dB}
    opt = s["opt"]
    norm = opt.step(s["grads"])
    out = {"w": s["w"]}
    if "master" in s:
        out["master"] = opt.master
    if s["clip"] is not None:
        out["norm"] = norm
    if s["state"] == "f32":
        out["m"], out["v"] = opt.m, opt.v
    else:
        out["m"], out["root_v"] = ops.dequantize_mxfp8(opt.m, opt.ms), ops.dequantize_mxfp8(opt.v, opt.vs)
    return out


# ---------------------------------------------------------------------------
# Definitions in 64 bits
# ---------------------------------------------------------------------------
def _hash64(x):
    for shift, factor in ((16, 0x7FEB352D), (15, 0x846CA68B)):
        x = ((x ^ (x >> shift)) * factor) & 0xFFFFFFFF
    return x ^ (x >> 16)


_GRID = None


def _grid():
    """The non-negative E4M3 values."""
    global _GRID
    if _GRID is None:
        low = [k * 2.0 ** -9 for k in range(8)]
        high = [(8 + k) * 2.0 ** (e - 3) for e in range(-6, 9) for k in range(8)]
        _GRID = torch.tensor([v for v in low + high if v <= 448], dtype=torch.float64, device=DEV)
    return _GRID


def _two_to(e):
    """2^e by a table."""
    return torch.tensor([2.0 ** k for k in range(-160, 161)], dtype=torch.float64, device=DEV)[e.long() + 160]


def _held(x, bits, least):
    """What an 8-bit state holds of the 64-bit values x of one tensor."""
    n = x.numel()
    b = torch.zeros((n + BLOCK - 1) // BLOCK * BLOCK, dtype=torch.float64, device=DEV)
    b[:n] = x
    b = b.view(-1, BLOCK)
    chance = torch.zeros(b.numel(), dtype=torch.float64, device=DEV)
    chance[:n] = bits.double() / 65536
    top = b.abs().amax(1)
    e = torch.ceil(torch.log2(top.clamp_min(1e-300) / 448)).clamp_min(-127)
    e = torch.where(top > 448 * _two_to(e), e + 1, torch.where((top <= 448 * _two_to(e - 1)) & (e > -127), e - 1, e))
    a = b.abs() / _two_to(e).unsqueeze(1)
    grid = _grid()
    at = torch.searchsorted(grid, a.contiguous(), right=True) - 1
    low, high = grid[at], grid[(at + 1).clamp_max(grid.numel() - 1)]
    gap = torch.where(high > low, high - low, 1.0)
    q = torch.where((a - low) / gap + chance.view(-1, BLOCK) >= 1, high, low)
    if least:
        q = torch.where((a > 0) & (q == 0), grid[1], q)
    return (torch.copysign(q, b) * _two_to(e).unsqueeze(1)).view(-1)


def _adamw_exact(s):
    sizes = s["sizes"]
    t = int(s["t"]) + 1
    key = _hash64(_hash64(t & 0xFFFFFFFF) ^ s["seed"])
    norm = math.sqrt(sum(float(g.double().square().sum()) for g in _views(s["grad"], sizes)))
    c = min(1.0, s["clip"] / (norm + 1e-6)) if s["clip"] is not None else 1.0
    f64 = torch.float64
    wide = s["state"] == "mxfp8"
    out = {k: torch.zeros(s["grad"].numel(), dtype=f64, device=DEV) for k in ("w", "m", "root_v" if wide else "v")}
    held = {}
    for k in ("m", "v"):
        x = s[k]
        if wide:
            x = x.view(torch.float8_e4m3fn).double().view(-1, BLOCK) * _two_to(s[k + "s"].long() - 127).view(-1, 1)
        held[k] = x.double().view(-1)
    src = s["master"] if "master" in s else s["w"]
    at = 0
    for j, (n, slot, wd) in enumerate(zip(sizes, _slots(sizes), s["decay"])):
        here = slice(at, at + n)
        g = s["grad"][here].double() * c
        m = B1 * held["m"][here] + (1 - B1) * g
        old = held["v"][here]
        v = B2 * (old * old if wide else old) + (1 - B2) * g * g
        w = src[here].double()
        out["w"][here] = w * (1 - LR * wd) - LR * (m / (1 - B1 ** t)) / (torch.sqrt(v / (1 - B2 ** t)) + EPS)
        if wide:
            i = torch.arange(n, device=DEV)
            bits = _hash64((_hash64((_hash64((key + j) & 0xFFFFFFFF) + (i >> 32)) & 0xFFFFFFFF) + i) & 0xFFFFFFFF)
            out["m"][at:at + slot] = _held(m, bits >> 16, False)
            out["root_v"][at:at + slot] = _held(torch.sqrt(v), bits & 0xFFFF, True)
        else:
            out["m"][here], out["v"][here] = m, v
        at += slot
    if "master" in s:
        out["master"] = out["w"]
    if s["clip"] is not None:
        out["norm"] = torch.tensor(norm, dtype=f64)
    return out


def _lora_exact(s):
    back = s["op"] == "lora_bwd"
    f64 = torch.float64
    src, P, Q = (s["dy"], s["B"], s["A"]) if back else (s["x"], s["A"], s["B"])
    T, G, r = s["T"], s["G"], s["r"]
    out = torch.zeros(T, Q.shape[2], dtype=f64, device=DEV) if s["base"] is None else s["base"].double()
    hid = torch.zeros(T, r, dtype=f64, device=DEV)
    dA, dB = torch.zeros(G, r, s["K"], dtype=f64, device=DEV), torch.zeros(G, r, s["N"], dtype=f64, device=DEV)
    for a in range(G):
        rows = torch.nonzero(s["idx"] == a).view(-1)
        if rows.numel() == 0:
            continue
        z = float(s["scale"][a]) * (src[rows].double() @ P[a].double().t())
        hid[rows] = z
        out[rows] += z @ Q[a].double()
        if back:
            dA[a] = z.t() @ s["x"][rows].double()
            dB[a] = s["h"][rows].double().t() @ s["dy"][rows].double()
    return {"dx": out, "dA": dA, "dB": dB} if back else {"y": out, "h": hid}


def exact(case, seed):
    s = prepare(case, seed)
    return _adamw_exact(s) if case["op"] == "adamw" else _lora_exact(s)
