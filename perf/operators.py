"""Workloads of the operators around the expert MLP: the residual + RMS norm
that feeds it, the router that chooses the experts, and MXFP4 expert weights
(their cast and the grouped products that read them).

``listed()`` names fixed cases, ``draw(rng)`` makes one more from the same
ranges, ``prepare`` makes the inputs, ``run`` makes one pass (in plain torch
operations, or with the framework's calls when ``own`` is set), ``work``
counts the bytes and operations a pass cannot do without and ``exact`` gives
the operator's definition in 64 bits.

Definitions (T tokens, H hidden width, n experts, k chosen, blocks of 32):
  norm       h = bf16(x + residual) (h = x without a residual),
             rstd = 1 / sqrt(mean(h^2) + eps), y = h * rstd * gamma; y as bf16
             and / or MXFP8 (E4M3 codes, one E8M0 scale per 32 columns)
  norm bwd   t = dy * gamma, dx = rstd * (t - h * rstd^2 * mean(t * h)) + dres,
             dgamma = sum over tokens of dy * h * rstd
  router     scores s = softmax(logits) or sigmoid(logits); choice by s + bias
             inside the best groups; weights from s, renormalised or not,
             times a factor; experts with a logit of -inf and masked tokens
             are never chosen (index -1, weight 0); ties to the lowest index
  mxfp4      blocks of 32 along the contraction: scale 2^(floor(log2 amax) - 2),
             elements rounded to nearest even on 0, .5, 1, 1.5, 2, 3, 4, 6
             (saturating); product: rows of MXFP8 activations, grouped by
             expert, with the expert's MXFP4 weight [N, K], optionally with
             bias and the gated activation
"""
import math

import numpy as np
import torch

own = False
DEV = "cuda"
ALIGN = 32  # rows of one expert are padded to whole blocks of 32
NEG_INF = float("-inf")


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one decoded token entering the layer of the GPT-OSS-shaped workload
        {"name": "norm_decode", "op": "norm", "T": 1, "H": 2880, "residual": True, "out": "bf16"},
        # a training / prefill batch of the DeepSeek-V3-shaped workload, with
        # the 8-bit copy that an MXFP8 first product reads
        {"name": "norm_train", "op": "norm", "T": 8192, "H": 7168, "residual": True, "out": "both"},
        # its backward: gradients of the stream and of the norm's weight
        {"name": "norm_bwd_train", "op": "norm_bwd", "T": 8192, "H": 7168, "residual": True},
        # one decoded token over 256 experts in 8 groups (sigmoid scores, balance bias)
        {"name": "router_decode", "op": "router", "T": 1, "n": 256, "k": 8, "score": "sigmoid", "bias": True,
         "renorm": True, "groups": 8, "keep": 4, "top": 2, "dtype": "f32", "dead": 0, "masked": 0.0},
        # a training batch of the same router; a few padding tokens are masked
        {"name": "router_train", "op": "router", "T": 8192, "n": 256, "k": 8, "score": "sigmoid", "bias": True,
         "renorm": True, "groups": 8, "keep": 4, "top": 2, "dtype": "f32", "dead": 0, "masked": 0.02},
        # the skewed workload's router: softmax over 64 experts of which 8 are
        # switched off, probabilities not renormalised, bf16 logits
        {"name": "router_skew", "op": "router", "T": 32768, "n": 64, "k": 6, "score": "softmax", "bias": False,
         "renorm": False, "groups": 1, "keep": 1, "top": 1, "dtype": "bf16", "dead": 8, "masked": 0.0},
        # gradient of that router's weights with respect to its logits, training
        {"name": "router_bwd_skew", "op": "router_bwd", "T": 32768, "n": 64, "k": 6, "score": "softmax",
         "bias": False, "renorm": False, "groups": 1, "keep": 1, "top": 1, "dtype": "f32", "dead": 8, "masked": 0.0},
        # casting the down projection of one GPT-OSS-shaped layer, stored [E, F, H]:
        # blocks run along F, so the cast transposes; then read back as values
        {"name": "mxfp4_cast_cols", "op": "mxfp4_cast", "G": 32, "R": 2880, "C": 2880, "col": True},
        # casting a small layer's up projection along its rows
        {"name": "mxfp4_cast_rows", "op": "mxfp4_cast", "G": 4, "R": 1024, "C": 256, "col": False},
        # one decoded token, top-4: the up projection with bias and clamped SwiGLU
        {"name": "mxfp4_up_decode", "op": "mxfp4_product", "E": 32, "K": 2880, "N": 5760, "tokens": 1, "k": 4,
         "glu": True, "spread": "even"},
        # a small serving batch of the DeepSeek-V3-shaped shard, uneven over its
        # 32 experts: the down projection
        {"name": "mxfp4_down_batch", "op": "mxfp4_product", "E": 32, "K": 2048, "N": 7168, "tokens": 64, "k": 8,
         "glu": False, "spread": "skew"},
        # a long prompt batch of the GPT-OSS-shaped layer: the up projection
        {"name": "mxfp4_up_prompt", "op": "mxfp4_product", "E": 32, "K": 2880, "N": 5760, "tokens": 16384, "k": 4,
         "glu": True, "spread": "even"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        c = _draw(rng)
        if 3072 not in c.values():
            return c


def _draw(rng):
    op = rng.choice(["norm", "norm_bwd", "router", "router_bwd", "mxfp4_cast", "mxfp4_product"])
    if op in ("norm", "norm_bwd"):
        out = rng.choice(["bf16", "mxfp8", "both"])
        H = 32 * _log(rng, 2, 512) if op == "norm" and out != "bf16" else 8 * _log(rng, 8, 2048)
        T = max(1, min(_log(rng, 1, 32768), 8192 * 7168 // H))
        c = {"op": op, "T": T, "H": H, "residual": rng.random() < 0.7}
        if op == "norm":
            c["out"] = out
        return c
    if op in ("router", "router_bwd"):
        groups = rng.choice([1, 1, 4, 8])
        n = groups * _log(rng, max(2, 8 // groups), 512 // groups)
        score = rng.choice(["softmax", "sigmoid"])
        bias = score == "sigmoid" and rng.random() < 0.7
        keep = rng.randint(max(1, groups // 2), groups)
        k = rng.randint(1, min(16, n // groups * keep))
        dead = rng.choice([0, 0, n // 8])
        T = max(1, min(_log(rng, 1, 32768), 32768 * 64 // n))
        top = 2 if groups > 1 and n // groups >= 2 and score == "sigmoid" else 1
        return {"op": op, "T": T, "n": n, "k": k, "score": score, "bias": bias, "renorm": rng.random() < 0.6,
                "groups": groups, "keep": keep, "top": top, "dtype": rng.choice(["f32", "bf16"]), "dead": dead,
                "masked": rng.choice([0.0, 0.0, 0.1])}
    if op == "mxfp4_cast":
        G, R, C = rng.choice([1, 4, 8, 32]), 32 * _log(rng, 1, 180), 32 * _log(rng, 1, 180)
        while G * R * C > 32 * 2880 * 2880:
            G = max(1, G // 2)
        return {"op": op, "G": G, "R": R, "C": C, "col": rng.random() < 0.5}
    glu = rng.random() < 0.5
    E, k = rng.choice([(4, 2), (8, 4), (16, 4), (32, 4), (32, 8), (64, 6)])
    K, N = 32 * _log(rng, 4, 160), 64 * _log(rng, 2, 100)
    while E * K * N > 32 * 2880 * 5760:
        N = max(64, 64 * (N // 128))
        if N == 64:
            K = max(64, 32 * (K // 64))
    tokens = max(1, min(_log(rng, 1, 16384), 16384 * 4 * 2880 * 5760 // (k * K * N)))
    return {"op": op, "E": E, "K": K, "N": N, "tokens": tokens, "k": k, "glu": glu,
            "spread": rng.choice(["even", "skew"])}


def _counts(case):
    """Rows of the experts, busiest first: the same for every seed (the seed
    says which expert has which count)."""
    E, rows = case["E"], case["tokens"] * case["k"]
    if case["spread"] == "even":
        return [rows // E + (1 if e < rows % E else 0) for e in range(E)]
    share = [(e + 1) ** -1.2 for e in range(E)]
    c = [min(case["tokens"], int(rows * s / sum(share))) for s in share]
    e = 0
    while sum(c) < rows:  # what rounding and the limit of one row a token left over
        if c[e % E] < case["tokens"]:
            c[e % E] += min(case["tokens"] - c[e % E], max(1, (rows - sum(c)) // 8))
        e += 1
    return c


def work(case):
    op = case["op"]
    if op == "norm":
        T, H = case["T"], case["H"]
        b = T * H * 2 + H * 2 + T * 4
        if case["residual"]:
            b += 2 * T * H * 2
        if case["out"] in ("bf16", "both"):
            b += T * H * 2
        if case["out"] in ("mxfp8", "both"):
            b += T * H + T * H // 32 + T * H * 2  # codes, scales, and the values read back from them
        return {"bytes": b, "flops": 6 * T * H}
    if op == "norm_bwd":
        T, H = case["T"], case["H"]
        return {"bytes": T * H * 2 * (4 if case["residual"] else 3) + T * 4 + H * 6, "flops": 12 * T * H}
    if op in ("router", "router_bwd"):
        T, n, k = case["T"], case["n"], case["k"]
        es = 4 if case["dtype"] == "f32" else 2
        b = T * n * es + T * k * 8
        if op == "router":
            return {"bytes": b + n * 4 * (2 if case["bias"] else 1) + (T if case["masked"] else 0),
                    "flops": 4 * T * n}
        return {"bytes": b + T * n * es, "flops": 6 * T * n}
    if op == "mxfp4_cast":
        n = case["G"] * case["R"] * case["C"]
        return {"bytes": 2 * n + n // 2 + n // 32 + 2 * n, "flops": 4 * n}
    K, N = case["K"], case["N"]
    c = _counts(case)
    R, live = sum(c), sum(1 for x in c if x)
    out = N // 2 if case["glu"] else N
    return {"bytes": live * N * (K // 2 + K // 32) + R * (K + K // 32) + R * out * 2 + (live * N * 2 if case["glu"] else 0),
            "flops": 2 * R * N * K}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 1000003 + 17)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)


def _pitch(K):
    return (K + 127) // 128 * 128


def prepare(case, seed):
    g, op, bf = _gen(seed), case["op"], torch.bfloat16
    s = {"case": case}
    if op in ("norm", "norm_bwd"):
        T, H = case["T"], case["H"]
        # a residual stream a few times larger than the branch added to it,
        # with a few columns that carry large values
        wide = 1.0 + 20.0 * (torch.rand(H, generator=g, device=DEV) < 0.003).float()
        s["gamma"] = (1.0 + 0.2 * _randn(g, H)).to(bf)
        s["eps"] = 1e-5
        if op == "norm":
            s["x"] = _randn(g, T, H).to(bf)
            s["residual"] = (3.0 * _randn(g, T, H) * wide).to(bf) if case["residual"] else None
        else:
            s["h"] = (3.0 * _randn(g, T, H) * wide).to(bf)
            s["rstd"] = torch.rsqrt(s["h"].float().square().mean(1) + s["eps"])
            s["dy"] = _randn(g, T, H).to(bf)
            s["dres"] = _randn(g, T, H).to(bf) if case["residual"] else None
        return s
    if op in ("router", "router_bwd"):
        T, n, k = case["T"], case["n"], case["k"]
        logits = _randn(g, T, n) * 1.5 + 0.5 * _randn(g, 1, n)
        if case["dead"]:  # experts switched off by a logit of -inf
            logits[:, torch.randperm(n, generator=g, device=DEV)[:case["dead"]]] = NEG_INF
        s["logits"] = logits.to(bf) if case["dtype"] == "bf16" else logits
        s["bias"] = 0.05 * _randn(g, n) if case["bias"] else None
        s["mask"] = (torch.rand(T, generator=g, device=DEV) >= case["masked"]).to(torch.uint8) if case["masked"] else None
        if op == "router_bwd":
            own_idx, _, _ = _router_plain(s)
            s["idx"] = own_idx
            s["dprob"] = _randn(g, T, k)
        return s
    if op == "mxfp4_cast":
        s["w"] = torch.empty(case["G"], case["R"], case["C"], dtype=bf, device=DEV)
        for e in range(case["G"]):
            s["w"][e] = (_randn(g, case["R"], case["C"]) * case["C"] ** -0.5).to(bf)
        return s
    E, K, N = case["E"], case["K"], case["N"]
    order = np.random.RandomState(int(seed) % (1 << 31)).permutation(E)
    counts = np.zeros(E, dtype=np.int64)
    counts[order] = _counts(case)
    off = np.zeros(E + 1, dtype=np.int64)
    off[1:] = np.cumsum((counts + ALIGN - 1) // ALIGN * ALIGN)
    R = int(off[E])
    cap = (R + 127) // 128 * 128
    row = np.full((E, int(max(counts.max(), 1))), cap, dtype=np.int64)  # row of every expert's i-th token; cap: none
    real = np.zeros(cap, dtype=bool)
    for e in range(E):
        row[e, :counts[e]] = off[e] + np.arange(counts[e])
        real[off[e]:off[e] + counts[e]] = True
    s.update(R=R, counts=torch.tensor(counts, dtype=torch.int32, device=DEV),
             offsets=torch.tensor(off, dtype=torch.int32, device=DEV),
             rows=torch.tensor(row, device=DEV), status=torch.zeros(1, dtype=torch.int32, device=DEV))
    x = _randn(g, cap, K) * torch.tensor(real, device=DEV)[:, None]
    codes, scale = _mx8_parts(x.view(cap, K // 32, 32))
    s["xq"] = codes.view(torch.uint8).view(cap, K)
    s["xs"] = scale.to(torch.uint8).view(cap, K // 32)
    # the weights: packed 4-bit codes (rows of a pitch of 128 elements) and the
    # scales in the order the tensor cores copy them
    s["wq"] = torch.zeros(E, N, _pitch(K) // 2, dtype=torch.uint8, device=DEV)
    ws = torch.zeros(E, (N + 255) // 256 * 256, _pitch(K) // 32, dtype=torch.uint8, device=DEV)
    for e in range(E):
        c, b = _mx4_parts((_randn(g, N, K) * K ** -0.5).view(N, K // 32, 32))
        c = c.view(N, K // 2, 2)
        s["wq"][e, :, :K // 2] = (c[..., 0] | (c[..., 1] << 4)).to(torch.uint8)
        ws[e, :N, :K // 32] = b.to(torch.uint8).view(N, K // 32)
    nt, kb = ws.shape[1] // 256, ws.shape[2] // 4
    s["ws"] = ws.view(E, nt, 2, 4, 32, kb, 4).permute(0, 1, 5, 2, 4, 3, 6).contiguous().view(-1)
    if case["glu"]:
        s["bias"] = (0.02 * _randn(g, E, N)).to(bf)
    return s


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------
def _exponents(v, emax):
    """E8M0 byte of blocks of 32 (last axis): floor(log2 amax) - emax + 127, not below 0."""
    bits = v.abs().amax(-1, keepdim=True).contiguous().view(torch.int32)
    return ((bits >> 23) - emax).clamp(min=0)


def _pow2(e):
    """2^(e - 127) of an int32 tensor of E8M0 bytes."""
    return (e.clamp(min=1) << 23).view(torch.float32)


def _mx8_parts(v):
    """(E4M3 codes, E8M0 bytes) of float32 blocks."""
    b = _exponents(v, 8)
    return (v * _pow2(254 - b)).clamp(-448.0, 448.0).to(torch.float8_e4m3fn), b


def _e2m1(v):
    """v rounded to nearest even on 0, .5, 1, 1.5, 2, 3, 4, 6, saturating; sign kept apart."""
    a = v.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return (torch.round(a / step) * step).clamp(max=6.0)


def _mx4_parts(v):
    """(4-bit codes, E8M0 bytes) of float32 blocks."""
    b = _exponents(v, 2)
    r = _e2m1(v * _pow2(254 - b))
    code = torch.where(r < 2, r * 2, torch.where(r < 4, r + 2, r * 0.5 + 4)).to(torch.int32)
    return code | ((v < 0).to(torch.int32) << 3), b


def _norm_plain(s):
    c = s["case"]
    T, H = c["T"], c["H"]
    o = {}
    h = s["x"]
    if s["residual"] is not None:
        h = (s["x"].float() + s["residual"].float()).to(torch.bfloat16)
        o["h"] = h
    h = h.float()
    o["rstd"] = torch.rsqrt((h * h).sum(1) / H + s["eps"])
    y = h * o["rstd"][:, None] * s["gamma"].float()
    if c["out"] in ("bf16", "both"):
        o["y"] = y.to(torch.bfloat16)
    if c["out"] in ("mxfp8", "both"):
        q, b = _mx8_parts(y.view(T, H // 32, 32))
        o["v"] = (q.float() * _pow2(b)).view(T, H).to(torch.bfloat16)
    return o


def _norm_bwd_plain(s):
    dy, h, r = s["dy"].float(), s["h"].float(), s["rstd"][:, None]
    t = dy * s["gamma"].float()
    dx = r * (t - h * (r * r * ((t * h).sum(1, keepdim=True) / h.shape[1])))
    if s["dres"] is not None:
        dx = dx + s["dres"].float()
    return {"dx": dx.to(torch.bfloat16), "dgamma": (dy * h * r).sum(0)}


def _scores(x, kind):
    """Scores of float32 logits; an expert with a logit of -inf scores 0."""
    if kind == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-x))
    top = x.amax(1, keepdim=True)
    e = torch.exp(x - torch.where(top == NEG_INF, 0.0, top))
    return e / e.sum(1, keepdim=True).clamp(min=1e-38)


def _router_plain(s):
    c = s["case"]
    T, n, k, G = c["T"], c["n"], c["k"], c["groups"]
    x = s["logits"].float()
    sc = _scores(x, c["score"])
    # the logits order the experts as the scores do: without a bias they are the keys
    key = x if s["bias"] is None else torch.where(x == NEG_INF, NEG_INF, sc + s["bias"])
    if G > 1:
        gk = (key if c["top"] == 1 or s["bias"] is not None else torch.where(x == NEG_INF, NEG_INF, sc)).view(T, G, n // G)
        gs = torch.sort(gk, dim=2, descending=True).values[:, :, :c["top"]].sum(2)
        order = torch.sort(gs, dim=1, descending=True, stable=True).indices[:, :c["keep"]]
        keep = torch.zeros(T, G, dtype=torch.bool, device=x.device).scatter_(1, order, True)
        key = torch.where(keep.repeat_interleave(n // G, 1), key, NEG_INF)
    if s["mask"] is not None:
        key = torch.where(s["mask"][:, None] != 0, key, NEG_INF)
    val, idx = torch.sort(key, dim=1, descending=True, stable=True)
    val, idx = val[:, :k], idx[:, :k]
    idx = torch.where(val == NEG_INF, -1, idx)
    p = _weights(x, sc, idx, c)
    load = torch.zeros(n + 1, dtype=torch.int32, device=x.device)
    load.index_add_(0, idx.reshape(-1) + 1, torch.ones_like(idx, dtype=torch.int32).reshape(-1))
    return idx.to(torch.int32), p, load[1:]


def _weights(x, sc, idx, c):
    """Weights of the chosen experts (0 where idx is -1), times the factor 2.5 of sigmoid routers."""
    at = idx.clamp(min=0).long()
    w = torch.where(idx < 0, 0.0, sc.gather(1, at))
    if c["renorm"] and c["score"] == "softmax":  # the softmax over the chosen logits
        xs = torch.where(idx < 0, NEG_INF, x.gather(1, at))
        w = torch.where(idx < 0, 0.0, _scores(xs, "softmax"))
    elif c["renorm"]:
        w = w / (w.sum(1, keepdim=True) + 1e-20)
    return w * _factor(c)


def _factor(c):
    return 2.5 if c["score"] == "sigmoid" else 1.0


def _router_bwd_plain(s):
    c = s["case"]
    x = s["logits"].float()
    sc = _scores(x, c["score"])
    idx = s["idx"].long()
    on, at, f = idx >= 0, idx.clamp(min=0), _factor(c)
    g = torch.where(on, s["dprob"], 0.0)
    w = _weights(x, sc, idx, c) / f
    d = torch.zeros(x.shape[0], x.shape[1] + 1, device=x.device)  # column 0 takes the empty slots
    if c["renorm"]:
        inner = (g * w).sum(1, keepdim=True)
        dsel = f * torch.where(on, g - inner, 0.0)
        if c["score"] == "softmax":
            dsel = dsel * w
        else:
            ssel = torch.where(on, sc.gather(1, at), 0.0)
            dsel = dsel / (ssel.sum(1, keepdim=True) + 1e-20) * ssel * (1.0 - ssel)
        d.scatter_add_(1, idx + 1, dsel)
        return d[:, 1:].to(s["logits"].dtype)
    if c["score"] == "softmax":
        d.scatter_add_(1, idx + 1, f * g * w)
        d = d[:, 1:] - sc * (f * (g * w).sum(1, keepdim=True))
        return d.to(s["logits"].dtype)
    d.scatter_add_(1, idx + 1, f * g * w * (1.0 - w))
    return d[:, 1:].to(s["logits"].dtype)


def _cast_plain(s):
    w = s["w"].float()
    if s["case"]["col"]:
        w = w.transpose(1, 2).contiguous()
    v = w.view(*w.shape[:2], -1, 32)
    b = _exponents(v, 2)
    v = _e2m1(v * _pow2(254 - b)) * torch.sign(v) * _pow2(b)
    return v.view(w.shape).to(torch.bfloat16)


def _weights_of(s, dt):
    """The MXFP4 weights [E, N, K] as dt."""
    c = s["case"]
    E, K, N = c["E"], c["K"], c["N"]
    nt, kb = (N + 255) // 256, _pitch(K) // 128
    b = s["ws"].view(E, nt, kb, 2, 32, 4, 4).permute(0, 1, 3, 5, 4, 2, 6).reshape(E, nt * 256, kb * 4)[:, :N, :K // 32]
    q = s["wq"][:, :, :K // 2].int()
    q = torch.stack((q & 15, q >> 4), 3).view(E, N, K)
    grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0.0, -.5, -1, -1.5, -2, -3, -4, -6], device=q.device, dtype=dt)
    return (grid[q].view(E, N, K // 32, 32) * _pow2(b.int())[..., None].to(dt)).view(E, N, K)


def _glu(u, g):
    """Clamped SwiGLU of the GPT-OSS-shaped workload: (u + 1) g sigmoid(1.702 g), g clamped to +-7."""
    g = g.clamp(-7.0, 7.0)
    return (u + 1.0) * g / (1.0 + torch.exp(-1.702 * g))


def _product_in(s, dt):
    c = s["case"]
    E, K, N = c["E"], c["K"], c["N"]
    cap = s["xq"].shape[0]
    a = s["xq"].view(torch.float8_e4m3fn).to(dt).view(cap, K // 32, 32) * _pow2(s["xs"].int())[..., None].to(dt)
    a = torch.cat((a.view(cap, K), torch.zeros(1, K, device=a.device, dtype=dt)))  # row cap: no token
    pre = torch.bmm(a[s["rows"]], _weights_of(s, dt).transpose(1, 2))  # [E, rows of the busiest, N]
    if c["glu"]:
        pre = (pre + s["bias"].to(dt)[:, None, :]).view(E, -1, N // 64, 2, 32)
        pre = _glu(pre[..., 0, :], pre[..., 1, :]).reshape(E, -1, N // 2)
    y = torch.zeros(cap + 1, pre.shape[2], device=a.device, dtype=dt)
    y[s["rows"].view(-1)] = pre.reshape(-1, pre.shape[2])
    return y[:s["R"]].contiguous() if dt == torch.float64 else y[:s["R"]].to(torch.bfloat16)


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def run(s):
    c = s["case"]
    op = c["op"]
    if not own:
        if op == "norm":
            return _norm_plain(s)
        if op == "norm_bwd":
            return _norm_bwd_plain(s)
        if op == "router":
            idx, prob, load = _router_plain(s)
            return {"idx": idx, "prob": prob, "load": load}
        if op == "router_bwd":
            return {"dlogits": _router_bwd_plain(s)}
        if op == "mxfp4_cast":
            return {"v": _cast_plain(s)}
        return {"y": _product_in(s, torch.float32)}
    from grouped_gemm_glu_gb300 import lib as L
    from grouped_gemm_glu_gb300 import ops
    if op == "norm":
        o = ops.rmsnorm(s["x"], s["gamma"], s["eps"], residual=s["residual"], bf16=c["out"] != "mxfp8",
                        mxfp8=c["out"] != "bf16")
        r = {"rstd": o["rstd"]}
        if c["residual"]:
            r["h"] = o["h"]
        if c["out"] != "mxfp8":
            r["y"] = o["y"]
        if c["out"] != "bf16":
            r["v"] = ops.dequantize_mxfp8(o["q"], o["s"])
        return r
    if op == "norm_bwd":
        dx, dgamma = ops.rmsnorm_bwd(s["dy"], s["h"], s["gamma"], s["rstd"], dres=s["dres"])
        return {"dx": dx, "dgamma": dgamma}
    if op in ("router", "router_bwd"):
        prm = L.router_params(c["score"], renorm=c["renorm"], scale=_factor(c), n_group=c["groups"],
                              topk_group=c["keep"], group_top=c["top"])
        if op == "router_bwd":
            return {"dlogits": ops.router_bwd(s["logits"], s["idx"], s["dprob"], prm)}
        o = ops.router(s["logits"], c["k"], prm, bias=s["bias"], token_mask=s["mask"])
        return {"idx": o["idx"], "prob": o["prob"], "load": o["load"]}
    if op == "mxfp4_cast":
        q, sc = ops.quantize_mxfp4(s["w"], col=c["col"])
        return {"v": ops.dequantize_mxfp4(q, sc, c["R"] if c["col"] else c["C"])}
    if c["glu"]:
        prm = L.glu_params("swiglu", alpha=1.702, up_offset=1.0, gate_lo=-7.0, gate_hi=7.0)
        o = ops.fc1_fwd_mxfp4(s["xq"], s["xs"], s["wq"], s["ws"], s["counts"], s["offsets"], c["N"] // 2, prm,
                              out_mode=L.OUT_BF16, b1p=s["bias"], save_pre=False, status=s["status"])
        return {"y": o["y"][:s["R"]]}
    y = ops.fc2_fwd_mxfp4(s["xq"], s["xs"], s["wq"], s["ws"], s["counts"], s["offsets"], status=s["status"])
    return {"y": y[:s["R"]]}


# ---------------------------------------------------------------------------
# 64 bits
# ---------------------------------------------------------------------------
def _block_round64(v, emax, top, mant):
    """Blocks of 32 (last axis) of a float64 tensor on a power-of-two scale and
    a minifloat grid with `mant` mantissa bits, largest value `top` and
    smallest exponent emin (0 for E2M1, -6 for E4M3), as float64."""
    emin = 0 if mant == 1 else -6
    a = v.abs().amax(-1, keepdim=True)
    e = torch.where(a > 0, torch.floor(torch.log2(torch.where(a > 0, a, 1.0))) - emax, 0.0)
    x = v / torch.exp2(e)
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** emin))) - mant)
    return (torch.round(x / step) * step).clamp(-top, top) * torch.exp2(e)


def exact(case, seed):
    s = prepare(case, seed)
    op, d = case["op"], torch.float64
    if op == "norm":
        x = s["x"].to(d)
        o = {}
        if s["residual"] is not None:
            x = (x + s["residual"].to(d)).to(torch.bfloat16).to(d)
            o["h"] = x
        rms = torch.sqrt(torch.mean(x ** 2, dim=1, keepdim=True) + s["eps"])
        y = x / rms * s["gamma"].to(d)
        o["rstd"] = 1.0 / rms[:, 0]
        if case["out"] != "mxfp8":
            o["y"] = y
        if case["out"] != "bf16":
            o["v"] = _block_round64(y.view(y.shape[0], -1, 32), 8, 448.0, 3).view(y.shape)
        return o
    if op == "norm_bwd":
        # y_i = g_i h_i r with r = (mean h^2 + eps)^(-1/2): dL/dh_i = g_i dy_i r + (dL/dr) dr/dh_i, dr/dh_i = -r^3 h_i / H
        dy, h, gm, r = s["dy"].to(d), s["h"].to(d), s["gamma"].to(d), s["rstd"].to(d)
        dr = torch.einsum("th,th,h->t", dy, h, gm)
        dx = dy * gm * r[:, None] - h * (dr * r ** 3 / h.shape[1])[:, None]
        if s["dres"] is not None:
            dx += s["dres"].to(d)
        return {"dx": dx, "dgamma": torch.einsum("th,th,t->h", dy, h, r)}
    if op in ("router", "router_bwd"):
        x = s["logits"].to(d)
        sc = torch.sigmoid(x) if case["score"] == "sigmoid" else torch.nan_to_num(torch.softmax(x, 1), nan=0.0)
        if op == "router":
            # choice: greedy, one expert at a time, the first of the largest keys
            key = x.clone() if s["bias"] is None else sc + s["bias"].to(d)
            key[x == NEG_INF] = NEG_INF
            if case["groups"] > 1:
                gk = key if case["top"] == 1 or s["bias"] is not None else torch.where(x == NEG_INF, NEG_INF, sc)
                gs = gk.view(case["T"], case["groups"], -1).topk(case["top"], dim=2).values.sum(2)
                out = torch.ones_like(gs, dtype=torch.bool)
                for _ in range(case["keep"]):
                    out[torch.arange(case["T"], device=x.device), torch.where(out, gs, math.nan).nan_to_num(NEG_INF).argmax(1)] = False
                key.view(case["T"], case["groups"], -1)[out] = NEG_INF
            if s["mask"] is not None:
                key[s["mask"] == 0] = NEG_INF
            chosen = []
            for _ in range(case["k"]):
                v, i = key.max(1, keepdim=True)
                first = (key == v).int().argmax(1, keepdim=True)
                chosen.append(torch.where(v == NEG_INF, -1, first))
                key.scatter_(1, first, NEG_INF)
            idx = torch.cat(chosen, 1)
        else:
            idx = s["idx"].long()
        on, at, f = idx >= 0, idx.clamp(min=0), _factor(case)
        sel = torch.where(on, sc.gather(1, at), 0.0)
        if case["score"] == "softmax" and case["renorm"]:
            xs = torch.where(on, x.gather(1, at), NEG_INF)
            w = torch.nan_to_num(torch.softmax(xs, 1), nan=0.0)
        elif case["renorm"]:
            w = sel / (sel.sum(1, keepdim=True) + 1e-20)
        else:
            w = sel
        if op == "router":
            return {"idx": None, "prob": f * w, "load": None}
        # vector-Jacobian products of the three steps: weights <- selected scores <- scores <- logits
        gr = torch.where(on, s["dprob"].to(d) * f, 0.0)
        ds = torch.zeros(case["T"], case["n"] + 1, dtype=d, device=x.device)
        if case["renorm"] and case["score"] == "softmax":
            ds.scatter_add_(1, idx + 1, w * (gr - (gr * w).sum(1, keepdim=True)))
            return {"dlogits": ds[:, 1:]}
        if case["renorm"]:
            gr = torch.where(on, (gr - (gr * w).sum(1, keepdim=True)) / (sel.sum(1, keepdim=True) + 1e-20), 0.0)
        ds.scatter_add_(1, idx + 1, gr)
        ds = ds[:, 1:]
        if case["score"] == "sigmoid":
            return {"dlogits": ds * sc * torch.sigmoid(-x)}
        return {"dlogits": sc * (ds - (ds * sc).sum(1, keepdim=True))}
    if op == "mxfp4_cast":
        w = s["w"].transpose(1, 2) if case["col"] else s["w"]
        v = torch.empty(w.shape, dtype=d, device=w.device)
        for e in range(case["G"]):
            b = w[e].to(d).contiguous()
            v[e] = _block_round64(b.view(b.shape[0], -1, 32), 2, 6.0, 1).view(b.shape)
        return {"v": v}
    # the product, expert by expert
    E, K, N = case["E"], case["K"], case["N"]
    if 2.0 * sum(_counts(case)) * N * K > 4e12:
        return None
    off = s["offsets"].tolist()
    cnt = s["counts"].tolist()
    mag = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
    grid = torch.tensor(mag + tuple(-m for m in mag), dtype=d, device=DEV)
    kb = _pitch(K) // 128
    scales = s["ws"].view(E, -1, kb, 2, 32, 4, 4)
    y = torch.zeros(s["R"], N // 2 if case["glu"] else N, dtype=d, device=DEV)
    for e in range(E):
        if not cnt[e]:
            continue
        lo, hi = off[e], off[e] + cnt[e]
        n = torch.arange(N, device=DEV)[:, None]
        b = torch.arange(K // 32, device=DEV)[None, :]
        byte = scales[e][n // 256, b // 4, n % 256 // 128, n % 32, n % 128 // 32, b % 4]
        w = torch.empty(N, K, dtype=d, device=DEV)
        q = s["wq"][e, :, :K // 2].long()
        w[:, 0::2], w[:, 1::2] = grid[q % 16], grid[q // 16]
        w = w.view(N, K // 32, 32) * torch.exp2(byte.to(d) - 127.0)[..., None]
        a = s["xq"][lo:hi].view(torch.float8_e4m3fn).to(d).view(-1, K // 32, 32)
        a = a * torch.exp2(s["xs"][lo:hi].to(d) - 127.0)[..., None]
        r = a.view(-1, K) @ w.view(N, K).T
        if case["glu"]:
            r = (r + s["bias"][e].to(d)).view(hi - lo, N // 64, 2, 32)
            u, g = r[:, :, 0].reshape(hi - lo, -1), r[:, :, 1].reshape(hi - lo, -1).clamp(-7.0, 7.0)
            r = (u + 1.0) * g * torch.sigmoid(1.702 * g)
        y[lo:hi] = r
    return {"y": y}
