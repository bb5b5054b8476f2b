"""GPU tests of the AdamW step against its formula in 64 bits.

Tolerances (u = 2^-24, a rounding to fp32; P = |b1 m|, Q = |(1 - b1) g'|):
  * norm: eight squares are added by fused multiply-adds (relative error at
    most 8 u), these sums with their errors, the root halves it and the result
    is rounded: 5 u; the clipping factor c has that error too;
  * m = fma(b1, m, a1 g): both constants rounded (u each), a product and the sum
    rounded: |err| <= 2 u P + 3 u Q, and 5 u Q for c: at most 8 u (P + Q);
  * v likewise with g squared (one rounding more) and c twice: 16 u v (all
    terms are positive);
  * w: the quotient's error is m's over the denominator, plus the square root's
    approximation (2 u, and 8 u from v), root, eps and their sum (3 u), the
    division (2 ulp = 4 u), step (u), the product with it inside an fma; w keep
    rounds keep, the product and the sum: |err| <= 4 u |w| + 32 u step (P + Q) /
    denominator;
  * 8-bit moments hold exactly the 64-bit formula's values; with clipping an
    element within c's error of its turning point may turn: 5 u of its value,
    which is at most 16 distances of codes: 80 u < 2^-17 of a distance (and of
    a block's largest value at the limit of its scale: not drawn here).
"""
import pytest
import torch

from adamw_ref import U, held, random_bits, step, two_to
from grouped_gemm_glu_gb300 import lib as L
from grouped_gemm_glu_gb300 import ops
from grouped_gemm_glu_gb300.optim import AdamW

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F64 = torch.float64
BF, F32 = torch.bfloat16, torch.float32


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _randn(g, n):
    return torch.randn(n, generator=g)


class Case:
    """Tensors of given sizes, some of them views off their storage's alignment."""

    def __init__(self, sizes, wtypes, gtypes, seed=0, offset=0, **kw):
        g = _gen(seed)
        self.g, self.sizes = g, sizes
        pick = lambda ts, i: ts[i % len(ts)]
        self.wt, self.gt = [pick(wtypes, i) for i in range(len(sizes))], [pick(gtypes, i) for i in range(len(sizes))]
        self.offset = offset
        self.w = [self._put(_randn(g, n) * 0.05, t) for n, t in zip(sizes, self.wt)]
        self.kw = dict(lr=1e-3, betas=(0.9, 0.95), eps=1e-8, weight_decay=[0.1 * (i % 3) for i in range(len(sizes))],
                       seed=12345, grad_dtype=self.gt)
        self.kw.update(kw)
        self.opt = AdamW(self.w, **self.kw)
        self.scale = [float(torch.exp(_randn(g, 1)) * 0.01) for _ in sizes]

    def _put(self, v, t):
        full = torch.zeros(v.numel() + self.offset, dtype=t, device=DEV)
        full[self.offset:] = v.to(DEV).to(t)
        return full[self.offset:]

    def grads(self):
        out = []
        for n, t, s in zip(self.sizes, self.gt, self.scale):
            v = _randn(self.g, n) * s
            v[torch.rand(n, generator=self.g) < 0.05] = 0
            if n > 70:
                v[32:64] = 0  # a whole block without a gradient
            out.append(self._put(v, t))
        return out

    def before(self):
        o = self.opt
        mom = [tuple(x.cpu().to(F64) for x in o.moments(i)) for i in range(len(self.sizes))]
        ws = []
        for w, at in zip(self.w, o._at):
            ws.append((o.master[at:at + w.numel()] if w.dtype == BF else w).cpu().to(F64))
        return ws, mom, int(o.t)

    def check(self, grads, was, norm=None):
        """After a step with grads from the state `was`."""
        ws, mom, t = was
        kw, o = self.kw, self.opt
        assert int(o.t) == t + 1
        lr = float(torch.tensor(kw["lr"], dtype=F32))
        total = sum(float(g.cpu().to(F64).square().sum()) for g in grads) ** 0.5
        clip = kw.get("max_norm")
        c = min(1.0, clip / (total + 1e-6)) if clip else 1.0
        if clip:
            assert abs(float(norm) - total) <= 5 * U * total
        now = self.before()
        b1, b2 = kw["betas"]
        for i, n in enumerate(self.sizes):
            gd = grads[i].cpu().to(F64)
            wd = float(torch.tensor(kw["weight_decay"][i], dtype=F32))
            w, m, v = step(ws[i], mom[i][0], mom[i][1], gd, t + 1, lr, kw["betas"], kw["eps"], wd, c)
            pq = (b1 * mom[i][0]).abs() + ((1 - b1) * c * gd).abs()
            denom = torch.sqrt(v / (1 - b2 ** (t + 1))) + kw["eps"]
            lim = 4 * U * ws[i].abs() + 32 * U * lr / (1 - b1 ** (t + 1)) * pq / denom
            bad = (now[0][i] - w).abs() > lim
            assert not bad.any(), (i, n, int(bad.sum()), float(((now[0][i] - w).abs() - lim).max()))
            if self.w[i].dtype == BF:
                assert torch.equal(self.w[i].cpu(), now[0][i].float().to(BF))
            if o.state == "f32":
                assert bool(((now[1][i][0] - m).abs() <= 8 * U * pq).all()), (i, n)
                assert bool(((now[1][i][1] - v).abs() <= 16 * U * v).all()), (i, n)
            else:
                bits = random_bits(kw["seed"], t + 1, i, torch.arange(n))
                root = torch.sqrt(now[1][i][1])  # of exact squares
                for got, x, b, least in ((now[1][i][0], m, bits >> 16, False), (root, torch.sqrt(v), bits & 0xFFFF, True)):
                    want, margin = held(x, b, least)
                    off = got != want
                    assert not bool((off & (margin > (2.0 ** -17 if clip else 0.0))).any()), (i, n, int(off.sum()))


SIZES = [1, 31, 32, 33, 0, 257, 2047, 2048, 2049, 5003, 70001]


@pytest.mark.parametrize("state", ["f32", "mxfp8"])
@pytest.mark.parametrize("wtypes,gtypes", [((F32,), (F32,)), ((BF,), (BF,)), ((BF, F32), (BF, F32, F32))])
@pytest.mark.parametrize("clip", [None, 0.5, 1e6])
@pytest.mark.parametrize("offset", [0, 1])
def test_steps(state, wtypes, gtypes, clip, offset):
    c = Case(SIZES, wtypes, gtypes, seed=3 + offset, offset=offset, state=state, max_norm=clip)
    for _ in range(3):
        was = c.before()
        g = c.grads()
        norm = c.opt.step(g)
        assert (norm is None) == (clip is None)
        c.check(g, was, norm)


@pytest.mark.parametrize("state", ["f32", "mxfp8"])
@pytest.mark.parametrize("count", [65, 513, 4001, 8100])
def test_many_tensors(state, count):
    # more than the short launch's addresses, more than one launch's
    c = Case([1 + (i * 7) % 50 for i in range(count)], (BF,), (BF,), state=state, max_norm=0.25)
    was = c.before()
    g = c.grads()
    c.check(g, was, c.opt.step(g))


@pytest.mark.parametrize("n", [1, 64, 100000])
def test_wide_ranges_in_8_bits(n):
    # values far below their block's largest: codes below the normal ones, the least code, exact zeros
    c = Case([n], (F32,), (F32,), state="mxfp8", betas=(0.9, 0.999))
    for k in range(4):
        was = c.before()
        g = [x * torch.exp2(torch.randint(-30, 1, x.shape, generator=_gen(k)).float().to(DEV)) for x in c.grads()]
        c.opt.step(g)
        c.check(g, was)
    m, v = c.opt.moments(0)
    assert bool((v[(g[0] != 0)] > 0).all())  # the least code


def test_sums_on_the_turning_points():
    # gradients and codes of few bits: b1 m + (1 - b1) g falls on codes' turning points far more often than by chance
    n = 1 << 16
    c = Case([n], (F32,), (BF,), state="mxfp8", betas=(0.5, 0.75))
    gen = _gen(1)
    for _ in range(3):
        was = c.before()
        g = [(torch.randint(-8, 9, (n,), generator=gen).float() * 0.125).to(BF).to(DEV)]
        c.opt.step(g)
        c.check(g, was)


def test_rounding_is_unbiased():
    # 2^20 equal elements: the mean of what is held is the value, within 5 standard deviations of the mean
    # (a two-point distribution over one distance of codes: at most half a distance each)
    n = 1 << 20
    w = torch.zeros(n, device=DEV)
    opt = AdamW([w], lr=0.0, betas=(0.9, 0.999), state="mxfp8", seed=7)
    g = torch.full((n,), 0.0137, device=DEV)
    opt.step([g])
    m, v = (x.to(F64) for x in opt.moments(0))
    for got, x in ((m, 0.1 * float(g[0])), (v.sqrt(), (0.001 * float(g[0]) ** 2) ** 0.5)):
        gap = float(got.max() - got.min())
        assert 0 < gap <= 0.13 * x and abs(float(got.mean()) - x) <= 5 * 0.5 * gap / n ** 0.5
    # and sqrt(v) falls by sqrt(b2) a step on average, which rounding to the nearest would never do
    r = float(v.sqrt().mean())
    z = torch.zeros_like(g)
    steps = 100
    for _ in range(steps):
        opt.step([z])
    # E[sqrt(b2) s] each step; deviation of the mean of n independent elements: at most steps^.5 / 2 distances
    # a element (codes below the start lie no further apart), 5 standard deviations
    want = r * 0.999 ** (steps / 2)
    assert abs(float(opt.moments(0)[1].to(F64).sqrt().mean()) - want) <= 5 * 0.5 * gap * (steps / n) ** 0.5


@pytest.mark.parametrize("state", ["f32", "mxfp8"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), 3e19])
def test_norm_that_is_not_finite_changes_nothing(state, bad):
    c = Case([100, 5000], (BF,), (F32,), state=state, max_norm=1.0)
    c.opt.step(c.grads())
    keep = {k: v.clone() for k, v in c.opt.state_dict().items()}
    w = [x.clone() for x in c.w]
    g = c.grads()
    g[1][4321] = bad
    norm = c.opt.step(g)
    assert not bool(torch.isfinite(norm))
    assert all(torch.equal(a, b) for a, b in zip(w, c.w))
    assert all(torch.equal(v, keep[k]) for k, v in c.opt.state_dict().items())
    was = c.before()
    g = c.grads()
    c.check(g, was, c.opt.step(g))  # and the next one goes on


def test_nonfinite_gradients_without_clipping_stay_in_their_block():
    for state in ("f32", "mxfp8"):
        c = Case([200], (F32,), (F32,), state=state)
        g = c.grads()
        g[0][70] = float("nan")
        g[0][130] = float("inf")
        c.opt.step(g)
        assert [int(i) for i in torch.nonzero(~torch.isfinite(c.w[0])).view(-1)] == [70, 130]
        m, v = c.opt.moments(0)
        off = torch.nonzero(~torch.isfinite(m)).view(-1).tolist()
        assert off == ([70, 130] if state == "f32" else list(range(64, 96)) + list(range(128, 160)))


@pytest.mark.parametrize("state", ["f32", "mxfp8"])
def test_captured_steps_equal_eager_ones(state):
    a = Case(SIZES, (BF, F32), (BF,), seed=5, state=state, max_norm=0.1)
    b = Case(SIZES, (BF, F32), (BF,), seed=5, state=state, max_norm=0.1)
    grads = [torch.zeros_like(x) for x in a.grads()]
    b.grads()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    keep = a.opt.state_dict()
    weights = [x.clone() for x in a.w]
    with torch.cuda.stream(s):
        a.opt.step(grads)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            a.opt.step(grads)
    torch.cuda.synchronize()
    for x, y in zip(a.w, weights):
        x.copy_(y)
    a.opt.load_state_dict(keep)
    for lr in (1e-3, 1e-3, 3e-4):
        new = a.grads()
        other = b.grads()
        assert all(torch.equal(x, y) for x, y in zip(new, other))
        for x, y in zip(grads, new):
            x.copy_(y)
        a.opt.set_lr(lr)
        b.opt.set_lr(lr)
        g.replay()
        b.opt.step(other)
        assert torch.equal(a.opt.norm, b.opt.norm)
        assert all(torch.equal(x, y) for x, y in zip(a.w, b.w))
        assert all(torch.equal(v, b.opt.state_dict()[k]) for k, v in a.opt.state_dict().items())


def test_steps_on_another_stream_and_same_results_twice():
    c = [Case([100003], (BF,), (BF,), seed=9, state="mxfp8", max_norm=0.1) for _ in range(2)]
    g = [x.grads() for x in c]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        c[0].opt.step(g[0])
    torch.cuda.current_stream().wait_stream(s)
    c[1].opt.step(g[1])
    assert torch.equal(c[0].w[0], c[1].w[0]) and torch.equal(c[0].opt.m, c[1].opt.m) and torch.equal(c[0].opt.v, c[1].opt.v)


def test_neighbours_are_left_alone():
    # weights that are stretches of one buffer, with gaps: the gaps keep their values
    for t in (F32, BF):
        buf = torch.full((9000,), 7.0, dtype=t, device=DEV)
        ws = [buf[3:1004], buf[1010:1011], buf[2000:4051]]
        opt = AdamW(ws, lr=1e-2)
        opt.step([torch.ones_like(w) for w in ws])
        mask = torch.ones(9000, dtype=torch.bool, device=DEV)
        for a, b in ((3, 1004), (1010, 1011), (2000, 4051)):
            mask[a:b] = False
        assert bool((buf[mask] == 7.0).all())
        # the step takes lr (1 + 0.01 * 7) = 0.0107 off: a bf16 7, whose neighbours are 2^-5 away, keeps its value (its
        # master does not)
        for w, at in zip(ws, opt._at):
            moved = w if t == F32 else opt.master[at:at + w.numel()]
            assert bool(((moved.double() - (7 - 0.0107)).abs() < 1e-5).all())
            assert t == F32 or bool((w == 7.0).all())


def test_state_travels():
    a = Case([1000, 77], (BF, F32), (F32,), state="mxfp8")
    a.opt.step(a.grads())
    b = AdamW([w.clone() for w in a.w], **{**a.kw})
    b.load_state_dict(a.opt.state_dict())
    g = a.grads()
    a.opt.step(g)
    b.step(g)
    assert all(torch.equal(x, y) for x, y in zip(a.w, b.weights))
    with pytest.raises(ValueError):
        AdamW([w.clone() for w in a.w], lr=1e-3).load_state_dict(a.opt.state_dict())


def test_more_than_2_to_32_elements():
    n = (1 << 32) + 1000
    if torch.cuda.mem_get_info()[0] < 80 << 30:
        pytest.skip("80 GB of free device memory are needed")
    w = torch.zeros(n, dtype=F32, device=DEV)
    g = torch.zeros(n, dtype=BF, device=DEV)
    tail = slice(n - 4096, n)
    gv = (_randn(_gen(2), 4096) * 0.01).to(BF)
    g[tail] = gv.to(DEV)
    opt = AdamW([w], lr=1e-3, betas=(0.9, 0.95), weight_decay=0.0, grad_dtype=BF, state="mxfp8", seed=5, max_norm=1e9)
    norm = opt.step([g])
    total = float(gv.to(F64).square().sum()) ** 0.5
    assert abs(float(norm) - total) <= 5 * U * total
    z = torch.zeros(4096, dtype=F64)
    wr, m, v = step(z, z, z, gv, 1, float(torch.tensor(1e-3)), (0.9, 0.95), 1e-8, 0.0)
    assert float((w[tail].cpu().to(F64) - wr).abs().max()) <= 64 * U * 1e-3
    assert float(w[: n - 4096].abs().max()) == 0.0
    idx = torch.arange(n - 4096, n)
    bits = random_bits(5, 1, 0, idx)
    # (the stretch starts inside a block: compare from its first whole block on)
    skip = -(n - 4096) % 32
    up = (n + 31) // 32 * 32
    q = slice(n - 4096 + skip, up)
    s = slice(q.start // 32, up // 32)
    got = opt.m[q].cpu().view(torch.float8_e4m3fn).to(F64).view(-1, 32) * two_to(opt.ms[s].cpu().long() - 127).view(-1, 1)
    want, _ = held(m[skip:], bits[skip:] >> 16, False)
    assert torch.equal(got.view(-1)[: want.numel()], want)
    del w, g, opt
    torch.cuda.empty_cache()


def test_refusals():
    w = torch.zeros(64, device=DEV)
    opt = AdamW([w, torch.zeros(4, 4, device=DEV, dtype=BF)], lr=1e-3)
    ok = [torch.zeros(64, device=DEV), torch.zeros(4, 4, device=DEV, dtype=BF)]
    opt.step(ok)
    for bad in ([ok[0]], [ok[0], ok[0]], [ok[0].to(BF), ok[1]], [ok[0].cpu(), ok[1]], [ok[0], ok[1].view(16)],
                [torch.zeros(128, device=DEV)[::2], ok[1]]):
        with pytest.raises(ValueError):
            opt.step(bad)
    for kw in (dict(lr=-1.0), dict(betas=(1.0, 0.9)), dict(betas=(0.9, -0.1)), dict(eps=-1e-8), dict(max_norm=0.0),
               dict(weight_decay=[0.1, 0.1]), dict(weight_decay=-0.1), dict(state="int8"), dict(grad_dtype=torch.float16)):
        with pytest.raises(ValueError):
            AdamW([w], **{"lr": 1e-3, **kw})
    for ws in ([w, w], [w[:40], w[30:]], [w[::2]], [w.half()], [w.cpu()]):
        with pytest.raises(ValueError):
            AdamW(ws, lr=1e-3)
    AdamW([], lr=1e-3).step([])
    assert ops.read_status(ops.new_status(DEV)) == L.MOE_OK


@pytest.mark.parametrize("state", ["f32", "mxfp8"])
@pytest.mark.parametrize("betas", [(0.0, 0.0), (0.0, 0.999), (0.9, 0.0)])
def test_betas_of_zero(state, betas):
    c = Case([33, 5003], (BF, F32), (BF, F32), seed=8, state=state, betas=betas, max_norm=0.5)
    for _ in range(2):
        was = c.before()
        g = c.grads()
        c.check(g, was, c.opt.step(g))


def test_replaced_memory():
    # the step goes on with the memory that the weight had, and leaves the new one alone
    w = torch.ones(5000, device=DEV)
    old = w.detach()
    opt = AdamW([w], lr=0.5, weight_decay=0.0)
    w.data = torch.ones(5000, device=DEV)
    del old
    others = [torch.ones(5000, device=DEV) for _ in range(4)]  # (would take freed memory)
    opt.step([torch.ones(5000, device=DEV)])
    assert bool((w == 1).all()) and all(bool((o == 1).all()) for o in others)
    assert bool((opt._memory[0] < 1).all())
