"""Rows without an adapter: the output is base's bits (negative zeros and every
NaN among them), in place or not, forward and backward."""
import pytest
import torch

from grouped_gemm_glu_gb300 import ops

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16


def _bits(t):
    return t.contiguous().view(torch.int16)


def _every_value(rows, cols):
    """Rows that hold all 65536 patterns in turn."""
    n = rows * cols
    return (torch.arange(n, device=DEV) * 7 + 32760).remainder(65536).to(torch.int32).to(torch.int16).view(rows, cols).view(BF)


@pytest.mark.parametrize("T,r,G", [(1, 8, 1), (6, 16, 3), (40, 16, 3), (64, 64, 2), (300, 16, 3), (700, 40, 1), (513, 128, 5)])
@pytest.mark.parametrize("order", ["rows", "runs"])
@pytest.mark.parametrize("inplace", [False, True])
def test_rows_without_an_adapter_are_bases_bits(T, r, G, order, inplace):
    g = torch.Generator().manual_seed(T + r)
    K, N = 136, 264
    f = lambda *s: torch.randn(*s, generator=g).to(BF).to(DEV)
    A, B, scale = f(G, r, K), f(G, r, N), torch.ones(G, device=DEV)
    idx = torch.randint(-1, G, (T,), generator=g)
    if order == "runs":
        idx = torch.sort(idx).values
    idx[0] = -1
    idx[T // 2] = G + 5
    idx = idx.to(torch.int32).to(DEV)
    none = (idx < 0) | (idx >= G)
    x, dy = f(T, K), f(T, N)
    base = _every_value(T, N)
    keep = _bits(base).clone()
    o = ops.lora(x, A, B, idx, scale, base=base, out=base if inplace else None)
    assert torch.equal(_bits(o["y"])[none], keep[none])
    assert not bool(_bits(o["h"])[none].any())
    base = _every_value(T, K)
    keep = _bits(base).clone()
    h = torch.zeros(T, r, dtype=BF, device=DEV)
    dx, _, _ = ops.lora_bwd(dy, x, h, A, B, idx, scale, base=base, out=base if inplace else None)
    assert torch.equal(_bits(dx)[none], keep[none])
    # without base they are zero, of the positive kind
    assert not bool(_bits(ops.lora(x, A, B, idx, scale)["y"])[none].any())
    assert not bool(_bits(ops.lora_bwd(dy, x, h, A, B, idx, scale)[0])[none].any())
