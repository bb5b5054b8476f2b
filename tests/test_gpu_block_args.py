"""What MoeBlock and MoeServer refuse: the layer behind a block works on raw
addresses and a fixed number of tokens, so sizes, types and layouts that it
would misread are errors of the host, before anything is launched."""
import pytest
import torch

from grouped_gemm_glu_gb300 import block
from grouped_gemm_glu_gb300 import lib as L
from grouped_gemm_glu_gb300.block import MoeBlock, MoeServer
from grouped_gemm_glu_gb300.layer import MoeLayer

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
T, H, E, F, K = 64, 256, 4, 128, 2


def _z(*s, dt=torch.bfloat16):
    return torch.zeros(*s, dtype=dt, device=DEV)


def _server(**kw):
    a = dict(W1=_z(E, 2 * F, H), W2=_z(E, F, H), gamma=_z(H), Wr=_z(E, H), k=K, router=L.router_params(),
             params=L.glu_params("swiglu"))
    return MoeServer(**{**a, **kw})


def _block(**kw):
    ly = MoeLayer(_z(E, 2 * F, H), _z(E, F, H), T, K, (T * K + 31 * E + 127) // 128 * 128, L.glu_params("swiglu"))
    return MoeBlock(**{**dict(layer=ly, gamma=_z(H), Wr=_z(E, H), router=L.router_params()), **kw})


def test_block_refuses_other_sizes_types_and_layouts():
    b, x = _block(), _z(T, H)
    for bad in (x[: T - 1], torch.cat((x, x[:1])), x[:, : H // 2], x.float(), _z(H, T).t(), x[:1].expand(T, H), x.cpu()):
        with pytest.raises(ValueError):
            b.forward(bad)
    for kw in (dict(residual=x[: T - 1]), dict(residual=x[:1].expand(T, H)), dict(token_mask=_z(T - 1, dt=torch.bool))):
        with pytest.raises(ValueError):
            b.forward(x, **kw)
    b.forward(x, x)
    for bad in (x[: T - 1], x.float(), _z(H, T).t(), x[:1].expand(T, H)):
        with pytest.raises(ValueError):
            b.backward(bad, x)
        with pytest.raises(ValueError):
            b.backward(x, bad)
    for kw in (dict(gamma=_z(H // 2)), dict(gamma=_z(H, dt=torch.float32)), dict(Wr=_z(E, H // 2)), dict(Wr=_z(H)),
               dict(Wr=_z(E, H, dt=torch.float32))):
        with pytest.raises(ValueError):
            _block(**kw)


def test_server_refuses_other_sizes_types_and_layouts():
    for kw in (dict(W1=_z(E, H, 2 * F).transpose(1, 2)), dict(W1=_z(1, 2 * F, H).expand(E, 2 * F, H)), dict(W1=_z(2 * F, H)),
               dict(W1=_z(E, 2 * F, H, dt=torch.float32)), dict(W2=_z(E - 1, F, H)), dict(W2=_z(E, F, H // 2)),
               dict(W2=_z(E, F // 2, H)), dict(W2=_z(E, H, F).transpose(1, 2)), dict(b1=_z(E, F)), dict(b1=_z(1, 2 * F).expand(E, 2 * F)),
               dict(gamma=_z(H // 2)), dict(Wr=_z(E, H // 2)), dict(params=L.glu_params("srelu"))):
        with pytest.raises(ValueError):
            _server(**kw)
    s, x = _server(), _z(3, H)
    for bad in (x[:, : H // 2], x.float(), _z(H, 3).t(), x[0], x.cpu()):
        with pytest.raises(ValueError):
            s.step(bad)
    with pytest.raises(ValueError):
        s.step(x, x[:2])


def test_strided_router_weight_is_taken():
    g = torch.Generator(device=DEV).manual_seed(0)
    Wr = torch.randn(H, E, generator=g, device=DEV).to(torch.bfloat16).t()
    x = torch.randn(T, H, generator=g, device=DEV).to(torch.bfloat16)
    a, b = _block(Wr=Wr, gamma=torch.ones_like(_z(H))), _block(Wr=Wr.contiguous(), gamma=torch.ones_like(_z(H)))
    a.forward(x)
    b.forward(x)
    # (the products may add in another order)
    assert torch.allclose(a.logits.float(), b.logits.float(), rtol=2.0 ** -7, atol=2.0 ** -7)
    assert a.backward(x, x)["dWr"].shape == (E, H)


def test_server_casts_report_to_its_status(monkeypatch):
    """A tile of a weight that never arrives shows in the server's status word."""
    seen, cast = [], block.ops.quantize_mxfp4
    monkeypatch.setattr(block.ops, "quantize_mxfp4", lambda *a, **kw: (seen.append(kw.get("status")), cast(*a, **kw))[1])
    s = _server()
    assert len(seen) == 2 and all(t is s.status for t in seen)


def test_server_takes_an_empty_batch():
    s, x = _server(), _z(0, H)
    for res in (None, x):
        out, h = s.step(x, res)
        assert out.shape == h.shape == (0, H) and out.dtype == h.dtype == torch.bfloat16
    with pytest.raises(ValueError):
        s.step(_z(0, H // 2))
