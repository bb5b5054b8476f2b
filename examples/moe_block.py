"""The MoE block end to end on synthetic weights: one training step of norm,
router and experts, and the serving forward on MXFP4 experts for a prompt and
for single tokens.

  python examples/moe_block.py [--workload tiny|gptoss] [--tokens N]

Build the library first: python -c "import __graft_entry__ as g; g.build()"
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from grouped_gemm_glu_gb300 import lib as L  # noqa: E402
from grouped_gemm_glu_gb300 import ops, synth  # noqa: E402
from grouped_gemm_glu_gb300.block import MoeBlock, MoeServer  # noqa: E402
from grouped_gemm_glu_gb300.layer import MoeLayer  # noqa: E402


def ms(fn, n=10):
    """Median time of fn captured in a CUDA graph."""
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        fn()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            fn()
    t = []
    for _ in range(n):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        g.replay()
        b.record()
        torch.cuda.synchronize()
        t.append(a.elapsed_time(b))
    return sorted(t)[n // 2]


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--workload", default="tiny", choices=("tiny", "gptoss"))
    ap.add_argument("--tokens", type=int, default=None, help="tokens of the training step and of the prompt")
    a = ap.parse_args()
    w = synth.WORKLOADS[a.workload]
    T = a.tokens or w.T
    g = torch.Generator(device="cuda").manual_seed(0)
    rn = lambda *s, sc=1.0: (torch.randn(*s, generator=g, device="cuda") * sc).to(torch.bfloat16)
    gamma, Wr = torch.ones(w.H, dtype=torch.bfloat16, device="cuda"), rn(w.n_experts, w.H, sc=w.H ** -0.5)
    W1, W2 = rn(w.E, w.N1, w.H, sc=w.H ** -0.5), rn(w.E, w.F, w.H, sc=w.F ** -0.5)
    b1 = rn(w.E, w.N1, sc=0.02) if w.bias else None
    glu = (L.glu_params("swiglu", alpha=1.702, up_offset=1.0, gate_lo=-7.0, gate_hi=7.0) if w.gpt_oss
           else L.glu_params(w.act))
    router = L.router_params("softmax", renorm=True)
    x, res, dout = rn(T, w.H), rn(T, w.H), rn(T, w.H)

    layer = MoeLayer(W1, W2, T, w.k, (T * w.k + 31 * w.E + 127) // 128 * 128, glu, b1=b1)
    block = MoeBlock(layer, gamma, Wr, router)

    def train():
        block.forward(x, res)
        return block.backward(dout, dout)

    grads = train()
    print(f"training step, {T} tokens: {ms(train):.3f} ms; |dx| {float(grads['dx'].float().norm()):.4g}, busiest expert "
          f"{int(block.load.max())} of {T * w.k} rows")

    server = MoeServer(W1, W2, gamma, Wr, w.k, router, glu, b1=b1)
    ref, _ = block.forward(x, res)
    out, _ = server.step(x, res)
    rel = float((out.float() - ref.float()).norm() / ref.float().norm())
    print(f"serving forward on MXFP4 experts, {T} tokens: {ms(lambda: server.step(x, res)):.3f} ms "
          f"(differs from the bf16-weight forward by {rel:.3f} in the 2-norm)")
    for n in (1, 16):
        print(f"serving forward, {n} token(s): {1e3 * ms(lambda: server.step(x[:n], res[:n])):.1f} us")
    if ops.read_status(layer.status) or ops.read_status(server.status):
        raise SystemExit("a kernel reported an error")


if __name__ == "__main__":
    main()
