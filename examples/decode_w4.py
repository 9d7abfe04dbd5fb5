"""One decode step on 4-bit weights: router, experts and an output projection.

Quantises random weights of a small mixture-of-experts layer to a 4-bit format,
captures  route -> experts -> projection  into one CUDA graph over buffers that
a program would keep, replays it on new tokens, and checks the result against
the same layer in 64 bits on the dequantised weights.

    python examples/decode_w4.py [--format mxfp4|int4] [--tokens 4] [--steps 3]
"""

from __future__ import annotations

import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import fp8_block_scale_x128_gb300 as fb  # noqa: E402

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def dequantised(codes: torch.Tensor, scales: torch.Tensor, fmt: int, group: int) -> torch.Tensor:
    """float64 [..., K] of a quantised weight."""
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).int()
    if fmt == fb.FP8BS_W4_MXFP4:
        v = torch.tensor(E2M1 + tuple(-t for t in E2M1), dtype=torch.float64, device=codes.device)[c]
        s = 2.0 ** (scales.double() - 127)
    else:
        v, s = c.double() - 8, scales.double()
    return (v.unflatten(-1, (-1, group)) * s.unsqueeze(-1)).flatten(-2)


class Layer:
    """A mixture-of-experts layer (E routed experts and a shared one) and its
    output projection, with the buffers of one decode step."""

    def __init__(self, tokens: int, hidden: int, inter: int, experts: int, k: int, out: int, fmt: int, group: int,
                 seed: int = 0):
        dev = torch.device("cuda")
        g = torch.Generator(device=dev)
        g.manual_seed(seed)
        self.fmt, self.group, self.k, self.experts = fmt, group, k, experts

        def weight(rows, cols):
            return fb.fp8bs_quant_weight_w4(torch.randn((rows, cols), generator=g, device=dev) * 0.02, fmt, group)

        E = experts + 1
        self.router = (torch.randn((experts, hidden), generator=g, device=dev) * 0.02).to(torch.bfloat16)
        c, s = weight(E * 2 * inter, hidden)
        self.w13, self.s13 = c.view(E, 2 * inter, -1), s.view(E, 2 * inter, -1)
        c, s = weight(E * hidden, inter)
        self.w2, self.s2 = c.view(E, hidden, -1), s.view(E, hidden, -1)
        self.wo, self.so = weight(out, hidden)
        self.x = torch.zeros((tokens, hidden), dtype=torch.bfloat16, device=dev)
        self.ids = torch.zeros((tokens, k + 1), dtype=torch.int32, device=dev)
        self.weights = torch.zeros((tokens, k + 1), dtype=torch.float32, device=dev)
        self.y = torch.zeros((tokens, hidden), dtype=torch.bfloat16, device=dev)
        self.out = torch.zeros((tokens, out), dtype=torch.bfloat16, device=dev)
        self.route_ws = fb.new_moe_route_workspace(tokens, experts, hidden)
        self.moe_ws = fb.new_moe_w4_workspace(tokens, k + 1, inter)

    def step(self) -> None:
        fb.fp8bs_moe_route(self.x, self.router, self.k, shared="one", ids=self.ids, weights=self.weights,
                           workspace=self.route_ws)
        fb.fp8bs_moe_w4a16(self.x, self.ids, self.weights, self.w13, self.s13, self.w2, self.s2, self.fmt, self.group,
                           y=self.y, workspace=self.moe_ws)
        # nothing unfinished writes the projection's weight: it may be read early
        fb.fp8bs_gemv_w4a16(self.y, self.wo, self.so, self.fmt, self.group, y=self.out, pdl=True)

    def reference(self) -> torch.Tensor:
        x = self.x.double()
        logits = x @ self.router.double().t()
        top = logits.topk(self.k, dim=1)
        w = torch.softmax(top.values, 1)
        y = torch.zeros_like(x)
        for m in range(x.shape[0]):
            chosen = [(int(e), float(v)) for e, v in zip(top.indices[m], w[m])] + [(self.experts, 1.0)]
            for e, v in chosen:
                gate, up = (dequantised(self.w13[e], self.s13[e], self.fmt, self.group) @ x[m]).chunk(2)
                y[m] += v * (dequantised(self.w2[e], self.s2[e], self.fmt, self.group) @ (torch.nn.functional.silu(gate) * up))
        return y @ dequantised(self.wo, self.so, self.fmt, self.group).t()


def main(argv=None) -> float:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--format", choices=("mxfp4", "int4"), default="mxfp4")
    ap.add_argument("--tokens", type=int, default=4)
    ap.add_argument("--hidden", type=int, default=1024)
    ap.add_argument("--inter", type=int, default=256)
    ap.add_argument("--experts", type=int, default=32)
    ap.add_argument("--k", type=int, default=4)
    ap.add_argument("--out", type=int, default=1000)
    ap.add_argument("--steps", type=int, default=3)
    a = ap.parse_args(argv)
    fb.build()
    fmt, group = (fb.FP8BS_W4_MXFP4, 32) if a.format == "mxfp4" else (fb.FP8BS_W4_INT4, 128)
    layer = Layer(a.tokens, a.hidden, a.inter, a.experts, a.k, a.out, fmt, group)
    layer.step()  # set-up outside the capture
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.step()
    worst = 0.0
    for i in range(a.steps):
        layer.x.copy_(torch.randn(layer.x.shape, generator=torch.Generator().manual_seed(100 + i)).to(torch.bfloat16))
        graph.replay()
        torch.cuda.synchronize()
        ref = layer.reference()
        rel = float((layer.out.double() - ref).norm() / ref.norm())
        worst = max(worst, rel)
        print(f"step {i}: experts of token 0: {layer.ids[0].tolist()}, output off by {rel:.2e} (relative 2-norm)")
    status = fb.fp8bs_check_error(layer.moe_ws)
    if status != 0:
        raise fb.Fp8bsError(status, "fp8bs_moe_w4a16")
    return worst


if __name__ == "__main__":
    main()
