"""Decode steps of a small mixture-of-experts model with 4-bit weights.

    python examples/decode_w4_moe.py [--tokens 4] [--layers 4] [--hidden 2048] [--steps 64] ...

A block is x = norm(x + P x), x = norm(x + experts(x)): a projection and a
mixture of experts, their weights quantised to 4 bits when the model is made
(`quantize_w4`), the product `gemm_nt_w4` and the layer `MoeLayer`.  The step
runs once eagerly, is checked in 64 bits against the weights' own values
(`dequantize_w4`) and with the experts that the layer chose, and is then
captured into a HIP graph that is replayed, each step on the one before.
Weights are random.
"""
from __future__ import annotations

import argparse
import math
import sys
import time
from pathlib import Path

import torch

ROOT = Path(__file__).resolve().parent.parent
if str(ROOT) not in sys.path:
    sys.path.insert(0, str(ROOT))

from dense_gemm_18_amd import MoeLayer, W4Weight, dequantize_w4, gemm_nt_w4, quantize_w4  # noqa: E402


def normal(gen, scale, *shape, dtype):
    return (torch.randn(shape, generator=gen, device="cuda") * scale).to(dtype)


def norm(x):
    return x / x.float().square().mean(-1, keepdim=True).add(1e-6).sqrt().to(x.dtype)


class Block:
    """One projection and one mixture of experts."""

    def __init__(self, gen, a):
        dtype, H, I, E = a.dtype, a.hidden, a.inner, a.experts
        self.proj = quantize_w4(normal(gen, 1 / math.sqrt(H), H, H, dtype=dtype), group=a.group,
                                zeros=True)
        # one expert at a time, so the 16-bit weights of a single one are held
        packed = []
        for rows, cols in ((2 * I, H), (H, I)):
            each = [quantize_w4(normal(gen, 1 / math.sqrt(cols), rows, cols, dtype=dtype),
                                group=a.group, zeros=True) for _ in range(E)]
            packed.append(W4Weight(*(torch.stack([getattr(w, part) for w in each])
                                     for part in ("q", "scales", "zeros")),
                                   shape=(E, rows, cols), group=a.group))
        self.moe = MoeLayer(normal(gen, 2 / math.sqrt(H), E, H, dtype=dtype), *packed,
                            topk=a.topk)
        self.w13, self.w2 = packed

    def __call__(self, x):
        x = norm(x + gemm_nt_w4(x, self.proj))
        y, ids, weights = self.moe(x)
        return norm(x + y), ids, weights

    def in_64_bits(self, x, ids, weights):
        x = norm64(x + x @ dequantize_w4(self.proj).double().T)
        w13, w2 = dequantize_w4(self.w13), dequantize_w4(self.w2)
        y = torch.zeros_like(x)
        for t in range(x.shape[0]):
            for e, w in zip(ids[t].tolist(), weights[t].tolist()):
                gate, up = (w13[e].double() @ x[t]).chunk(2)
                y[t] += w * (w2[e].double() @ (gate * torch.sigmoid(gate) * up))
        return norm64(x + y)


def norm64(x):
    return x / x.square().mean(-1, keepdim=True).add(1e-6).sqrt()


def step(blocks, x):
    routed = []
    for block in blocks:
        x, ids, weights = block(x)
        routed.append((ids, weights))
    return x, routed


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--tokens", type=int, default=4)
    p.add_argument("--layers", type=int, default=4)
    p.add_argument("--hidden", type=int, default=2048)
    p.add_argument("--inner", type=int, default=1024)
    p.add_argument("--experts", type=int, default=16)
    p.add_argument("--topk", type=int, default=4)
    p.add_argument("--group", type=int, default=64)
    p.add_argument("--steps", type=int, default=64)
    p.add_argument("--f16", action="store_true", help="float16 instead of bfloat16")
    a = p.parse_args(argv)
    a.dtype = torch.float16 if a.f16 else torch.bfloat16
    gen = torch.Generator(device="cuda").manual_seed(0)
    blocks = [Block(gen, a) for _ in range(a.layers)]
    start = norm(normal(gen, 1.0, a.tokens, a.hidden, dtype=a.dtype))

    out, routed = step(blocks, start)
    want = start.double()
    for block, (ids, weights) in zip(blocks, routed):
        want = block.in_64_bits(want, ids, weights)
    error = float((out.double() - want).norm() / want.norm())

    # the captured step reads x and leaves the next x there
    x = start.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(blocks, x)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        x.copy_(step(blocks, x)[0])
    eager = start
    for _ in range(2):
        graph.replay()
        eager = step(blocks, eager)[0]
    torch.cuda.synchronize()
    same = torch.equal(x, eager)

    times = {}
    for name, run in (("eager", lambda: step(blocks, x)), ("graph", graph.replay)):
        torch.cuda.synchronize()
        begun = time.perf_counter()
        for _ in range(a.steps):
            run()
        torch.cuda.synchronize()
        times[name] = (time.perf_counter() - begun) / max(1, a.steps) * 1e6
    print(f"{a.layers} blocks, {a.tokens} tokens, hidden {a.hidden}, {a.topk} of {a.experts} "
          f"experts of {a.inner}, {a.dtype}, groups of {a.group}: relative error {error:.2e}, "
          f"eager {times['eager']:.0f} us a step, graph {times['graph']:.0f} us, "
          f"graph {'equals' if same else 'DIFFERS FROM'} eager", flush=True)
    return error, same


if __name__ == "__main__":
    main()
