"""A stack of residual MLP blocks trained for a few steps, its activations kept in
8 bits (place_batchnorm_activation_amd.residual), against the same stack in plain torch
operations: loss of each step, time of a step and peak memory of both.

    python examples/residual_mlp.py [--rows 8192] [--cols 2048] [--hidden 4096]
                                    [--layers 4] [--steps 8] [--dtype bf16]
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from place_batchnorm_activation_amd.residual import ResidualMLP, ResNorm  # noqa: E402


class Stack(torch.nn.Module):
    def __init__(self, cols, hidden, layers, dtype, device):
        super().__init__()
        self.blocks = torch.nn.ModuleList(
            ResidualMLP(cols, hidden, gate=True, device=device, dtype=dtype) for _ in range(layers))
        self.last = ResNorm(cols, post="rms", pre="rms", device=device)

    def forward(self, x):
        r, b = x, None
        for block in self.blocks:
            r, b = block(r, b)
        return self.last(r, b)[1]

    def plain(self, x):
        """The same function in torch operations, all activations kept by autograd."""
        def rms(x, w, eps):
            x = x.float()
            return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps) * w

        def boundary(norm, r, b):
            if b is not None:
                p = rms(b, norm.post_weight, norm.eps)
                r = r + norm.alpha * (p if norm.gate is None else p * norm.gate)
            return r.to(x.dtype), rms(r, norm.pre_weight, norm.eps).to(x.dtype)

        r, b = x, None
        for block in self.blocks:
            r, n = boundary(block.norm, r, b)
            g, u = (n @ block.up.weight.t()).chunk(2, -1)
            b = (torch.nn.functional.silu(g.float()) * u.float()).to(x.dtype) @ \
                block.down.weight.t()
        return boundary(self.last, r, b)[1]


def train(model, forward, x, target, steps, lr):
    opt = torch.optim.SGD(model.parameters(), lr=lr)
    losses, peak, begin = [], 0, 0.0
    for i in range(steps):
        if i == 1:
            torch.cuda.synchronize()
            torch.cuda.reset_peak_memory_stats()
            begin = time.perf_counter()
        loss = (forward(x).float() - target).square().mean()
        losses.append(loss.detach())
        opt.zero_grad(set_to_none=True)
        loss.backward()
        opt.step()
    torch.cuda.synchronize()
    ms = (time.perf_counter() - begin) / max(1, steps - 1) * 1e3
    peak = torch.cuda.max_memory_allocated()
    return [float(v) for v in losses], ms, peak


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__,
                                 formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("rows", 8192), ("cols", 2048), ("hidden", 4096), ("layers", 4),
                        ("steps", 8)):
        ap.add_argument("--" + name, type=int, default=value)
    ap.add_argument("--dtype", choices=("f32", "bf16", "f16"), default="bf16")
    ap.add_argument("--lr", type=float, default=0.05)
    a = ap.parse_args(argv)
    dtype = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[a.dtype]
    gen = torch.Generator(device="cuda").manual_seed(0)
    x = torch.randn(a.rows, a.cols, generator=gen, device="cuda").to(dtype)
    target = torch.randn(a.rows, a.cols, generator=gen, device="cuda")
    results = []
    for kind in ("kept in 8 bits", "plain"):
        torch.manual_seed(1)
        model = Stack(a.cols, a.hidden, a.layers, dtype, "cuda")
        losses, ms, peak = train(model, model if kind != "plain" else model.plain, x, target,
                                 a.steps, a.lr)
        print("%-15s %8.2f ms a step, peak %7.1f MiB, loss %s" % (
            kind, ms, peak / 2 ** 20, " ".join("%.5f" % v for v in losses)), flush=True)
        results.append((losses, ms, peak))
        del model
        torch.cuda.empty_cache()
    return results


if __name__ == "__main__":
    main()
