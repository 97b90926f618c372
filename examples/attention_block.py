"""A stack of causal transformer blocks (ResidualAttention and ResidualMLP) trained for a few
steps, against the same stack in plain torch operations: loss of each step, time of a step
and peak memory of both; then a few tokens generated through a cache.

    python examples/attention_block.py [--batch 2] [--rows 2048] [--cols 1024] [--heads 8]
                                       [--kv-heads 2] [--layers 2] [--steps 6] [--dtype bf16]
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from place_batchnorm_activation_amd import RotarySpec  # noqa: E402
from place_batchnorm_activation_amd.attention import KVCache, ResidualAttention  # noqa: E402
from place_batchnorm_activation_amd.residual import ResidualMLP, ResNorm  # noqa: E402


class Stack(torch.nn.Module):
    def __init__(self, cols, heads, kv_heads, layers, dtype, device):
        super().__init__()
        turn = RotarySpec(cols // heads, device=device)
        self.blocks = torch.nn.ModuleList()
        for _ in range(layers):
            self.blocks.append(ResidualAttention(cols, heads, kv_heads, rotary=turn, device=device,
                                                 dtype=dtype))
            self.blocks.append(ResidualMLP(cols, 2 * cols, device=device, dtype=dtype))
        self.last = ResNorm(cols, post="rms", pre="rms", device=device)

    def forward(self, x, caches=None):
        r, b, i = x, None, 0
        for block in self.blocks:
            if isinstance(block, ResidualAttention):
                r, b = block(r, b, cache=None if caches is None else caches[i])
                i += 1
            else:
                r, b = block(r, b)
        return self.last(r, b)[1]

    def plain(self, x):
        """The same function in torch operations."""
        def rms(x, w, eps):
            x = x.float()
            return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps) * w

        def boundary(norm, r, b):
            if b is not None:
                r = r + norm.alpha * rms(b, norm.post_weight, norm.eps)
            return r.to(x.dtype), rms(r, norm.pre_weight, norm.eps).to(x.dtype)

        def turned(t, co, si):
            a, c = t.float().chunk(2, -1)
            return torch.cat((a * co - c * si, c * co + a * si), -1)

        r, b = x, None
        S = x.shape[1]
        hidden = torch.ones(S, S, dtype=torch.bool, device=x.device).triu(1)
        for block in self.blocks:
            r, n = boundary(block.norm, r, b)
            if isinstance(block, ResidualMLP):
                g, u = (n @ block.up.weight.t()).chunk(2, -1)
                b = (torch.nn.functional.silu(g.float()) * u.float()).to(x.dtype) @ \
                    block.down.weight.t()
                continue
            H, KV, D = block.heads, block.kv_heads, block.head_dim
            qkv = (n @ block.qkv.weight.t()).unflatten(-1, (H + 2 * KV, D)).transpose(1, 2)
            q, k, v = qkv.split((H, KV, KV), 1)
            angle = torch.arange(S, device=x.device)[:, None] * block.rotary.inv_freq
            co, si = angle.cos().float(), angle.sin().float()
            q, k = turned(q, co, si), turned(k, co, si).repeat_interleave(H // KV, 1)
            v = v.float().repeat_interleave(H // KV, 1)
            s = q @ k.transpose(-1, -2).contiguous() * D ** -0.5
            p = torch.softmax(s.masked_fill(hidden, -float("inf")), -1)
            b = (p @ v).to(x.dtype).transpose(1, 2).flatten(-2) @ block.out.weight.t()
        return boundary(self.last, r, b)[1]


def train(model, forward, x, target, steps, lr):
    opt = torch.optim.SGD(model.parameters(), lr=lr)
    losses, begin = [], 0.0
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
    return [float(v) for v in losses], ms, torch.cuda.max_memory_allocated()


@torch.no_grad()
def generate(model, x, tokens):
    """The outputs of x's rows one after another, each over the caches of the ones before."""
    blocks = [b for b in model.blocks if isinstance(b, ResidualAttention)]
    caches = [KVCache(x.shape[0], tokens, b.kv_heads, b.head_dim, x.dtype, x.device) for b in blocks]
    return torch.cat([model(x[:, i:i + 1], caches) for i in range(tokens)], 1)


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__,
                                 formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("batch", 2), ("rows", 2048), ("cols", 1024), ("heads", 8),
                        ("kv-heads", 2), ("layers", 2), ("steps", 6), ("tokens", 16)):
        ap.add_argument("--" + name, type=int, default=value)
    ap.add_argument("--dtype", choices=("f32", "bf16", "f16"), default="bf16")
    ap.add_argument("--lr", type=float, default=0.05)
    a = ap.parse_args(argv)
    dtype = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[a.dtype]
    gen = torch.Generator(device="cuda").manual_seed(0)
    x = torch.randn(a.batch, a.rows, a.cols, generator=gen, device="cuda").to(dtype)
    target = torch.randn(a.batch, a.rows, a.cols, generator=gen, device="cuda")
    results = []
    for kind in ("the library's", "plain"):
        torch.manual_seed(1)
        model = Stack(a.cols, a.heads, a.kv_heads, a.layers, dtype, "cuda")
        losses, ms, peak = train(model, model if kind != "plain" else model.plain, x, target,
                                 a.steps, a.lr)
        print("%-15s %8.2f ms a step, peak %7.1f MiB, loss %s" % (
            kind, ms, peak / 2 ** 20, " ".join("%.5f" % v for v in losses)), flush=True)
        results.append((losses, ms, peak))
        if kind != "plain":
            n = min(a.tokens, a.rows)
            with torch.no_grad():
                off = (generate(model, x, n).float() - model(x)[:, :n].float()).abs().max()
            print("%d tokens through the caches: at most %.2g from the whole rows' pass"
                  % (n, float(off)), flush=True)
        del model
        torch.cuda.empty_cache()
    return results


if __name__ == "__main__":
    main()
