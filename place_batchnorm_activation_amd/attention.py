"""PyTorch modules of attention: what a block needs next to the norms, linear layers and gated
units of residual.py, and the same for feature maps.

  attention          softmax(scale q k^T) v with autograd: keeps q, k, v, the output and one
                     number a row; the backward recomputes the probabilities
  rotary             rotary positions with several axes, with autograd
  KVCache            keys and values of the tokens so far, for generation
  ResidualAttention  the attention half of a residual block, as ResidualMLP is the other
  MapAttention       attention over the pixels of a feature map behind a group norm

The products with weights are torch's and KeptLinear's; everything between them runs in the
library's HIP kernels.
"""
from __future__ import annotations

from typing import Optional

import torch
from torch.autograd.function import once_differentiable

from . import (AttentionSpec, RotarySpec, attention_lse, attention_workspace,
               iabn_attention_backward, iabn_attention_forward, iabn_rotary)
from .groupnorm import GroupNormAct
from .residual import KeptLinear, ResNorm


def _heads(t):
    """t with contiguous head elements (a copy only where they are not)."""
    return t if t.stride(-1) == 1 or t.shape[-1] <= 1 else t.contiguous()


def _head_dim(D):
    """D, where the attention takes heads of so many elements."""
    if D % 8 or not 8 <= D <= 128:
        raise ValueError("heads of %d elements: a multiple of 8 up to 128 is needed" % D)
    return D


def _fresh(t):
    return torch.empty(t.shape, dtype=t.dtype, device=t.device)


def _outputs(t, packed):
    """Memory for an output shaped as t: rows in no packed sequence, which the library
    leaves alone, are zeros."""
    return torch.zeros(t.shape, dtype=t.dtype, device=t.device) if packed else _fresh(t)


def _kept(seq):
    """A call's sequences as (names, tensors) and plain values, for autograd to keep the tensors
    (which it checks for later writes)."""
    names = [n for n, v in seq.items() if isinstance(v, torch.Tensor)]
    return names, [seq[n] for n in names], {n: v for n, v in seq.items() if n not in names}


class AttentionFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, spec, seq):
        q, k, v = _heads(q), _heads(k), _heads(v)
        train = any(ctx.needs_input_grad)
        out = _outputs(q, seq.get("q_starts") is not None)
        lse = attention_lse(q) if train else None
        iabn_attention_forward(spec, q, k, v, out, lse, attention_workspace(spec, q, k, **seq),
                               **seq)
        if train:
            names, tensors, plain = _kept(seq)
            ctx.save_for_backward(q, k, v, out, lse, *tensors)
            ctx.cfg = (spec, names, plain)
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        q, k, v, out, lse, *tensors = ctx.saved_tensors
        spec, names, plain = ctx.cfg
        seq = dict(plain, **dict(zip(names, tensors)))
        packed_q, packed_k = seq.get("q_starts") is not None, seq.get("k_starts") is not None
        dq, dk, dv = _outputs(q, packed_q), _outputs(k, packed_k), _outputs(v, packed_k)
        iabn_attention_backward(spec, q, k, v, out, lse, _heads(dout), dq, dk, dv,
                                attention_workspace(spec, q, k, backward=True, **seq), **seq)
        need = ctx.needs_input_grad
        return dq if need[0] else None, dk if need[1] else None, dv if need[2] else None, None, None


def _common(*tensors):
    """The tensors in autocast's type, or in what they promote to."""
    if torch.is_autocast_enabled("cuda"):
        dtype = torch.get_autocast_dtype("cuda")
    else:
        dtype = tensors[0].dtype
        for t in tensors[1:]:
            dtype = torch.promote_types(dtype, t.dtype)
    return [t if t.dtype == dtype else t.to(dtype) for t in tensors]


def attention(q, k, v, causal=False, window=(-1, -1), scale=None, **sequences):
    """softmax(scale q k^T) v over the keys that each query sees.  q [batch, rows, heads,
    head_dim], k, v [batch, rows, kv_heads, head_dim] (heads a multiple of kv_heads); causal and
    window as in AttentionSpec.  sequences: q_lens, k_lens (int32 [batch] on the GPU; rows
    behind a length get zeros), or for packed [rows, heads, head_dim] tensors q_starts,
    k_starts (int32 [batch + 1]) with max_q, max_k; rows in no sequence get zeros."""
    q, k, v = _common(q, k, v)
    return AttentionFunction.apply(q, k, v, AttentionSpec(scale, causal, window), sequences)


class RotaryFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, spec, positions, q, k):
        q, k = _heads(q), None if k is None else _heads(k)
        qo, ko = _fresh(q), None if k is None else _fresh(k)
        iabn_rotary(spec, positions, q, qo, k, ko)
        ctx.save_for_backward(positions)
        ctx.spec = spec
        return qo, ko

    @staticmethod
    @once_differentiable
    def backward(ctx, dq, dk):
        positions, = ctx.saved_tensors
        g, h = _heads(dq), None if dk is None else _heads(dk)
        go, ho = _fresh(g), None if h is None else _fresh(h)
        iabn_rotary(ctx.spec, positions, g, go, h, ho, inverse=True)
        return None, None, go, ho


def rotary(spec: RotarySpec, positions, q, k=None):
    """q (and k) turned by the positions: (q, k), or q alone without k."""
    qo, ko = RotaryFunction.apply(spec, positions, q, k)
    return qo if k is None else (qo, ko)


class QKVAttentionFunction(torch.autograd.Function):
    """The output of attention from a projection qkv [..., heads + 2 kv_heads, head_dim], whose
    queries and keys are first turned where they lie: qkv must be an intermediate that nothing
    else reads or keeps (KeptLinear keeps its input, not its output).  Autograd is told: a leaf is
    refused here, and an operation that kept qkv for its own backward refuses it there.  Keeps
    qkv as turned, the output and the rows' log-sum-exp; the backward writes one gradient for
    the projection, without joining parts."""

    @staticmethod
    def forward(ctx, qkv, positions, heads, kv_heads, turn, spec, seq):
        if turn is not None and qkv.is_leaf and qkv.requires_grad:
            raise RuntimeError("a leaf that requires a gradient would be turned in place: pass a "
                               "copy of it")
        q, k, v = qkv.split((heads, kv_heads, kv_heads), -2)
        if turn is not None:
            iabn_rotary(turn, positions, q, q, k, k)
            torch.autograd.graph.increment_version(qkv)
        out = _outputs(q, seq.get("q_starts") is not None)
        train = ctx.needs_input_grad[0]
        lse = attention_lse(q) if train else None
        iabn_attention_forward(spec, q, k, v, out, lse, attention_workspace(spec, q, k, **seq),
                               **seq)
        if train:
            names, tensors, plain = _kept(seq)
            # detached: its own graph, which the turn does not follow, has no part in the backward
            ctx.save_for_backward(qkv.detach(), positions, out, lse, *tensors)
            ctx.cfg = (heads, kv_heads, turn, spec, names, plain)
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        qkv, positions, out, lse, *tensors = ctx.saved_tensors
        heads, kv_heads, turn, spec, names, plain = ctx.cfg
        seq = dict(plain, **dict(zip(names, tensors)))
        parts = (heads, kv_heads, kv_heads)
        q, k, v = qkv.split(parts, -2)
        grad = _outputs(qkv, seq.get("q_starts") is not None)
        dq, dk, dv = grad.split(parts, -2)
        iabn_attention_backward(spec, q, k, v, out, lse, _heads(dout), dq, dk, dv,
                                attention_workspace(spec, q, k, backward=True, **seq), **seq)
        if turn is not None:
            iabn_rotary(turn, positions, dq, dq, dk, dk, inverse=True)
        return grad, None, None, None, None, None, None


def _projected(layer, turn, *inputs):
    """The layer's output; where it will be turned in place, a copy if a hook may have kept it, or
    a layer of another kind may."""
    t = layer(*inputs)
    if turn is None or type(layer) in (KeptLinear, torch.nn.Linear) and not (
            layer._forward_hooks or torch.nn.modules.module._global_forward_hooks):
        return t
    return t.clone()


class KVCache:
    """Keys and values of up to `capacity` tokens of each of `batch` sequences, and how many
    each holds (lens, int32 on the device).  append writes new tokens behind them without a
    host synchronisation; `used` is the host's upper bound of lens, and what would not fit
    is refused."""

    def __init__(self, batch, capacity, kv_heads, head_dim, dtype=torch.bfloat16, device="cuda"):
        self.k = torch.zeros(batch, capacity, kv_heads, head_dim, dtype=dtype, device=device)
        self.v = torch.zeros_like(self.k)
        self.lens = torch.zeros(batch, dtype=torch.int32, device=device)
        self.used, self.capacity = 0, capacity

    def append(self, k, v, counts=None):
        """k, v [batch, rows, kv_heads, head_dim]; counts: int32 [batch] of the rows that
        count (between 0 and rows; the ones behind are written over by the next append),
        None: all of them.  Cast to the cache's type, and without their graph."""
        B, n = k.shape[:2]
        if k.shape != (self.k.shape[0], n) + self.k.shape[2:] or v.shape != k.shape:
            raise ValueError("k is %s, v %s, expected %s" % (
                tuple(k.shape), tuple(v.shape), (self.k.shape[0], n) + tuple(self.k.shape[2:])))
        if self.used + n > self.capacity:
            raise ValueError("%d tokens behind %d do not fit a cache of %d" % (n, self.used,
                                                                             self.capacity))
        if torch.cuda.is_current_stream_capturing():
            raise RuntimeError("a replayed append would not be counted on the host, and could "
                               "pass the cache's end")
        if n == 0:
            return
        step = torch.arange(n, device=k.device)
        # the device's own lens, held within the bound that was checked
        at = self.lens.long().clamp(0, self.used)[:, None] + step
        b = torch.arange(B, device=k.device)[:, None].expand(B, n)
        self.k.index_put_((b, at), k.detach().to(self.k.dtype))
        self.v.index_put_((b, at), v.detach().to(self.v.dtype))
        self.lens += self._counted(n, counts)
        self.used += n

    def _take_back(self, n, counts=None):
        """Undoes the last append, of n rows with these counts, whose rows are written over by
        the next one."""
        if n > 0:
            self.lens -= self._counted(n, counts)
            self.used -= n

    @staticmethod
    def _counted(n, counts):
        return n if counts is None else counts.to(torch.int32).clamp(0, n)


class ResidualAttention(torch.nn.Module):
    """forward(r, b) -> (r', b'): adds the last block's output b to the residual stream r
    (None: nothing) and makes this block's, b' = out(attention(rotary(qkv(n)))), n = pre(r').
    Takes its place among ResidualMLP blocks; the next ResNorm takes both.

    rotary: a RotarySpec for the queries and keys, or None.  The norm keeps codes in 8
    bits, which the projection's weight gradient reads too; the attention keeps the
    projection, its output and one number a row.

    r, b [batch, rows, cols], or packed [rows, cols] with starts (int32 [batch + 1]) and
    max_len.  positions as iabn_rotary takes them (default: 0, 1, 2, ... on every axis of
    unpacked rows, behind a cache's tokens).  lens: int32 [batch], the rows that count.  cache: a
    KVCache that the rows' keys and values are appended to and which they attend
    (without gradients); a refused call leaves it as it was."""

    def __init__(self, cols, heads, kv_heads=None, head_dim=None, post="rms", pre="rms", alpha=1.0,
                 gate=False, rotary: Optional[RotarySpec] = None, causal=True, window=(-1, -1),
                 scale=None, device=None, dtype=None):
        super().__init__()
        kv_heads = heads if kv_heads is None else kv_heads
        head_dim = cols // heads if head_dim is None else head_dim
        if heads % kv_heads:
            raise ValueError("%d heads are no multiple of %d key heads" % (heads, kv_heads))
        if rotary is not None and rotary.head_dim != head_dim:
            raise ValueError("the rotary spec has heads of %d, the block of %d"
                             % (rotary.head_dim, head_dim))
        self.heads, self.kv_heads, self.head_dim = heads, kv_heads, _head_dim(head_dim)
        self.rotary = rotary
        self.spec = AttentionSpec(scale, causal, window)
        self.norm = ResNorm(cols, post, pre, alpha, gate=gate, device=device)
        self.qkv = KeptLinear(cols, (heads + 2 * kv_heads) * head_dim, bias=False, device=device,
                              dtype=dtype)
        self.out = torch.nn.Linear(heads * head_dim, cols, bias=False, device=device, dtype=dtype)

    def _positions(self, shape, device, cache):
        at = torch.arange(shape[1], dtype=torch.int32, device=device)
        if cache is not None:
            at = cache.lens[:, None] + at
        return at[..., None].expand(*at.shape, self.rotary.axes).contiguous()

    def forward(self, r, b=None, positions=None, lens=None, starts=None, max_len=None,
                cache: Optional[KVCache] = None):
        r, n, kept = self.norm(r, b)
        if n.dim() != (2 if starts is not None else 3):
            raise ValueError("r is %s, expected [batch, rows, cols], or [rows, cols] with starts"
                             % (tuple(r.shape),))
        if self.rotary is not None and positions is None:
            if starts is not None:
                raise ValueError("packed rows need their positions")
            positions = self._positions(n.shape, n.device, cache)
        H, KV, D = self.heads, self.kv_heads, self.head_dim
        qkv = _projected(self.qkv, self.rotary, n, kept).view(*n.shape[:-1], H + 2 * KV, D)
        if cache is not None:
            a = self._cached(qkv, positions, lens, starts, cache)
        else:
            seq = {}
            if starts is not None:
                seq = dict(q_starts=starts, k_starts=starts, max_q=max_len, max_k=max_len)
            elif lens is not None:
                seq = dict(q_lens=lens, k_lens=lens)
            a = QKVAttentionFunction.apply(qkv, positions, H, KV, self.rotary, self.spec, seq)
        return r, self.out(a.flatten(-2))

    def _cached(self, qkv, positions, lens, starts, cache):
        if torch.is_grad_enabled() and qkv.requires_grad:
            raise RuntimeError("a cache keeps no graph: use torch.no_grad()")
        if starts is not None:
            raise ValueError("a cache takes unpacked rows")
        if cache.k.dtype != qkv.dtype:
            raise TypeError("the cache is %s, the block's heads are %s" % (cache.k.dtype, qkv.dtype))
        q, k, v = qkv.split((self.heads, self.kv_heads, self.kv_heads), -2)
        if self.rotary is not None:
            iabn_rotary(self.rotary, positions, q, q, k, k)
        cache.append(k, v, lens)
        try:
            out = _fresh(q)
            keys, values = cache.k[:, :cache.used], cache.v[:, :cache.used]
            seq = dict(k_lens=cache.lens)
            if lens is not None:
                seq["q_lens"] = lens
            iabn_attention_forward(self.spec, q, keys, values, out, None,
                                   attention_workspace(self.spec, q, keys, **seq), **seq)
        except Exception:                          # a refused call leaves the cache as it was
            cache._take_back(q.shape[1], lens)
            raise
        return out


class MapAttention(torch.nn.Module):
    """Attention over the pixels of a feature map [N, C, H, W] (channels last) or a video's
    [N, C, T, H, W]: x + out(attention(rotary(qkv(norm(x))))), norm a GroupNormAct, positions
    the pixels' coordinates, an axis each, with an equal share of every head's pairs.
    rotary=False: none."""

    def __init__(self, channels, heads, groups=32, eps=1e-5, rotary=True, base=100.0, axes=2,
                 device=None, dtype=None):
        super().__init__()
        if channels % heads:
            raise ValueError("%d heads do not divide %d channels" % (heads, channels))
        self.heads, self.axes, D = heads, axes, _head_dim(channels // heads)
        self.norm = GroupNormAct(groups, channels, eps, activation="identity", device=device)
        self.qkv = KeptLinear(channels, 3 * channels, device=device, dtype=dtype)
        self.out = torch.nn.Linear(channels, channels, device=device, dtype=dtype)
        self.spec = AttentionSpec()
        self.rotary = None
        if rotary:
            share = D // 2 // axes
            self.rotary = RotarySpec(D, [share] * axes, base, ramp="axis",
                                     device="cuda" if device is None else device)

    def forward(self, x):
        if x.dim() != 2 + self.axes:
            raise ValueError("x is %s, expected [N, C] and %d extents" % (tuple(x.shape),
                                                                         self.axes))
        rows = self.norm(x).movedim(1, -1).flatten(1, -2)
        positions = None
        if self.rotary is not None:
            grid = [torch.arange(n, dtype=torch.int32, device=x.device) for n in x.shape[2:]]
            positions = torch.stack(torch.meshgrid(*grid, indexing="ij"), -1).flatten(0, -2)
        qkv = _projected(self.qkv, self.rotary, rows)
        qkv = qkv.view(*rows.shape[:-1], 3 * self.heads, qkv.shape[-1] // (3 * self.heads))
        a = QKVAttentionFunction.apply(qkv, positions, self.heads, self.heads, self.rotary,
                                       self.spec, {})
        y = self.out(a.flatten(-2)).unflatten(1, x.shape[2:]).movedim(-1, 1)
        return x + y.to(x.dtype)
