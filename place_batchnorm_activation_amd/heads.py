"""Binding of attention, rotary positions and group norm of include/iabn.h.

Attention and rotary positions take tensors of heads [batch, rows, heads, head_dim] (or packed
[rows, heads, head_dim]) with contiguous head elements and any other strides, so slices
of a wider projection and transposed views are taken without a copy.  The group norm
takes rows x channels as the other operators of blocks do (block.py).  Shapes, types and
devices are checked here, since the library sees only addresses; everything is computed
in the library's HIP kernels.
"""
from __future__ import annotations

import ctypes
import math
import struct

import torch

from . import _check, _dtype_code, _F, _I64, _INT, _P, _SZ, lib
from .block import _cols, _flat, _name, _rows, _space, _stream

GN_ACTS = {"silu": 0, "gelu": 1, "gelu_tanh": 2, "identity": 3, "leaky_relu": 4}
_POS_TYPES = {torch.int32: 0, torch.int64: 1, torch.float32: 2}


# iabn_heads: address and three strides, passed as the bytes of the struct
_HEADS = struct.Struct("=4q").pack


class _Problem(ctypes.Structure):
    _fields_ = [("batch", _I64), ("heads", _I64), ("kv_heads", _I64), ("head_dim", _I64),
                ("q_len", _I64), ("k_len", _I64), ("dtype", _INT), ("scale", _F),
                ("left", _I64), ("right", _I64), ("q_starts", _P), ("k_starts", _P),
                ("q_rows", _I64), ("k_rows", _I64), ("q_lens", _P), ("k_lens", _P)]


class _Rotary(ctypes.Structure):
    _fields_ = [("batch", _I64), ("rows", _I64), ("head_dim", _I64), ("pairs", _I64),
                ("axes", _I64), ("dtype", _INT), ("interleaved", _INT), ("inv_freq", _P),
                ("axis", _P), ("positions", _P), ("pos_type", _INT), ("pos_batch", _I64),
                ("pos_row", _I64)]


class _GroupNorm(ctypes.Structure):
    _fields_ = [("n", _I64), ("hw", _I64), ("c", _I64), ("groups", _I64), ("dtype", _INT),
                ("weight", _P), ("bias", _P), ("act", _INT), ("act_param", _F), ("eps", _F)]


lib.iabn_attention_workspace_size.argtypes = [_P, _INT]
lib.iabn_attention_workspace_size.restype = _SZ
lib.iabn_attention_forward.argtypes = [_P] * 7 + [_SZ, _P]
lib.iabn_attention_backward.argtypes = [_P] * 11 + [_SZ, _P]
lib.iabn_rotary.argtypes = [_P, _P, _I64, _P, _P, _I64, _P, _INT, _P]
lib.iabn_group_norm_workspace_size.argtypes = [_P]
lib.iabn_group_norm_workspace_size.restype = _SZ
lib.iabn_group_norm_forward.argtypes = [_P] + [_P, _I64] * 2 + [_P, _P, _SZ, _P]
lib.iabn_group_norm_backward.argtypes = [_P] + [_P, _I64] * 3 + [_P] * 4 + [_SZ, _P]
for _fn in ("iabn_attention_forward", "iabn_attention_backward", "iabn_rotary",
            "iabn_group_norm_forward", "iabn_group_norm_backward"):
    getattr(lib, _fn).restype = _INT


# ---------------------------------------------------------------------------
# tensors of heads

def _heads(t, name, shape, dtype=None, device=None):
    """t as the library takes it; shape is what it must be, dtype and device (an index) too
    where given."""
    if t.shape != shape:
        raise ValueError("%s is %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    if dtype is not None and (t.dtype != dtype or t.get_device() != device):
        raise TypeError("%s is %s on %s, expected %s on %s" % (
            name, t.dtype, t.device, dtype, "cpu" if device < 0 else "cuda:%d" % device))
    st = t.stride()
    if st[-1] != 1 and shape[-1] > 1 and t.numel() > 0:
        raise ValueError("%s: a head's elements must be contiguous" % name)
    if len(st) == 4:
        return _HEADS(t.data_ptr(), st[0], st[1], st[2])
    return _HEADS(t.data_ptr(), 0, st[0], st[1])


def _counts(t, name, n, ref):
    return None if t is None else _flat(t, name, n, torch.int32, ref.get_device())


class AttentionSpec:
    """What an attention computes: the factor of its scores (None: 1 / sqrt(head_dim)) and
    which keys a query sees: window = (left, right) keys to either side of its own place
    (negative: unbounded), causal the same as right = 0.  The last query stands at the last
    key."""

    __slots__ = ("scale", "left", "right")

    def __init__(self, scale=None, causal=False, window=(-1, -1)):
        left, right = (int(w) for w in window)
        if causal and right > 0:
            raise ValueError("causal, and a window of %d keys ahead" % right)
        self.scale = scale
        self.left, self.right = left, 0 if causal else right

    def _problem(self, q, k, q_starts, k_starts, q_lens, k_lens, max_q, max_k):
        """The problem that q [batch, rows, heads, head_dim] (packed, with starts: no batch) and
        k make."""
        if q.dim() != (3 if q_starts is not None else 4):
            raise ValueError("q is %s, expected %s" % (tuple(q.shape), "[rows, heads, head_dim] "
                             "with q_starts" if q_starts is not None else
                             "[batch, rows, heads, head_dim]"))
        if k.dim() != (3 if k_starts is not None else 4):
            raise ValueError("k is %s, expected %s" % (tuple(k.shape), "[rows, heads, head_dim] "
                             "with k_starts" if k_starts is not None else
                             "[batch, rows, heads, head_dim]"))
        qs, ks = q.shape, k.shape
        H, D, KV = qs[-2], qs[-1], ks[-2]
        batch = qs[0] if q_starts is None else ks[0] if k_starts is None else \
            q_starts.numel() - 1
        if k_starts is None and ks[0] != batch:
            raise ValueError("q has %d sequences, k %d" % (batch, ks[0]))
        if H and (KV == 0 or H % KV):
            raise ValueError("%d query heads are no multiple of %d key heads" % (H, KV))
        for starts, most, side in ((q_starts, max_q, "q"), (k_starts, max_k, "k")):
            if starts is not None and most is None:
                raise ValueError("packed %s needs max_%s, the most rows of a sequence"
                                 % (side, side))
        scale = 1.0 / math.sqrt(max(1, D)) if self.scale is None else self.scale
        return _Problem(
            batch, H, KV, D, qs[1] if q_starts is None else max_q,
            ks[1] if k_starts is None else max_k, _dtype_code(q), scale, self.left,
            self.right, _counts(q_starts, "q_starts", batch + 1, q),
            _counts(k_starts, "k_starts", batch + 1, q), qs[0], ks[0],
            _counts(q_lens, "q_lens", batch, q), _counts(k_lens, "k_lens", batch, q))


def attention_lse(q):
    """Uninitialised log-sum-exp of queries q: fp32 [batch, heads, rows], packed [heads,
    rows]."""
    *batch, rows, heads, _ = q.shape
    return torch.empty(*batch, heads, rows, dtype=torch.float32, device=q.device)


def iabn_attention_workspace_size(spec, q, k, backward=False, q_starts=None, k_starts=None,
                                  q_lens=None, k_lens=None, max_q=None, max_k=None) -> int:
    p = spec._problem(q, k, q_starts, k_starts, q_lens, k_lens, max_q, max_k)
    return lib.iabn_attention_workspace_size(ctypes.byref(p), int(bool(backward)))


def attention_workspace(spec, q, k, backward=False, **sequences):
    """A workspace tensor for iabn_attention_forward (or _backward) of these queries and
    keys; None where it needs none."""
    size = iabn_attention_workspace_size(spec, q, k, backward, **sequences)
    return torch.empty(size, dtype=torch.uint8, device=q.device) if size else None


def _lse(lse, q):
    if lse is None:
        return None
    return _flat(lse, "lse", q.numel() // max(1, q.shape[-1]), torch.float32, q.get_device())


def iabn_attention_forward(spec, q, k, v, out, lse=None, workspace=None, q_starts=None,
                           k_starts=None, q_lens=None, k_lens=None, max_q=None, max_k=None,
                           stream=None):
    """out = softmax(scale q k^T) v over the keys that each query sees, and lse
    (attention_lse) for the backward.  q, out [batch, rows, heads, head_dim], k, v
    [batch, rows, kv_heads, head_dim]; q_lens, k_lens: int32 [batch] lengths on the GPU.
    Packed: [rows, heads, head_dim] with q_starts (k_starts) int32 [batch + 1] on the GPU
    and max_q (max_k), the most rows of a sequence."""
    p = spec._problem(q, k, q_starts, k_starts, q_lens, k_lens, max_q, max_k)
    qs, ks, on = q.shape, k.shape, (q.dtype, q.get_device())
    at = (_heads(q, "q", qs), _heads(k, "k", ks, *on), _heads(v, "v", ks, *on),
          _heads(out, "out", qs, *on))
    lp = _lse(lse, q)
    ws, wb = _space(workspace, q)
    s = _stream(stream, q)
    _check("iabn_attention_forward", lib.iabn_attention_forward(ctypes.byref(p), *at, lp, ws, wb,
                                                                s))


def iabn_attention_backward(spec, q, k, v, out, lse, dout, dq, dk, dv, workspace, q_starts=None,
                            k_starts=None, q_lens=None, k_lens=None, max_q=None, max_k=None,
                            stream=None):
    """dq, dk and dv from dout and the forward's out and lse; workspace:
    attention_workspace(..., backward=True)."""
    p = spec._problem(q, k, q_starts, k_starts, q_lens, k_lens, max_q, max_k)
    qs, ks, on = q.shape, k.shape, (q.dtype, q.get_device())
    at = (_heads(q, "q", qs), _heads(k, "k", ks, *on), _heads(v, "v", ks, *on),
          _heads(out, "out", qs, *on), _heads(dout, "dout", qs, *on), _heads(dq, "dq", qs, *on),
          _heads(dk, "dk", ks, *on), _heads(dv, "dv", ks, *on))
    if lse is None:
        raise ValueError("the backward needs the forward's lse")
    lp = _lse(lse, q)
    ws, wb = _space(workspace, q)
    s = _stream(stream, q)
    _check("iabn_attention_backward", lib.iabn_attention_backward(
        ctypes.byref(p), *at[:4], lp, *at[4:], ws, wb, s))


# ---------------------------------------------------------------------------
# rotary positions

class RotarySpec:
    """How positions turn the heads.  sections: pairs of each axis (time, height, width; one
    axis by default, all of head_dim turning), in runs one after another, or with
    mixed=True dealt out in turn.  The frequency of a pair is base ** (-i / n), i counted over
    all n pairs, or with ramp="axis" over its own axis's.  inv_freq (float64) and axis
    (int32), tensors of a value for each pair, replace all of that where given, with `axes`
    coordinates a position.  interleaved: pairs (2p, 2p + 1) instead of halves."""

    __slots__ = ("head_dim", "axes", "interleaved", "inv_freq", "axis")

    def __init__(self, head_dim, sections=None, base=10000.0, ramp="shared", mixed=False,
                 interleaved=False, inv_freq=None, axis=None, axes=1, device="cuda"):
        if inv_freq is None:
            sections = [head_dim // 2] if sections is None else [int(n) for n in sections]
            if not sections or min(sections) < 0 or sum(sections) < 1:
                raise ValueError("sections %s hold no pairs" % (sections,))
            if ramp not in ("shared", "axis"):
                raise ValueError('ramp must be "shared" or "axis", got %r' % (ramp,))
            axes, pairs = len(sections), sum(sections)
            if mixed:
                left, order = list(sections), []
                while len(order) < pairs:
                    for a in range(axes):
                        if left[a]:
                            left[a] -= 1
                            order.append(a)
            else:
                order = [a for a, n in enumerate(sections) for _ in range(n)]
            seen, power = [0] * axes, []
            for p, a in enumerate(order):
                power.append(seen[a] / sections[a] if ramp == "axis" else p / pairs)
                seen[a] += 1
            inv_freq = torch.tensor([float(base) ** -e for e in power], dtype=torch.float64,
                                    device=device)
            axis = torch.tensor(order, dtype=torch.int32, device=device) if axes > 1 else None
        if inv_freq.dim() != 1 or not 1 <= inv_freq.numel() <= head_dim // 2:
            raise ValueError("inv_freq is %s, expected up to %d pairs" % (tuple(inv_freq.shape),
                                                                        head_dim // 2))
        self.head_dim, self.axes, self.interleaved = head_dim, axes, bool(interleaved)
        self.inv_freq, self.axis = inv_freq, axis

    @property
    def pairs(self):
        return self.inv_freq.numel()


def iabn_rotary(spec, positions, q, q_out, k=None, k_out=None, inverse=False, stream=None):
    """q_out = q turned by the positions (k_out = k likewise, where given); inverse: by the
    negative angles, which is the gradient.  q [batch, rows, heads, head_dim] or packed
    [rows, heads, head_dim]; positions int32, int64 or float32 [rows] or [batch, rows] for
    one axis, [rows, axes] or [batch, rows, axes] else (packed: [rows], [rows, axes]).  An
    output may be exactly its input."""
    if q.dim() not in (3, 4):
        raise ValueError("q is %s, expected [batch, rows, heads, head_dim]" % (tuple(q.shape),))
    packed = q.dim() == 3
    qs, dtype, dev = q.shape, q.dtype, q.get_device()
    lead, D = tuple(qs[:-2]), qs[-1]
    if D != spec.head_dim:
        raise ValueError("the spec has heads of %d, q of %d" % (spec.head_dim, D))
    B, S = (1, lead[0]) if packed else lead
    axes = spec.axes
    shape, stride = tuple(positions.shape), positions.stride()
    if shape == lead + (axes,) or shape == (S, axes):
        if axes > 1 and positions.numel() and stride[-1] != 1:
            raise ValueError("a position's coordinates must be contiguous")
        stride = stride[:-1]
    elif axes > 1 or shape not in (lead, (S,)):
        raise ValueError("positions are %s, expected %s" % (shape, lead + (axes,)))
    if positions.dtype not in _POS_TYPES:
        raise TypeError("positions are int32, int64 or float32, got %s" % positions.dtype)
    if positions.get_device() != dev:
        raise TypeError("positions are on %s, q on %s" % (positions.device, q.device))
    pos_batch, pos_row = stride if len(stride) == 2 else (0, stride[0])
    n = spec.inv_freq.numel()
    r = _Rotary(B, S, D, n, axes, _dtype_code(q), int(spec.interleaved),
                _flat(spec.inv_freq, "inv_freq", n, torch.float64, dev),
                _flat(spec.axis, "axis", n, torch.int32, dev), positions.data_ptr(),
                _POS_TYPES[positions.dtype], pos_batch, pos_row)
    qp, qo = _heads(q, "q", qs), _heads(q_out, "q_out", qs, dtype, dev)
    KV, kp, ko = 0, None, None
    if (k is None) != (k_out is None):
        raise ValueError("k and k_out go together")
    if k is not None:
        KV = k.shape[-2] if k.dim() == q.dim() else -1
        k_shape = lead + (KV, D)
        kp = _heads(k, "k", k_shape, dtype, dev)
        ko = _heads(k_out, "k_out", k_shape, dtype, dev)
    s = _stream(stream, q)
    _check("iabn_rotary", lib.iabn_rotary(ctypes.byref(r), qp, qs[-2], qo, kp, KV, ko,
                                          int(bool(inverse)), s))


# ---------------------------------------------------------------------------
# group norm

def _group_norm(x, groups, weight, bias, act, act_param, eps):
    """(layer, (address, ld) of x) of a tensor [samples, ..., channels]."""
    if x.dim() < 2:
        raise ValueError("x is %s, expected [samples, ..., channels]" % (tuple(x.shape),))
    p, ld = _map(x, "x")
    N, C, dev = x.shape[0], x.shape[-1], x.get_device()
    if groups < 1 or C % groups:
        raise ValueError("%d groups do not divide %d channels" % (groups, C))
    return _GroupNorm(N, math.prod(x.shape[1:-1]), C, groups, _dtype_code(x),
                      _cols(weight, "weight", C, dev), _cols(bias, "bias", C, dev),
                      _name(act, GN_ACTS, "act"), act_param, eps), (p, ld)


def _map(t, name):
    """(address, ld) of a tensor as rows of channels."""
    return (t.data_ptr(), t.shape[-1]) if t.is_contiguous() else _rows(t, name)[:2]


def _of(t, name, x):
    """(address, ld) of a tensor shaped as x, of its type and device."""
    if t is None:
        return None, 0
    if t.shape != x.shape:
        raise ValueError("%s is %s, expected %s" % (name, tuple(t.shape), tuple(x.shape)))
    if t.dtype != x.dtype or t.get_device() != x.get_device():
        raise TypeError("%s is %s on %s, expected %s on %s" % (name, t.dtype, t.device, x.dtype,
                                                              x.device))
    return _map(t, name)


def _gn_stats(stats, x, groups):
    return None if stats is None else _flat(stats, "stats", 2 * x.shape[0] * groups,
                                            torch.float32, x.get_device())


def iabn_group_norm_workspace_size(x, groups) -> int:
    layer, _ = _group_norm(x, groups, None, None, "identity", 0.0, 0.0)
    return lib.iabn_group_norm_workspace_size(ctypes.byref(layer))


def group_norm_workspace(x, groups):
    """A workspace tensor for both passes over tensors shaped as x."""
    return torch.empty(iabn_group_norm_workspace_size(x, groups), dtype=torch.uint8,
                       device=x.device)


def iabn_group_norm_forward(x, y, groups, weight, bias, workspace, act="identity", act_param=0.01,
                            eps=1e-5, stats=None, stream=None):
    """y = act(group norm of x) for x [samples, ..., channels]; weight and bias fp32
    [channels] or None; stats fp32 [samples, groups, 2] for the backward, or None.  y may be
    exactly x."""
    layer, (p, ld) = _group_norm(x, groups, weight, bias, act, act_param, eps)
    yp, ldy = _of(y, "y", x)
    st = _gn_stats(stats, x, groups)
    ws, wb = _space(workspace, x)
    s = _stream(stream, x)
    _check("iabn_group_norm_forward", lib.iabn_group_norm_forward(
        ctypes.byref(layer), p, ld, yp, ldy, st, ws, wb, s))


def iabn_group_norm_backward(x, dy, dx, groups, weight, bias, stats, workspace, act="identity",
                             act_param=0.01, dweight=None, dbias=None, stream=None):
    """dx, dweight and dbias (each may be None) from x, dy and the forward's stats."""
    layer, (p, ld) = _group_norm(x, groups, weight, bias, act, act_param, 0.0)
    C, dev = x.shape[-1], x.get_device()
    gp, ldg = _of(dy, "dy", x)
    dp, ldd = _of(dx, "dx", x)
    st, dwp, dbp = (_gn_stats(stats, x, groups), _cols(dweight, "dweight", C, dev),
                    _cols(dbias, "dbias", C, dev))
    ws, wb = _space(workspace, x)
    s = _stream(stream, x)
    _check("iabn_group_norm_backward", lib.iabn_group_norm_backward(
        ctypes.byref(layer), p, ld, gp, ldg, dp, ldd, st, dwp, dbp, ws, wb, s))
