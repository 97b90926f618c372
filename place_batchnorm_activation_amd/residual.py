"""PyTorch modules of a residual block that keeps its activations in 8 bits.

The memory trade of In-Place ABN for blocks of row norms, linear layers and gated
activations: for its backward pass a block keeps codes (one byte an element, one scale
for 32) instead of tensors.

  ResNorm     r' = r + alpha * gate * post(b), n = pre(r'): the boundary between two
              blocks.  Keeps the codes of both norms' xhat and the rows' statistics.
  KeptLinear  a linear layer on n whose weight gradient reads the same codes of xhat
              that the norm keeps (n = weight * xhat + bias, applied to the product), or
              its own codes of any input.
  GLULinear   the gated activation and the down projection after it: keeps the codes
              of gate and up and rebuilds the projection's input from them.
  ResidualMLP the block of the three.

The norms, the activation and the weight gradient of KeptLinear run in the library's
HIP kernels; the other products are torch's.  Outputs are computed from the tensors
themselves: keeping codes changes gradients only, by the codes' rounding (at most
half a step of 1/127 to 1/64 of the largest of 32 neighbours).
"""
from __future__ import annotations

import math
from typing import NamedTuple, Optional

import torch
from torch.amp import custom_bwd, custom_fwd
from torch.autograd.function import once_differentiable

from . import (ResNormSpec, codes_empty, iabn_codes_pack, iabn_glu_backward, iabn_glu_forward,
               iabn_linear_wgrad, iabn_resnorm_backward, iabn_resnorm_forward,
               linear_wgrad_workspace, resnorm_workspace)


class Kept(NamedTuple):
    """Codes of a layer's input, which is scale * value + shift (None: 1 and 0).  `of`
    says which tensor that is (its address and version): a layer given another one would
    return that input's weight gradient, so it refuses.  None: not checked."""
    codes: torch.Tensor
    exps: torch.Tensor
    scale: Optional[torch.Tensor]
    shift: Optional[torch.Tensor]
    of: Optional[tuple] = None

    def fits(self, x):
        """Whether these are codes of x, or of x's rows in another shape."""
        if self.codes.shape[0] * x.shape[-1] != x.numel():
            return False
        return self.of is None or (x.is_contiguous() and x.data_ptr() == self.of[0] and
                                   x._version == self.of[1])


def _flat(t):
    """t as rows x columns with contiguous columns and rows that do not overlap (a copy only
    where its strides do not allow it); None stays None."""
    if t is None:
        return None
    if t.stride(-1) != 1 and t.shape[-1] > 1 or 0 in t.stride():
        t = t.contiguous()
    t = t.reshape(-1, t.shape[-1])
    return t.contiguous() if t.stride(0) < t.shape[1] else t


def _gate_rows(gate, shape):
    """A gate [..., cols] as [groups, cols], each group a run of consecutive rows of a tensor
    of `shape`.  Leading dimensions past the first must be those of the tensor (ones after
    them): anything else would put its rows in another order than broadcasting does."""
    if gate.dim() < 1 or gate.shape[-1] != shape[-1]:
        raise ValueError("gate is %s, expected [..., %d]" % (tuple(gate.shape), shape[-1]))
    lead, rows = list(gate.shape[:-1]), math.prod(shape[:-1])
    while lead and lead[-1] == 1:
        lead.pop()
    if gate.dim() > 2:
        if len(shape) > 2:
            fits = lead == list(shape[:len(lead)])
        else:
            fits = len(lead) < 2 or math.prod(lead) == rows
        if not fits:
            raise ValueError("gate is %s, which is not a gate for runs of rows of %s"
                             % (tuple(gate.shape), tuple(shape)))
    return gate.reshape(math.prod(lead), shape[-1]).contiguous()


class ResNormFunction(torch.autograd.Function):
    """(r_out, n, codes_n, exps_n); n and the codes are None without a pre-norm, the
    codes with keep="full" and keep=None (no backward will follow) too."""

    @staticmethod
    def forward(ctx, r, b, gate, post_weight, post_bias, pre_weight, pre_bias, post, pre, alpha,
                eps, keep):
        if b is not None and b.shape != r.shape:
            raise ValueError("b is %s, r %s" % (tuple(b.shape), tuple(r.shape)))
        shape, r2, b2 = r.shape, _flat(r), _flat(b)
        T, C = r2.shape
        layer = ResNormSpec(C, post, pre, alpha, eps, post_weight, post_bias, pre_weight, pre_bias)
        train = keep is not None and any(ctx.needs_input_grad)
        has_n, has_b = pre != "none", b is not None
        r_out = torch.empty(T, C, dtype=r.dtype, device=r.device)
        n = torch.empty_like(r_out) if has_n else None
        stats = lambda on: torch.empty(T, 2, device=r.device) if train and on else None  # noqa: E731
        post_stats, pre_stats = stats(has_b and post != "none"), stats(has_n)
        cn = eb = en = cb = None
        if train and keep == "codes":
            if has_b and (post != "none" or gate is not None):
                cb, eb = codes_empty(T, C, r.device)
            if has_n:
                cn, en = codes_empty(T, C, r.device)
        gate2 = None if gate is None else _gate_rows(gate, shape)
        iabn_resnorm_forward(layer, r2, b2, r_out, n, gate2, post_stats, pre_stats, cb, eb, cn, en)
        full = train and keep == "full"
        ctx.save_for_backward(gate2, post_weight, post_bias, pre_weight, pre_bias, post_stats,
                              pre_stats, cb, eb, cn, en, r_out if full and has_n else None,
                              b2 if full and has_b else None)
        ctx.cfg = (post, pre, alpha, eps, shape, has_b, None if gate is None else gate.shape)
        ctx.set_materialize_grads(False)
        for t in (cn, en):
            if t is not None:
                ctx.mark_non_differentiable(t)
        return r_out.view(shape), n.view(shape) if has_n else None, cn, en

    @staticmethod
    @once_differentiable
    def backward(ctx, dr_out, dn, *_):
        if dr_out is None and dn is None:
            return (None,) * 12
        (gate, post_weight, post_bias, pre_weight, pre_bias, post_stats, pre_stats, cb, eb, cn, en,
         r_out, b) = ctx.saved_tensors
        post, pre, alpha, eps, shape, has_b, gate_shape = ctx.cfg
        dr_out, dn = _flat(dr_out), _flat(dn)
        ref = dn if dn is not None else dr_out
        T, C = ref.shape
        need = ctx.needs_input_grad
        layer = ResNormSpec(C, post, pre, alpha, eps, post_weight, post_bias, pre_weight, pre_bias)
        dr = torch.empty_like(ref) if need[0] else None
        branch = has_b and any(need[1:5])
        db = torch.empty_like(ref) if branch else None
        vec = lambda i, on: torch.empty(C, device=ref.device) if need[i] and on else None  # noqa: E731
        dpw, dpb = vec(3, branch), vec(4, branch)
        dnw, dnb = vec(5, pre != "none"), vec(6, pre != "none")
        dgate = torch.empty_like(gate) if need[2] and branch and gate is not None else None
        saved = dict(r_out=r_out, b=b) if cn is None and cb is None else \
            dict(codes_n=cn, exps_n=en, codes_b=cb, exps_b=eb)
        groups = 1 if gate is None else max(1, gate.shape[0])
        ws = resnorm_workspace(T, C, max(1, T // groups), ref.device)
        iabn_resnorm_backward(layer, dr_out, dn, ws, post_stats=post_stats, pre_stats=pre_stats,
                              gate=gate, dr=dr, db=db, dpost_weight=dpw, dpost_bias=dpb,
                              dpre_weight=dnw, dpre_bias=dnb, dgate=dgate, **saved)
        if dgate is not None:
            dgate = dgate.view(gate_shape)
        return (dr.view(shape) if dr is not None else None,
                db.view(shape) if db is not None and need[1] else None, dgate, dpw, dpb, dnw, dnb,
                None, None, None, None, None)


class ResNorm(torch.nn.Module):
    """The boundary between two residual blocks: r' = r + alpha * gate * post(b) and
    n = pre(r') (post and pre: "none", "rms" or "layer"), in r's and b's type or what the two
    promote to.  Norm weights and biases are float32 and read so (a parameter of another type
    is cast in each call), biases with layer norms only.  gate=True learns a vector [cols];
    forward's own gate, [cols] or [groups, cols] for rows / groups consecutive rows each, takes
    its place (of the rows' type, or cast to float32); for rows [b, s, cols] also [b, 1, cols]
    or [b, s, cols].

    forward(r, b=None) -> (r', n, kept): kept is what KeptLinear takes for n, None with
    keep="full" (the backward then reads r' and b themselves), in inference and without a
    pre-norm."""

    def __init__(self, cols, post="none", pre="rms", alpha=1.0, eps=1e-5, gate=False, keep="codes",
                 device=None):
        super().__init__()
        if keep not in ("codes", "full"):
            raise ValueError('keep must be "codes" or "full", got %r' % (keep,))
        ResNormSpec(cols, post, pre, alpha, eps)             # checks the kinds
        self.cols, self.post, self.pre, self.alpha, self.eps = cols, post, pre, alpha, eps
        self.keep = keep
        p = lambda f, on: torch.nn.Parameter(f(cols, device=device)) if on else None  # noqa: E731
        self.post_weight, self.post_bias = p(torch.ones, post != "none"), p(torch.zeros,
                                                                           post == "layer")
        self.pre_weight, self.pre_bias = p(torch.ones, pre != "none"), p(torch.zeros,
                                                                        pre == "layer")
        self.gate = p(torch.ones, gate)

    def forward(self, r, b=None, gate=None):
        # r + b promotes as in torch; the vectors are read in float32 whatever a module-wide
        # .to(dtype) made of them
        if b is not None and b.dtype != r.dtype:
            dtype = torch.promote_types(r.dtype, b.dtype)
            r, b = r.to(dtype), b.to(dtype)
        gate = self.gate if gate is None else gate
        if gate is not None and gate.dtype != r.dtype:
            gate = gate.float()
        vec = [None if v is None else v.float() for v in (self.post_weight, self.post_bias,
                                                          self.pre_weight, self.pre_bias)]
        r_out, n, codes, exps = ResNormFunction.apply(
            r, b, gate, *vec, self.post, self.pre, self.alpha, self.eps,
            self.keep if torch.is_grad_enabled() else None)
        kept = None
        if codes is not None:
            kept = Kept(codes, exps, vec[2].detach(),
                        None if vec[3] is None else vec[3].detach(),
                        (n.data_ptr(), n._version))
        return r_out, n, kept

    def extra_repr(self):
        return "%d, post=%s, pre=%s, alpha=%g, eps=%g, gate=%s, keep=%s" % (
            self.cols, self.post, self.pre, self.alpha, self.eps, self.gate is not None, self.keep)


class KeptLinearFunction(torch.autograd.Function):
    """Under autocast the products run in its type, forward and backward; dw is written in
    the weight's own."""

    @staticmethod
    @custom_fwd(device_type="cuda")
    def forward(ctx, x, weight, bias, codes, exps, scale, shift):
        if ctx.needs_input_grad[1] and codes is None:
            x2 = _flat(x)
            codes, exps = codes_empty(x2.shape[0], x2.shape[1], x.device)
            iabn_codes_pack(x2, codes, exps)
        ctx.save_for_backward(weight, codes, exps, scale, shift)
        ctx.x_shape = x.shape
        return torch.nn.functional.linear(x, weight, bias)

    @staticmethod
    @once_differentiable
    @custom_bwd(device_type="cuda")
    def backward(ctx, dy):
        weight, codes, exps, scale, shift = ctx.saved_tensors
        need = ctx.needs_input_grad
        dy2 = _flat(dy)
        T, (N, K) = dy2.shape[0], weight.shape
        dx = dw = db = None
        if need[0]:
            dx = (dy2 @ weight).view(ctx.x_shape)
        if need[1]:
            dw = torch.empty(N, K, dtype=weight.dtype, device=dy.device)
            db = torch.empty(N, device=dy.device) if need[2] else None
            iabn_linear_wgrad(dy2, codes, exps, dw,
                              linear_wgrad_workspace(T, N, K, dy.dtype, dy.device), scale=scale,
                              shift=shift, dbias=db)
        elif need[2]:
            db = dy2.sum(0, dtype=torch.float32)
        return dx, dw, None if db is None else db.to(weight.dtype), None, None, None, None


class KeptLinear(torch.nn.Linear):
    """A linear layer that keeps its input in 8 bits: its own codes, or those of `kept`
    (ResNorm's third output for this input, which must come as the norm returned it, in any
    shape of the same rows).  An input of another type than the weight is cast to it (as the
    norms of a float32 stream give to 16-bit layers)."""

    def forward(self, x, kept: Optional[Kept] = None):
        codes = (None,) * 4
        if kept is not None and torch.is_grad_enabled():
            if not kept.fits(x):
                raise ValueError("kept (of %d rows) was made for another tensor than this input "
                                 "%s; without it the layer keeps its own codes"
                                 % (kept.codes.shape[0], tuple(x.shape)))
            codes = kept[:4]
        if x.dtype != self.weight.dtype and not torch.is_autocast_enabled("cuda"):
            x = x.to(self.weight.dtype)
        if not torch.is_grad_enabled():
            return super().forward(x)
        return KeptLinearFunction.apply(x, self.weight, self.bias, *codes)


class GLULinearFunction(torch.autograd.Function):
    @staticmethod
    @custom_fwd(device_type="cuda")
    def forward(ctx, h, weight, bias, act, train):
        h2 = _flat(h)
        T, F = h2.shape[0], weight.shape[1]
        if h2.shape[1] != 2 * F:
            raise ValueError("the input has %d columns, expected %d (gate and up halves of %d)"
                             % (h2.shape[1], 2 * F, F))
        a = torch.empty(T, F, dtype=h.dtype, device=h.device)
        codes = [None] * 4
        if train and any(ctx.needs_input_grad):
            codes = [*codes_empty(T, F, h.device), *codes_empty(T, F, h.device)]
        iabn_glu_forward(h2[:, :F], h2[:, F:], a, act, *codes)
        ctx.save_for_backward(weight, *codes)
        ctx.act, ctx.shape = act, h.shape
        return torch.nn.functional.linear(a, weight, bias).view(*h.shape[:-1], weight.shape[0])

    @staticmethod
    @once_differentiable
    @custom_bwd(device_type="cuda")
    def backward(ctx, dy):
        weight, cg, eg, cu, eu = ctx.saved_tensors
        need = ctx.needs_input_grad
        dy2 = _flat(dy)
        F = weight.shape[1]
        da = dy2 @ weight
        dh = torch.empty(dy2.shape[0], 2 * F, dtype=dy.dtype, device=dy.device)
        # the projection's input, rebuilt over the gradient that the kernel has read
        a = da if need[1] else None
        iabn_glu_backward(cg, eg, cu, eu, da, dh[:, :F], dh[:, F:], ctx.act, out=a)
        dw = dy2.t() @ a if need[1] else None
        db = dy2.sum(0, dtype=torch.float32).to(weight.dtype) if need[2] else None
        return dh.view(ctx.shape) if need[0] else None, dw, db, None, None


class GLULinear(torch.nn.Linear):
    """The down projection of a gated unit, with the activation before it: input
    [..., 2 * in_features], gate and up halves; act "silu", "gelu" or "gelu_tanh"."""

    def __init__(self, in_features, out_features, bias=True, act="silu", device=None, dtype=None):
        super().__init__(in_features, out_features, bias, device, dtype)
        self.act = act

    def forward(self, h):
        return GLULinearFunction.apply(h, self.weight, self.bias, self.act,
                                       torch.is_grad_enabled())


class ResidualMLP(torch.nn.Module):
    """forward(r, b) -> (r', b'): adds the last block's output b to the residual stream r
    (None: nothing) and makes this block's, b' = down(act(gate(n)) * up(n)), n = pre(r').
    The next ResNorm takes both.  hidden: the width of the gated unit."""

    def __init__(self, cols, hidden, post="rms", pre="rms", alpha=1.0, gate=False, act="silu",
                 device=None, dtype=None):
        super().__init__()
        self.norm = ResNorm(cols, post, pre, alpha, gate=gate, device=device)
        self.up = KeptLinear(cols, 2 * hidden, bias=False, device=device, dtype=dtype)
        self.down = GLULinear(hidden, cols, bias=False, act=act, device=device, dtype=dtype)

    def forward(self, r, b=None):
        r, n, kept = self.norm(r, b)
        return r, self.down(self.up(n, kept))
