"""PyTorch module of the group norm with an activation, channels last.

`GroupNormAct` takes the place of `GroupNorm` followed by SiLU, GELU, leaky ReLU or
nothing.  Unlike InPlaceABN it does not look at the batch, and it keeps its input for
the backward (these activations do not all have an inverse), but neither the norm's output
nor the activation's.  The arithmetic runs in the library's HIP kernels.
"""
from __future__ import annotations

import math

import torch
from torch.autograd.function import once_differentiable

from . import group_norm_workspace, iabn_group_norm_backward, iabn_group_norm_forward


def _pixels(t):
    """t [samples, pixels, channels] with contiguous channels and rows at one distance that do
    not overlap (a copy only where its strides do not allow it)."""
    N, P, C = t.shape
    if t.numel() == 0:
        return t.contiguous()
    row = t.stride(1) if P > 1 else t.stride(0)
    if t.stride(2) != 1 and C > 1 or N * P > 1 and row < C or \
            N > 1 and P > 1 and t.stride(0) != P * row:
        return t.contiguous()
    return t


class GroupNormActFunction(torch.autograd.Function):
    """y for x [samples, pixels, channels]."""

    @staticmethod
    def forward(ctx, x, weight, bias, groups, eps, activation, act_param):
        x = _pixels(x)
        y = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        train = any(ctx.needs_input_grad)
        stats = torch.empty(x.shape[0], groups, 2, device=x.device) if train else None
        iabn_group_norm_forward(x, y, groups, weight, bias, group_norm_workspace(x, groups),
                                act=activation, act_param=act_param, eps=eps, stats=stats)
        ctx.save_for_backward(x, weight, bias, stats)
        ctx.cfg = (groups, activation, act_param)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, weight, bias, stats = ctx.saved_tensors
        groups, activation, act_param = ctx.cfg
        need = ctx.needs_input_grad
        dy = _pixels(dy)
        dx = torch.empty(x.shape, dtype=x.dtype, device=x.device) if need[0] else None
        dw = torch.empty_like(weight) if need[1] else None
        db = torch.empty_like(bias) if need[2] else None
        iabn_group_norm_backward(x, dy, dx, groups, weight, bias, stats,
                                 group_norm_workspace(x, groups), act=activation,
                                 act_param=act_param, dweight=dw, dbias=db)
        return dx, dw, db, None, None, None, None


class GroupNormAct(torch.nn.Module):
    """GroupNorm(num_groups, num_channels) + activation on [N, C, *] tensors, with the same
    state-dict keys as GroupNorm.  The kernels read channels last: channels_last (and
    channels_last_3d) tensors are taken as they lie, others by a copy, and the output is
    channels last.  activation: "identity", "silu", "gelu", "gelu_tanh" or "leaky_relu"
    (act_param: its slope for negative inputs, 0 for ReLU).  Weight and bias are read in
    float32 (parameters of another type are cast in each call)."""

    def __init__(self, num_groups: int, num_channels: int, eps: float = 1e-5,
                 activation: str = "silu", act_param: float = 0.01, affine: bool = True,
                 device=None):
        super().__init__()
        if num_groups < 1 or num_channels % num_groups:
            raise ValueError("%d groups do not divide %d channels" % (num_groups, num_channels))
        self.num_groups, self.num_channels, self.eps = num_groups, num_channels, eps
        self.activation, self.act_param = activation, act_param
        if affine:
            self.weight = torch.nn.Parameter(torch.ones(num_channels, device=device))
            self.bias = torch.nn.Parameter(torch.zeros(num_channels, device=device))
        else:
            self.register_parameter("weight", None)
            self.register_parameter("bias", None)

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        if x.dim() < 2 or x.shape[1] != self.num_channels:
            raise ValueError("GroupNormAct expects [N, %d, ...], got %s" % (self.num_channels,
                                                                          tuple(x.shape)))
        last = x.movedim(1, -1)
        vec = [None if v is None else v.float() for v in (self.weight, self.bias)]
        rows = last.reshape(x.shape[0], math.prod(x.shape[2:]), x.shape[1])
        y = GroupNormActFunction.apply(rows, *vec, self.num_groups, self.eps, self.activation,
                                       self.act_param)
        return y.view(last.shape).movedim(-1, 1)

    def extra_repr(self) -> str:
        return "%d, %d, eps=%g, activation=%s, act_param=%g, affine=%s" % (
            self.num_groups, self.num_channels, self.eps, self.activation, self.act_param,
            self.weight is not None)
