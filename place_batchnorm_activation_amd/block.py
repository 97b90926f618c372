"""Binding of the residual-block operators of include/iabn.h.

Every function calls the entry point of the same name on tensors it takes as rows
x cols: the last dimension is the columns (contiguous), the leading ones collapse
to rows at one distance, so slices of a wider buffer are taken without a copy.
Shapes, types and devices are checked here, since the library sees only
addresses; everything is computed in the library's HIP kernels.
"""
from __future__ import annotations

import ctypes

import torch

from . import (_check, _dtype_arg, _dtype_code, _F, _I64, _INT, _P, _SZ, lib)
from . import _stream as _any_stream

GROUP = 32
GLU_ACTS = {"silu": 0, "gelu": 1, "gelu_tanh": 2}
NORMS = {"none": 0, "rms": 1, "layer": 2}
MAX_RESNORM_COLS = 16384

_R = [_P, _I64]
lib.iabn_codes_pack.argtypes = _R + [_I64, _I64, _INT, _P, _P, _P]
lib.iabn_codes_unpack.argtypes = [_P, _P, _I64, _I64, _P, _P] + _R + [_INT, _P]
lib.iabn_glu_forward.argtypes = _R * 3 + [_I64, _I64, _INT, _INT, _P, _P, _P, _P, _P]
lib.iabn_glu_backward.argtypes = [_P, _P, _P, _P] + _R * 4 + [_I64, _I64, _INT, _INT, _P]
lib.iabn_linear_wgrad_workspace_size.argtypes = [_I64, _I64, _I64, _INT]
lib.iabn_linear_wgrad_workspace_size.restype = _SZ
lib.iabn_linear_wgrad.argtypes = _R + [_INT, _P, _P, _P, _P] + _R + [_INT, _P, _INT, _I64, _I64,
                                                                    _I64, _P, _SZ, _P]
lib.iabn_resnorm_forward.argtypes = [_P] + _R * 4 + [_P] * 7
lib.iabn_resnorm_workspace_size.argtypes = [_I64, _I64, _I64]
lib.iabn_resnorm_workspace_size.restype = _SZ
lib.iabn_resnorm_backward.argtypes = [_P] + _R * 4 + [_P] * 6 + _R * 2 + [_P] * 6 + [_SZ, _P]
for _fn in ("iabn_codes_pack", "iabn_codes_unpack", "iabn_glu_forward", "iabn_glu_backward",
            "iabn_linear_wgrad", "iabn_resnorm_forward", "iabn_resnorm_backward"):
    getattr(lib, _fn).restype = _INT


# ---------------------------------------------------------------------------
# tensors as rows

def _rows(t, name):
    """(address, ld, rows, cols) of a tensor [..., cols]."""
    shape = t.shape
    if len(shape) == 2:
        T, C = shape
        ld, cs = t.stride()
        if cs != 1 and C > 1 and T > 0:          # of no rows, any strides will do
            raise ValueError("%s: the last dimension must be contiguous" % name)
        if T <= 1:
            ld = C
        elif ld < C:
            raise ValueError("%s: rows overlap (stride %d, %d columns)" % (name, ld, C))
        return t.data_ptr(), ld, T, C
    if len(shape) == 1:
        return _rows(t[None], name)
    if len(shape) == 0:
        raise ValueError("%s: a tensor [..., cols] is needed" % name)
    try:
        return _rows(t.view(-1, shape[-1]), name)
    except RuntimeError:
        raise ValueError("%s: its leading dimensions do not collapse to rows at one distance"
                         % name) from None


def _like(t, name, T, C, ref):
    """(address, ld) of an optional tensor of T x C of ref's type and device."""
    if t is None:
        return None, 0
    p, ld, t_rows, t_cols = _rows(t, name)
    if t_rows != T or t_cols != C:
        raise ValueError("%s is %d x %d, expected %d x %d" % (name, t_rows, t_cols, T, C))
    if t.dtype != ref.dtype or t.get_device() != ref.get_device():
        raise TypeError("%s is %s on %s, expected %s on %s" % (name, t.dtype, t.device, ref.dtype,
                                                              ref.device))
    return p, ld


def _flat(t, name, numel, dtype, device):
    """Address of an optional contiguous tensor of numel elements on GPU `device` (-1:
    the host)."""
    if t is None:
        return None
    if t.dtype != dtype or t.get_device() != device:
        raise TypeError("%s is %s on %s, expected %s on GPU %d" % (name, t.dtype, t.device, dtype,
                                                                  device))
    if t.numel() != numel or not t.is_contiguous():
        raise ValueError("%s: %d contiguous elements are needed, got %s" % (name, numel,
                                                                          tuple(t.shape)))
    return t.data_ptr()


def _cols(t, name, C, device):
    return None if t is None else _flat(t, name, C, torch.float32, device)


def code_cols(cols: int) -> int:
    """Columns of the codes of a tensor of `cols` columns: whole groups of 32."""
    return (cols + GROUP - 1) // GROUP * GROUP


def codes_empty(rows: int, cols: int, device="cuda"):
    """Uninitialised (codes, exps) for a tensor of rows x cols."""
    p = code_cols(cols)
    return (torch.empty(rows, p, dtype=torch.int8, device=device),
            torch.empty(rows, p // GROUP, dtype=torch.uint8, device=device))


def _codes(codes, exps, name, T, C, device):
    if codes is None and exps is None:
        return None, None
    if codes is None or exps is None:
        raise ValueError("codes and exps of %s go together" % name)
    p = code_cols(C)
    return (_flat(codes, "codes of " + name, T * p, torch.int8, device),
            _flat(exps, "exps of " + name, T * p // GROUP, torch.uint8, device))


def _name(v, table, what):
    if isinstance(v, str):
        if v not in table:
            raise ValueError("%s must be one of %s, got %r" % (what, sorted(table), v))
        return table[v]
    return int(v)


# the current stream as an integer, without torch's wrapper object (3 us a call) where this
# torch has the accessor that its own compiler uses
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _stream(stream, t):
    """The stream to launch on: the given one, or the current one of t's GPU.  The library
    reads addresses on the GPU, where a host tensor's would fault."""
    device = t.get_device()
    if device < 0:
        raise TypeError("the library's tensors live on the GPU, got %s" % t.device)
    if device != _current_device():
        raise ValueError("the tensors are on GPU %d, the current one is %d (torch.cuda.device)"
                         % (device, _current_device()))
    if stream is None:
        return _raw_stream(device) if _raw_stream else \
            torch.cuda.current_stream(device).cuda_stream
    return _any_stream(stream)


def _space(workspace, ref):
    """(address, bytes) of an optional workspace on ref's GPU."""
    if workspace is None:
        return None, 0
    if workspace.get_device() != ref.get_device() or not workspace.is_contiguous():
        raise ValueError("workspace: a contiguous tensor on %s is needed" % ref.device)
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


# ---------------------------------------------------------------------------
# codes

def iabn_codes_pack(x, codes, exps, stream=None):
    p, ld, T, C = _rows(x, "x")
    cp, ep = _codes(codes, exps, "x", T, C, x.get_device())
    s = _stream(stream, x)
    _check("iabn_codes_pack", lib.iabn_codes_pack(p, ld, T, C, _dtype_code(x), cp, ep,
                                                  s))


def iabn_codes_unpack(codes, exps, y, scale=None, shift=None, stream=None):
    """y = scale * value + shift (fp32 vectors of y's columns, or None)."""
    p, ld, T, C = _rows(y, "y")
    cp, ep = _codes(codes, exps, "y", T, C, y.get_device())
    s = _stream(stream, y)
    _check("iabn_codes_unpack", lib.iabn_codes_unpack(
        cp, ep, T, C, _cols(scale, "scale", C, y.get_device()), _cols(shift, "shift", C, y.get_device()), p,
        ld, _dtype_code(y), s))


# ---------------------------------------------------------------------------
# gated activation

def iabn_glu_forward(gate, up, out, act, codes_gate=None, exps_gate=None, codes_up=None,
                     exps_up=None, stream=None):
    """out = act(gate) * up (up None: act(gate)), and the inputs' codes where given."""
    gp, ldg, T, F = _rows(gate, "gate")
    up_p, ldu = _like(up, "up", T, F, gate)
    op, ldo = _like(out, "out", T, F, gate)
    cg, eg = _codes(codes_gate, exps_gate, "gate", T, F, gate.get_device())
    cu, eu = _codes(codes_up, exps_up, "up", T, F, gate.get_device())
    s = _stream(stream, gate)
    _check("iabn_glu_forward", lib.iabn_glu_forward(
        gp, ldg, up_p, ldu, op, ldo, T, F, _dtype_code(gate), _name(act, GLU_ACTS, "act"), cg,
        eg, cu, eu, s))


def iabn_glu_backward(codes_gate, exps_gate, codes_up, exps_up, dout, dgate, dup, act, out=None,
                      stream=None):
    """dgate and dup (None without codes_up) from the codes and dout; `out`, where
    given, receives act(gate) * up rebuilt from the codes."""
    dp, ldd, T, F = _rows(dout, "dout")
    gp, ldg = _like(dgate, "dgate", T, F, dout)
    up_p, ldu = _like(dup, "dup", T, F, dout)
    op, ldo = _like(out, "out", T, F, dout)
    cg, eg = _codes(codes_gate, exps_gate, "gate", T, F, dout.get_device())
    cu, eu = _codes(codes_up, exps_up, "up", T, F, dout.get_device())
    s = _stream(stream, dout)
    _check("iabn_glu_backward", lib.iabn_glu_backward(
        cg, eg, cu, eu, dp, ldd, gp, ldg, up_p, ldu, op, ldo, T, F, _dtype_code(dout),
        _name(act, GLU_ACTS, "act"), s))


# ---------------------------------------------------------------------------
# weight gradient

def iabn_linear_wgrad_workspace_size(rows, n, k, dtype) -> int:
    return lib.iabn_linear_wgrad_workspace_size(rows, n, k, _dtype_arg(dtype))


def linear_wgrad_workspace(rows, n, k, dtype, device="cuda"):
    """A workspace tensor for iabn_linear_wgrad; None where it needs none."""
    size = iabn_linear_wgrad_workspace_size(rows, n, k, dtype)
    return torch.empty(size, dtype=torch.uint8, device=device) if size else None


def iabn_linear_wgrad(dy, codes, exps, dw, workspace=None, scale=None, shift=None, dbias=None,
                      accumulate=False, stream=None):
    """dw [n, k] = dy^T (scale * x + shift) and dbias = the sum of dy's rows, x the
    tensor [rows, k] that the codes hold."""
    dp, ldd, T, N = _rows(dy, "dy")
    wp, ldw, n, K = _rows(dw, "dw")
    if n != N or dw.device != dy.device:
        raise ValueError("dw has %d rows on %s, expected %d on %s" % (n, dw.device, N, dy.get_device()))
    cp, ep = _codes(codes, exps, "x", T, K, dy.get_device())
    ws, wb = _space(workspace, dy)
    s = _stream(stream, dy)
    _check("iabn_linear_wgrad", lib.iabn_linear_wgrad(
        dp, ldd, _dtype_code(dy), cp, ep, _cols(scale, "scale", K, dy.get_device()),
        _cols(shift, "shift", K, dy.get_device()), wp, ldw, _dtype_code(dw),
        _cols(dbias, "dbias", N, dy.get_device()), int(bool(accumulate)), T, N, K, ws, wb,
        s))


# ---------------------------------------------------------------------------
# residual norms

class _Layer(ctypes.Structure):
    _fields_ = [("rows", _I64), ("cols", _I64), ("dtype", _INT), ("post", _INT), ("pre", _INT),
                ("post_weight", _P), ("post_bias", _P), ("pre_weight", _P), ("pre_bias", _P),
                ("alpha", _F), ("eps", _F), ("gate", _P), ("gate_dtype", _INT),
                ("rows_per_gate", _I64)]


class ResNormSpec:
    """What a boundary between two blocks computes: the norms on either side, their
    fp32 vectors of `cols` elements (None: weight 1, bias 0), the residual scale and
    eps.  The vectors are held, and read at each call."""

    __slots__ = ("cols", "post", "pre", "alpha", "eps", "post_weight", "post_bias", "pre_weight",
                 "pre_bias")

    def __init__(self, cols, post="none", pre="rms", alpha=1.0, eps=1e-5, post_weight=None,
                 post_bias=None, pre_weight=None, pre_bias=None):
        self.cols = cols
        self.post, self.pre = _name(post, NORMS, "post"), _name(pre, NORMS, "pre")
        self.alpha, self.eps = alpha, eps
        self.post_weight, self.post_bias = post_weight, post_bias
        self.pre_weight, self.pre_bias = pre_weight, pre_bias

    def _c(self, T, C, ref, gate):
        if C != self.cols:
            raise ValueError("the layer has %d columns, the tensors %d" % (self.cols, C))
        dev = ref.get_device()
        gp, gd, per = None, 0, 1
        if gate is not None:
            groups = gate.shape[0] if gate.dim() == 2 else 1
            if groups > 0 and T % groups or groups < 1 and T > 0:
                raise ValueError("gate: %d rows do not divide %d" % (groups, T))
            if gate.dtype != torch.float32 and gate.dtype != ref.dtype:
                raise TypeError("gate is %s, expected float32 or %s" % (gate.dtype, ref.dtype))
            gp = _flat(gate, "gate", groups * C, gate.dtype, dev)
            gd, per = _dtype_code(gate), max(1, T // max(1, groups))
        return _Layer(T, C, _dtype_code(ref), self.post, self.pre,
                      _cols(self.post_weight, "post_weight", C, dev),
                      _cols(self.post_bias, "post_bias", C, dev),
                      _cols(self.pre_weight, "pre_weight", C, dev),
                      _cols(self.pre_bias, "pre_bias", C, dev), self.alpha, self.eps, gp, gd, per)


def _stats(t, name, T, dev):
    return None if t is None else _flat(t, name, 2 * T, torch.float32, dev)


def iabn_resnorm_forward(layer, r, b, r_out, n, gate=None, post_stats=None, pre_stats=None,
                         codes_b=None, exps_b=None, codes_n=None, exps_n=None, stream=None):
    """r_out = r + alpha * gate * post(b), n = pre(r_out).  gate: [cols] or [1, cols] for
    every row, or [groups, cols] with rows / groups consecutive rows each."""
    rp, ldr, T, C = _rows(r, "r")
    bp, ldb = _like(b, "b", T, C, r)
    op, ldo = _like(r_out, "r_out", T, C, r)
    np_, ldn = _like(n, "n", T, C, r)
    dev = r.get_device()
    cb, eb = _codes(codes_b, exps_b, "b", T, C, dev)
    cn, en = _codes(codes_n, exps_n, "n", T, C, dev)
    c = layer._c(T, C, r, gate)
    s = _stream(stream, r)
    _check("iabn_resnorm_forward", lib.iabn_resnorm_forward(
        ctypes.byref(c), rp, ldr, bp, ldb, op, ldo, np_, ldn,
        _stats(post_stats, "post_stats", T, dev), _stats(pre_stats, "pre_stats", T, dev), cb, eb,
        cn, en, s))


def iabn_resnorm_workspace_size(rows, cols, rows_per_gate=1) -> int:
    return lib.iabn_resnorm_workspace_size(rows, cols, rows_per_gate)


def resnorm_workspace(rows, cols, rows_per_gate=1, device="cuda"):
    """A workspace tensor for iabn_resnorm_backward."""
    size = iabn_resnorm_workspace_size(rows, cols, max(1, rows_per_gate))
    return torch.empty(size, dtype=torch.uint8, device=device)


def iabn_resnorm_backward(layer, dr_out, dn, workspace, r_out=None, b=None, codes_n=None,
                          exps_n=None, codes_b=None, exps_b=None, post_stats=None,
                          pre_stats=None, gate=None, dr=None, db=None, dpost_weight=None,
                          dpost_bias=None, dpre_weight=None, dpre_bias=None, dgate=None,
                          stream=None):
    """Gradients of iabn_resnorm_forward from dr_out and dn (either may be None) and
    the saved tensors (r_out, b) or their codes."""
    ref = dn if dn is not None else dr_out
    if ref is None:
        raise ValueError("dr_out or dn is needed")
    _, _, T, C = _rows(ref, "dn" if dn is not None else "dr_out")
    dev = ref.get_device()
    dop, lddo = _like(dr_out, "dr_out", T, C, ref)
    dnp, lddn = _like(dn, "dn", T, C, ref)
    rp, ldr = _like(r_out, "r_out", T, C, ref)
    bp, ldb = _like(b, "b", T, C, ref)
    drp, lddr = _like(dr, "dr", T, C, ref)
    dbp, lddb = _like(db, "db", T, C, ref)
    cn, en = _codes(codes_n, exps_n, "n", T, C, dev)
    cb, eb = _codes(codes_b, exps_b, "b", T, C, dev)
    c = layer._c(T, C, ref, gate)
    dgp = None
    if dgate is not None:
        if gate is None:
            raise ValueError("dgate needs the gate")
        dgp = _flat(dgate, "dgate", gate.numel(), gate.dtype, dev)
    ws, wb = _space(workspace, ref)
    s = _stream(stream, ref)
    _check("iabn_resnorm_backward", lib.iabn_resnorm_backward(
        ctypes.byref(c), dop, lddo, dnp, lddn, rp, ldr, bp, ldb, cn, en, cb, eb,
        _stats(post_stats, "post_stats", T, dev), _stats(pre_stats, "pre_stats", T, dev), drp,
        lddr, dbp, lddb, _cols(dpost_weight, "dpost_weight", C, dev),
        _cols(dpost_bias, "dpost_bias", C, dev), _cols(dpre_weight, "dpre_weight", C, dev),
        _cols(dpre_bias, "dpre_bias", C, dev), dgp, ws, wb, s))
    if T == 0 and dgate is not None:
        # the library knows a gate's rows from those of the tensors, which are none here
        with torch.cuda.stream(torch.cuda.ExternalStream(s, device=dgate.device)):
            dgate.zero_()
