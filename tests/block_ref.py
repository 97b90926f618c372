"""Plain float64 forms of the residual-block operators, from their definitions, on
the CPU (numpy): the oracle of tests/test_block_*.py.  Shares no code with the
library."""
import math

import numpy as np
import torch

U = 2.0 ** -24                      # half an ulp of 1 in fp32
#: half an ulp of the storage types, relative, and the smallest step below which it is
#: absolute
HALF = {torch.float32: (2.0 ** -24, 2.0 ** -150), torch.bfloat16: (2.0 ** -8, 2.0 ** -134),
        torch.float16: (2.0 ** -11, 2.0 ** -25)}


def f64(t):
    return None if t is None else t.detach().cpu().to(torch.float64).numpy()


def rounding(ref, dtype):
    rel, small = HALF[dtype]
    return rel * np.abs(ref) + small


def within(got, ref, tol, what=""):
    """|got - ref| <= tol elementwise; non-finite values must be the same ones."""
    got = f64(got) if isinstance(got, torch.Tensor) else got
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    bad = ~np.isfinite(ref)
    assert np.array_equal(np.isnan(got[bad]), np.isnan(ref[bad])), what
    err = np.abs(np.where(bad, 0, got) - np.where(bad, 0, ref))
    worst = np.max(err / np.where(bad, 1, tol)) if err.size else 0.0
    assert worst <= 1.0, "%s: error %.3g of what is allowed" % (what, worst)


def encode(x):
    """(codes int8 [T, Cp], exps uint8 [T, Cp/32]) of x [T, C] (float64 values of a storage
    type), group by group in integers and exact scaling."""
    T, C = x.shape
    G = (C + 31) // 32
    codes, exps = np.zeros((T, G * 32), np.int8), np.zeros((T, G), np.uint8)
    pad = np.zeros((T, G * 32))
    pad[:, :C] = x
    pad = pad.reshape(T, G, 32)
    q = codes.reshape(T, G, 32)
    with np.errstate(invalid="ignore", over="ignore"):
        finite = np.isfinite(pad).all(-1)
        amax = np.abs(pad).max(-1)
    exps[~finite] = 255
    for e in range(-126, 122):
        # the first exponent under which the largest magnitude rounds to at most 127
        # (the last one takes what is left, limited to 127)
        todo = finite & (amax > 0) & (exps == 0)
        if not todo.any():
            break
        fits = todo & ((np.rint(np.ldexp(np.where(todo, amax, 0), -e)) <= 127) | (e == 121))
        exps[fits] = e + 127
        q[fits] = np.clip(np.rint(np.ldexp(pad[fits], -e)), -127, 127).astype(np.int8)
    return codes, exps


def decode(codes, exps, C):
    T = codes.shape[0]
    E = np.repeat(exps.astype(np.int64), 32, 1)
    v = np.ldexp(codes.astype(np.float64), (E - 127).astype(np.int32))
    v = np.where(E == 0, 0.0, v)
    return np.where(E == 255, np.nan, v)[:, :C]


_erf = np.vectorize(math.erf, otypes=[np.float64])


def act(x, name):
    """(act, act') in float64."""
    with np.errstate(over="ignore", under="ignore"):
        if name == "silu":
            s = 1 / (1 + np.exp(-x))
            return x * s, s * (1 + x * (1 - s))
        if name == "gelu":
            P = 0.5 * (1 + _erf(x / math.sqrt(2)))
            return x * P, P + x * np.exp(-x * x / 2) / math.sqrt(2 * math.pi)
        k = math.sqrt(2 / math.pi)
        t = np.tanh(k * (x + 0.044715 * x ** 3))
        return 0.5 * x * (1 + t), 0.5 * (1 + t) + 0.5 * x * (1 - t * t) * k * (1 + 0.134145 * x * x)


def norm(x, kind, eps):
    """(xhat, mean, rstd)."""
    m = x.mean(1, keepdims=True) if kind == "layer" else np.zeros((len(x), 1))
    if kind == "none":
        return x, m, np.ones((len(x), 1))
    r = 1 / np.sqrt(((x - m) ** 2).mean(1, keepdims=True) + eps)
    return (x - m) * r, m, r


def spread(gate, T, C):
    if gate is None:
        return np.ones((1, C))
    g = gate.reshape(-1, C)
    return np.repeat(g, T // len(g), 0)


def resnorm(r, b, p):
    """Forward; p: dict of post, pre, alpha, eps, weights (or None) and gate."""
    T, C = r.shape
    one = lambda w: np.ones(C) if w is None else w      # noqa: E731
    nil = lambda w: np.zeros(C) if w is None else w     # noqa: E731
    o = {}
    ro = r
    if b is not None:
        xb, mb, rb = norm(b, p["post"], p["eps"])
        br = xb * one(p["post_weight"]) + nil(p["post_bias"]) if p["post"] != "none" else xb
        ro = r + p["alpha"] * spread(p["gate"], T, C) * br
        o.update(xb=xb, mb=mb, rb=rb, branch=br)
    o["r_out"] = ro
    if p["pre"] != "none":
        xn, mn, rn = norm(ro, p["pre"], p["eps"])
        o.update(xn=xn, mn=mn, rn=rn, n=xn * one(p["pre_weight"]) + nil(p["pre_bias"]))
    return o


def resnorm_grad(dro, dn, xn, rn, xb, rb, p, gate_rows):
    """Backward, and for each output the sum of the magnitudes of its terms (what its
    rounding errors are relative to)."""
    T, C = (dn if dn is not None else dro).shape
    one = lambda w: np.ones(C) if w is None else w      # noqa: E731
    nil = lambda w: np.zeros(C) if w is None else w     # noqa: E731
    D = np.zeros((T, C)) if dro is None else dro
    mag = np.abs(D)
    o, m = {}, {}
    if dn is not None:
        q = dn * one(p["pre_weight"])
        c1 = (q * xn).mean(1, keepdims=True)
        c0 = q.mean(1, keepdims=True) if p["pre"] == "layer" else 0.0
        D = D + rn * (q - c0 - xn * c1)
        mag = mag + rn * (np.abs(q) + np.abs(q).mean(1, keepdims=True) +
                          np.abs(xn) * np.abs(q * xn).mean(1, keepdims=True))
        o["dpre_weight"], m["dpre_weight"] = (dn * xn).sum(0), np.abs(dn * xn).sum(0)
        o["dpre_bias"], m["dpre_bias"] = dn.sum(0), np.abs(dn).sum(0)
    o["dr"], m["dr"] = D, mag
    dz, mz = p["alpha"] * D, abs(p["alpha"]) * mag
    br = xb if p["post"] == "none" else xb * one(p["post_weight"]) + nil(p["post_bias"])
    mbr = np.abs(xb) if p["post"] == "none" else \
        np.abs(xb * one(p["post_weight"])) + np.abs(nil(p["post_bias"]))
    if p["gate"] is not None:
        o["dgate"] = (dz * br).reshape(gate_rows, -1, C).sum(1)
        m["dgate"] = (mz * mbr).reshape(gate_rows, -1, C).sum(1)
        g = spread(p["gate"], T, C)
        dz, mz = dz * g, mz * np.abs(g)
    if p["post"] == "none":
        o["db"], m["db"] = dz, mz
        return o, m
    o["dpost_weight"], m["dpost_weight"] = (dz * xb).sum(0), (mz * np.abs(xb)).sum(0)
    o["dpost_bias"], m["dpost_bias"] = dz.sum(0), mz.sum(0)
    h, mh = dz * one(p["post_weight"]), mz * np.abs(one(p["post_weight"]))
    e1 = (h * xb).mean(1, keepdims=True)
    e0 = h.mean(1, keepdims=True) if p["post"] == "layer" else 0.0
    o["db"] = rb * (h - e0 - xb * e1)
    m["db"] = rb * (mh + mh.mean(1, keepdims=True) +
                    np.abs(xb) * (mh * np.abs(xb)).mean(1, keepdims=True))
    return o, m
