"""Attention, rotary positions and group norm in float64, with bounds of their rounding.

A bound is an elementwise limit of |got - exact| for a kernel that computes in float32
and rounds where the library says it does.  With u half a step of the storage type
(bf16 2^-8, f16 2^-11, f32 2^-24) and e = 2^-24:

attention's forward.  A score s = scale * sum_d q k is formed by D fused products: off by at
most (D + 2) e S, S = scale * sum_d |q k|; P = exp(s - m) / l is off by a factor of the
score's and the maximum's error (twice the largest), and of the exponential's and the
sum's own (2^-22 and Sk e).  Call all of it x(row) = 2 (D + 2) e max_j S + 2^-22 + Sk e.  P is
rounded to the storage type before it meets v (u), the products' sum has Sk terms (Sk e):
|out - exact| <= u |exact| + (u + x + Sk e) sum_j P |v|.

Backward.  delta sees the rounded out: u |out| more in each of its terms, and D e; dP has D
products.  dS = P (dP - delta) is off by P (x (|dP| + |delta|) + D e (sum |dO v| +
sum |dO out|) + u sum |dO out|), and u |dS| for its own rounding; dq, dk and dv sum
those errors with |k|, |q| and |dO|, and are rounded themselves.

A result below the type's smallest normal number is rounded to whole steps of its subnormals:
float16's are 2^-24 apart, so that its rounding is off by up to 2^-25 (TINY) where u |exact|
is less.

Every bound is doubled: the terms above are first order, and u |exact| is of the exact
value where the kernel rounds its own.
"""
import math

import torch

HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 2.0 ** -150, torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}
E = 2.0 ** -24


def visible(lq, lk, left, right):
    """[lq, lk]: which keys each query sees."""
    at = torch.arange(lq)[:, None] + (lk - lq)
    j = torch.arange(lk)[None]
    see = torch.ones(lq, lk, dtype=torch.bool)
    if left >= 0:
        see &= j >= at - left
    if right >= 0:
        see &= j <= at + right
    return see


def _one(q, k, v, do, scale, see, u, tiny):
    """One head of one sequence, float64 on the CPU: values and bounds of out, lse and the
    gradients."""
    D, n = q.shape[1], max(1, k.shape[0])
    if q.shape[0] == 0 or k.shape[0] == 0:         # zeros, exactly
        val = dict(out=torch.zeros_like(q), dq=torch.zeros_like(q), dk=torch.zeros_like(k),
                   dv=torch.zeros_like(k), lse=torch.full((q.shape[0],), -math.inf,
                                                          dtype=torch.float64))
        return val, {n_: torch.zeros_like(t) for n_, t in val.items()}
    s = scale * (q @ k.T)
    sa = scale * (q.abs() @ k.abs().T)
    s = s.masked_fill(~see, -math.inf)
    lse = torch.logsumexp(s, 1)
    p = torch.exp(s - torch.where(lse == -math.inf, 0.0, lse)[:, None])
    p = p.masked_fill(~see, 0.0)
    x = 2 * (D + 2) * E * sa.masked_fill(~see, 0.0).amax(1, keepdim=True) + 2.0 ** -22 + n * E
    out = p @ v
    val = dict(out=out, lse=lse)
    bound = dict(out=u * out.abs() + (u + x + n * E) * (p @ v.abs()),
                 lse=x[:, 0] + 4 * E * lse.abs().nan_to_num(posinf=0.0))
    if do is not None:
        dp, delta = do @ v.T, (do * out).sum(1, keepdim=True)
        dpa, da = do.abs() @ v.abs().T, (do.abs() * out.abs()).sum(1, keepdim=True)
        ds = p * (dp - delta)
        eds = u * ds.abs() + p * (x * (dp.abs() + delta.abs()) + (D + 2) * E * (dpa + da) + u * da)
        # f16 keeps nothing below 2^-24 of what it is scaled to (P to 2^10, dS to 2^6 at the
        # column's largest): added to be safe, far below u of the largest
        m = max(1, q.shape[0])
        val.update(dq=scale * ds @ k, dk=scale * ds.T @ q, dv=p.T @ do)
        bound.update(
            dq=u * val["dq"].abs() + scale * (eds + n * E * ds.abs()) @ k.abs(),
            dk=u * val["dk"].abs() + scale * (eds + m * E * ds.abs()).T @ q.abs(),
            dv=u * val["dv"].abs() + (p * (u + x + m * E)).T @ do.abs())
        if u == HALF[torch.float16]:
            bound["dv"] += 2.0 ** -34 * (see.double().T @ do.abs())
            small = see * 2.0 ** -30
            bound["dk"] += scale * (small * ds.abs().amax(0, keepdim=True)).T @ q.abs()
            bound["dq"] += scale * (small * ds.abs().amax(1, keepdim=True)) @ k.abs()
    for name in bound:
        if name != "lse":
            bound[name] = bound[name] + tiny
    return val, {k_: 2 * b for k_, b in bound.items()}


def attention(q, k, v, dout=None, scale=None, left=-1, right=-1, q_lens=None, k_lens=None):
    """(values, bounds) of a batch: q [B, Sq, H, D], k, v [B, Sk, KV, D] of a storage type;
    lists of lengths.  Rows behind a length: zeros (lse -inf)."""
    B, Sq, H, D = q.shape
    Sk, KV = k.shape[1:3]
    G, u = H // KV if KV else 1, HALF[q.dtype]
    scale = 1 / math.sqrt(D) if scale is None else scale
    d = lambda t: None if t is None else t.detach().double().cpu()  # noqa: E731
    tiny = TINY[q.dtype]
    q, k, v, dout = d(q), d(k), d(v), d(dout)
    names = dict(out=q, lse=None, dq=q, dk=k, dv=k) if dout is not None else dict(out=q, lse=None)
    zero = lambda like: torch.zeros(B, H, Sq, dtype=torch.float64) if like is None \
        else torch.zeros_like(like)  # noqa: E731
    val, bound = ({n: zero(t) for n, t in names.items()} for _ in range(2))
    val["lse"].fill_(-math.inf)
    for b in range(B):
        lq = Sq if q_lens is None else q_lens[b]
        lk = Sk if k_lens is None else k_lens[b]
        see = visible(lq, lk, left, right)
        for h in range(H):
            g = h // G
            x, y = _one(q[b, :lq, h], k[b, :lk, g], v[b, :lk, g],
                        None if dout is None else dout[b, :lq, h], scale, see, u, tiny)
            for dst, src in ((val, x), (bound, y)):
                dst["out"][b, :lq, h] = src["out"]
                dst["lse"][b, h, :lq] = src["lse"]
                if dout is not None:
                    dst["dq"][b, :lq, h] = src["dq"]
                    dst["dk"][b, :lk, g] += src["dk"]
                    dst["dv"][b, :lk, g] += src["dv"]
    return val, bound


def within(got, want, bound, name=""):
    """Asserts that every element of got is as far from want as bound at the most."""
    got = got.detach().double().cpu()
    same = (got == want) | (got.isnan() & want.isnan())
    off = torch.where(same, 0.0, (got - want).abs())
    over = ~(off <= bound + 1e-300)
    if over.any():
        i = tuple(int(t) for t in over.nonzero()[0])
        worst = (off / (bound + 1e-300)).nan_to_num(nan=math.inf).max()
        raise AssertionError("%s: %d of %d over their bound (by up to %.3g), first at %s: %r, "
                             "expected %r within %.3g" % (name, int(over.sum()), over.numel(),
                                                          worst, i, float(got[i]), float(want[i]),
                                                          float(bound[i])))


def rotary(x, positions, inv_freq, axis, interleaved=False, inverse=False):
    """(value, bound) of x [B, S, H, D] turned; positions [B, S, axes]."""
    u, tiny = HALF[x.dtype], TINY[x.dtype]
    x = x.detach().double().cpu()
    n = inv_freq.numel()
    angle = positions.double().cpu()[..., axis.long().cpu()] * inv_freq.cpu()
    co, si = torch.cos(angle)[:, :, None], torch.sin(angle)[:, :, None]
    if inverse:
        si = -si
    y, mag = x.clone(), x.abs()
    a, b = (x[..., 0:2 * n:2], x[..., 1:2 * n:2]) if interleaved else (x[..., :n], x[..., n:2 * n])
    ra, rb = a * co - b * si, b * co + a * si
    m = a.abs() + b.abs()
    if interleaved:
        y[..., 0:2 * n:2], y[..., 1:2 * n:2] = ra, rb
        mag[..., 0:2 * n:2] = mag[..., 1:2 * n:2] = m
    else:
        y[..., :n], y[..., n:2 * n] = ra, rb
        mag[..., :n] = mag[..., n:2 * n] = m
    # the angle, a part of a turn in float32 (half a turn at the most: pi e of it, twice for the
    # conversion and the function's argument), sine and cosine to 2 ulps, two products and a sum
    bound = u * y.abs() + (4 * math.pi + 8) * E * mag + tiny
    bound[..., 2 * n:] = 0.0
    # angles in float64: positions to 2^31 times 2^-53
    return y, 2 * bound + 2.0 ** -52 * mag * (1 + angle.abs().max())


def group_norm(x, dy, groups, weight, bias, act, param, eps):
    """(values, bounds) for x, dy [N, HW, C] of a storage type, float64 on the CPU."""
    u, tiny = HALF[x.dtype], TINY[x.dtype]
    x = x.detach().double().cpu()
    N, HW, C = x.shape
    M = HW * (C // groups)
    sp = lambda t: t[..., None].expand(N, groups, C // groups).reshape(N, 1, C)  # noqa: E731
    xg = x.view(N, HW, groups, C // groups)
    mean = xg.mean((1, 3))
    var = (xg - mean[:, None, :, None]).square().mean((1, 3))
    rstd = 1 / torch.sqrt(var + eps)
    w = torch.ones(C, dtype=torch.float64) if weight is None else weight.double().cpu()
    b = torch.zeros(C, dtype=torch.float64) if bias is None else bias.double().cpu()
    xhat = (x - sp(mean)) * sp(rstd)
    z = xhat * w + b
    if act == "identity":
        y, d, d2 = z, torch.ones_like(z), torch.zeros_like(z)
    elif act == "leaky_relu":
        y, d, d2 = (torch.where(z >= 0, z, param * z),
                    torch.where(z >= 0, 1.0, param).double(), torch.zeros_like(z))
    elif act == "silu":
        s = torch.sigmoid(z)
        y, d, d2 = z * s, s * (1 + z * (1 - s)), torch.full_like(z, 0.5)
    elif act == "gelu":
        phi = torch.special.ndtr(z)
        dens = torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
        y, d, d2 = z * phi, phi + z * dens, torch.full_like(z, 0.8)
    else:
        c = math.sqrt(2 / math.pi)
        th = torch.tanh(c * (z + 0.044715 * z ** 3))
        y = z * (1 + th) / 2
        d = (1 + th) / 2 + z / 2 * (1 - th * th) * c * (1 + 0.134145 * z * z)
        d2 = torch.full_like(z, 0.8)
    # The statistics: a thread's sums about its first value have up to R = 64 + M / 2^10 terms
    # of size up to the largest distance in the group; those errors average over the lanes
    # but are taken whole: R e of the mean of squares about a value of the group, 4 times the
    # variance plus the largest squared distance over the rows of a lane
    R = 64 + M / 1024
    far = (xg - mean[:, None, :, None]).abs().amax((1, 3))
    emean = R * E * (far + torch.sqrt(var)) + E * mean.abs()
    evar = R * E * (4 * var + 2 * far.square() / max(1.0, min(M, 64)))
    erstd = 0.5 * rstd * evar / (var + eps) + 2 * E * rstd          # absolute
    exhat = sp(rstd) * (sp(emean) + 2 * E * (x.abs() + sp(mean.abs()))) + \
        xhat.abs() * (sp(erstd) / sp(rstd) + 2 * E)
    ez = exhat * w.abs() + 2 * E * (xhat * w).abs() + 2 * E * (z.abs() + b.abs())
    # the activations' own error: some ulps of values of size |z| or 1
    ea = 16 * E * (z.abs() + 1) if act not in ("identity", "leaky_relu") else 2 * E * z.abs()
    val = dict(y=y, stats=torch.stack((mean, rstd), -1))
    bound = dict(y=tiny + u * y.abs() + d.abs().clamp(min=1.2) * ez + ea,
                 stats=torch.stack((emean, erstd), -1))
    if dy is not None:
        g = dy.detach().double().cpu()
        dz = g * d
        # act' moves by d2 (at most) times z's error; a kink is crossed within ez of it
        kink = ((z.abs() <= 4 * ez) & (act == "leaky_relu")).double() * abs(1 - param)
        edz = g.abs() * (d2 * ez + ea.clamp(min=4 * E) + kink) + 2 * E * dz.abs()
        val["dweight"], val["dbias"] = (dz * xhat).sum((0, 1)), dz.sum((0, 1))
        bound["dweight"] = (edz * xhat.abs() + dz.abs() * exhat + R * E * (dz * xhat).abs()).sum((0, 1))
        bound["dbias"] = (edz + R * E * dz.abs()).sum((0, 1))
        q, eq = dz * w, edz * w.abs()
        mean_of = lambda t: sp(t.view(N, HW, groups, -1).mean((1, 3)))  # noqa: E731
        m1, m2 = mean_of(q), mean_of(q * xhat)
        em1 = mean_of(eq + R * E * q.abs())
        em2 = mean_of(eq * xhat.abs() + q.abs() * exhat + R * E * (q * xhat).abs())
        inner = q - m1 - xhat * m2
        val["dx"] = sp(rstd) * inner
        ei = eq + em1 + exhat * m2.abs() + xhat.abs() * em2 + 4 * E * (q.abs() + m1.abs() +
                                                                     (xhat * m2).abs())
        bound["dx"] = tiny + u * val["dx"].abs() + sp(rstd) * ei + sp(erstd) * inner.abs()
    return val, {k: 2 * v for k, v in bound.items()}
