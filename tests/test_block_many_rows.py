"""The residual norms where a workgroup takes several rows, at every width that has a
kernel of its own: the next row's loads, exchange slots used again, gates reloaded at a
group's end, sums over the rows of a workgroup and of whole groups in it.  Against plain
float64 forms computed on the GPU, so that thousands of rows stay quick.

Tolerances as in tests/test_block_ops.py: the storage type's rounding, and in fp32 32
roundings (2^-24) of the magnitudes that enter a value, sums of a row included, and one
more for each row that a sum over rows has.
"""
import pytest
import torch

iabn = pytest.importorskip("place_batchnorm_activation_amd")
pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.float32: (2.0 ** -24, 2.0 ** -150), torch.bfloat16: (2.0 ** -8, 2.0 ** -134),
        torch.float16: (2.0 ** -11, 2.0 ** -25)}
EPS, ALPHA = 1e-5, 0.75


def within(got, want, tol, what):
    rel, small = HALF[got.dtype]
    err = (got.double() - want).abs() / (tol + rel * want.abs() + small)
    assert bool(torch.isfinite(got).all()), what
    assert float(err.max()) <= 1.0, "%s: error %.3g of what is allowed" % (what, float(err.max()))


def unit(x, kind):
    mean = x.mean(1, keepdim=True) if kind == "layer" else torch.zeros_like(x[:, :1])
    rstd = ((x - mean).square().mean(1, keepdim=True) + EPS).rsqrt()
    return (x - mean) * rstd, mean, rstd


def decoded(codes, exps, C):
    """Values of codes, and half a step of each."""
    e = exps.double().repeat_interleave(32, 1)
    step = torch.where(e > 0, torch.exp2(e - 127), 0.0)
    return (codes.double() * step)[:, :C], 0.5 * step[:, :C]


def back(g, xhat, kind, rstd, mag):
    """Gradient through the normalisation, and the magnitudes of its terms."""
    m = rstd * (mag + mag.mean(1, keepdim=True) +
                xhat.abs() * (mag * xhat.abs()).mean(1, keepdim=True))
    flat = g.mean(1, keepdim=True) if kind == "layer" else 0.0
    return rstd * (g - flat - xhat * (g * xhat).mean(1, keepdim=True)), m


def threads(C):
    """Threads that hold a row of the backward."""
    v = (C + 31) // 32 * 4
    return next((n for n in (64, 128, 256) if v <= n), 512)


@pytest.mark.parametrize("codes", [False, True], ids=["full", "codes"])
@pytest.mark.parametrize("kind,dtype,gated", [("rms", torch.bfloat16, "vector"),
                                              ("layer", torch.float16, "groups"),
                                              ("rms", torch.float32, "groups")], ids=str)
@pytest.mark.parametrize("T,C,R", [(9000, 512, 3), (9000, 509, 3), (4500, 1024, 3), (4500, 999, 2),
                                   (2300, 2048, 2), (2300, 1537, 4), (1200, 4096, 3),
                                   (1200, 4095, 2), (2400, 2056, 2), (2100, 4200, 3),
                                   (2400, 4107, 2), (1100, 8200, 2), (1100, 8205, 5)])
def test_resnorm_of_several_rows_a_workgroup(T, C, R, kind, dtype, gated, codes):
    print("case:", T, C, R, kind, dtype, gated, codes, flush=True)
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    assert T > cus * max(1, 1024 // threads(C)), "too few rows for this device"
    R = T if gated == "vector" else R
    gen = torch.Generator(device="cuda").manual_seed(T + C + R)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda")       # noqa: E731
    r, b, dro, dn = (rand(T, C) * torch.exp(0.3 * rand(T, 1)) for _ in range(4))
    r, b, dro, dn = (t.to(dtype) for t in (r, b, dro, dn))
    gate = (0.5 + 0.3 * rand(T // R, C)).to(torch.float32 if gated == "vector" else dtype)
    v = {k: a + 0.3 * rand(C) for k, a in (("post_weight", 1.0), ("pre_weight", 1.0))}
    if kind == "layer":
        v.update(post_bias=0.3 * rand(C), pre_bias=0.3 * rand(C))
    layer = iabn.ResNormSpec(C, post=kind, pre=kind, alpha=ALPHA, eps=EPS, **v)
    new = lambda: torch.full((T, C), 7.0, device="cuda", dtype=dtype)     # noqa: E731
    ro, n, dr, db = new(), new(), new(), new()
    st = dict(post_stats=torch.empty(T, 2, device="cuda"),
              pre_stats=torch.empty(T, 2, device="cuda"))
    kept = {}
    if codes:
        kept["codes_b"], kept["exps_b"] = iabn.codes_empty(T, C)
        kept["codes_n"], kept["exps_n"] = iabn.codes_empty(T, C)
    iabn.iabn_resnorm_forward(layer, r, b, ro, n, gate=gate, **st, **kept)

    w = {k: t.double() for k, t in v.items()}
    zero = torch.zeros(C, device="cuda", dtype=torch.float64)
    wb, ob, wn, on = (w.get(k, zero) for k in ("post_weight", "post_bias", "pre_weight",
                                               "pre_bias"))
    g64 = gate.double().repeat_interleave(R, 0)
    xb, mb, rb = unit(b.double(), kind)
    want = r.double() + ALPHA * g64 * (xb * wb + ob)
    reach_b = b.double().abs().amax(1, keepdim=True) * rb
    amp = r.double().abs() + ALPHA * g64.abs() * (reach_b * wb.abs() + ob.abs())
    top = amp.amax(1, keepdim=True)
    within(ro, want, 32 * U * amp, "r_out")
    xn, mn, rn = unit(want, kind)
    within(n, xn * wn + on, 32 * U * (top * rn * (1 + xn.abs()) * wn.abs() + on.abs()), "n")
    for name, mean, rstd, t in (("post", mb, rb, reach_b / rb), ("pre", mn, rn, top)):
        s = st[name + "_stats"]
        within(s[:, :1], mean, 32 * U * t, name + " mean")
        within(s[:, 1:], rstd, (32 * U * t * rstd + 8 * U) * rstd, name + " rstd")
    if codes:
        for name, x, reach in (("b", xb, reach_b), ("n", xn, top * rn)):
            val, half = decoded(kept["codes_" + name], kept["exps_" + name], C)
            slack = 32 * U * x.abs().amax(1, keepdim=True) * (1 + reach)
            assert bool(((val - x).abs() <= half + slack).all()), name
        xb, xn = (decoded(kept["codes_" + i], kept["exps_" + i], C)[0] for i in "bn")
        saved = kept
    else:
        ps, ns = st["post_stats"].double(), st["pre_stats"].double()
        xb, xn = (b.double() - ps[:, :1]) * ps[:, 1:], (ro.double() - ns[:, :1]) * ns[:, 1:]
        saved = dict(r_out=ro, b=b)
    rn, rb = st["pre_stats"][:, 1:].double(), st["post_stats"][:, 1:].double()

    outs = dict(dr=dr, db=db, dgate=torch.full_like(gate, 3.0))
    outs.update({"d" + k: torch.full((C,), 3.0, device="cuda") for k in v})
    ws = iabn.resnorm_workspace(T, C, R)
    ws.fill_(255)
    iabn.iabn_resnorm_backward(layer, dro, dn, ws, gate=gate, **st, **saved, **outs)

    d = dn.double()
    res, mag = {}, {}

    def rows_sum(name, term, size):
        res[name], mag[name] = term.sum(0), (32 + T) * U * size.sum(0)

    rows_sum("dpre_weight", d * xn, (d * xn).abs())
    rows_sum("dpre_bias", d, d.abs())
    D, mD = back(d * wn, xn, kind, rn, (d * wn).abs())
    D, mD = D + dro.double(), mD + dro.double().abs()
    res["dr"], mag["dr"] = D, 33 * U * mD
    p, mp = xb * wb + ob, (xb * wb).abs() + ob.abs()
    D, mD = ALPHA * D, ALPHA * mD
    res["dgate"] = (D * p).view(-1, R, C).sum(1)
    mag["dgate"] = (32 + R) * U * (mD * mp).view(-1, R, C).sum(1)
    D, mD = D * g64, mD * g64.abs()
    rows_sum("dpost_weight", D * xb, mD * xb.abs())
    rows_sum("dpost_bias", D, mD)
    res["db"], m = back(D * wb, xb, kind, rb, mD * wb.abs())
    mag["db"] = 33 * U * m
    for k, got in outs.items():
        within(got, res[k], mag[k], k)
    # a second run, over its own inputs: the same bits
    first = {k: t.clone() for k, t in outs.items()}
    iabn.iabn_resnorm_backward(layer, dro, dn, ws, gate=gate, **st, **saved,
                               **dict(outs, dr=dro, db=dn))
    assert torch.equal(dro, first["dr"]) and torch.equal(dn, first["db"])
    for k, t in first.items():
        assert torch.equal(outs[k], t), k
