"""The residual-block operators on the GPU, through the binding, against plain
float64 forms (tests/block_ref.py).

Tolerances.  Codes are compared for equality.  A computed value may be off by the
rounding of its storage type plus, in fp32, a count of roundings (times U = 2^-24)
of the magnitudes that enter it, sums included:
  glu      40 U of the factors' magnitudes: two dozen operations, and exp's argument,
           whose rounding grows with |x| (|x| <= 12 here: 12*1.45 U)
  wgrad    T/16 + 8 accumulations, each at most an ulp (2 U: the matrix unit's
           rounding is not pinned), of sum |dy x|
  resnorm  32 U of the terms' magnitudes (a row's sums add in trees of depth < 20)
           and, for sums over rows, a rounding a row of the fp32 part
"""
import numpy as np
import pytest
import torch

import block_ref as ref

iabn = pytest.importorskip("place_batchnorm_activation_amd")
pytestmark = pytest.mark.gpu

DTYPES = [torch.float32, torch.bfloat16, torch.float16]
U = ref.U


def gen(seed):
    return torch.Generator().manual_seed(seed)


def values(g, T, C, dtype, spread=1.0):
    """Rows of different sizes with a few large columns and some zeros."""
    x = torch.randn(T, C, generator=g) * torch.exp(spread * torch.randn(T, 1, generator=g))
    x = x * torch.where(torch.rand(C, generator=g) < 0.02, 12.0, 1.0)
    x[torch.rand(T, C, generator=g) < 0.02] = 0.0
    return x.to(dtype)


class Slice:
    """A T x C view at column `off` of a wider buffer of one value, and a check that
    the rest of the buffer still holds it."""

    def __init__(self, T, C, dtype, off=3, extra=5, fill=7.0):
        self.buf = torch.full((T + 2, C + off + extra), fill, device="cuda").to(dtype)
        self.view = self.buf[1:T + 1, off:off + C]
        self.fill, self.C, self.off = self.buf[0, 0].clone(), C, off

    def check(self):
        b = self.buf.clone()
        b[1:-1, self.off:self.off + self.C] = self.fill
        assert bool((b == self.fill).all()), "written outside the tensor"


# ---------------------------------------------------------------------------
# codes

SHAPES = [(1, 1), (3, 7), (2, 8), (5, 31), (4, 32), (7, 33), (3, 100), (130, 64), (2, 1001),
          (9, 4096)]


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("T,C", SHAPES)
def test_codes_are_the_definitions(T, C, dtype):
    print("case:", T, C, dtype, flush=True)
    x = values(gen(T * 7 + C), T, C, dtype, 3.0)
    want_q, want_e = ref.encode(ref.f64(x))
    for sliced in (False, True):
        if sliced:
            s = Slice(T, C, dtype)
            s.view.copy_(x)
            xd = s.view
        else:
            xd = x.cuda()
        codes, exps = iabn.codes_empty(T, C)
        codes.fill_(99)
        exps.fill_(99)
        iabn.iabn_codes_pack(xd, codes, exps)
        assert np.array_equal(codes.cpu().numpy(), want_q)
        assert np.array_equal(exps.cpu().numpy(), want_e)
        for out in (torch.float32, torch.bfloat16):
            y = Slice(T, C, out)
            iabn.iabn_codes_unpack(codes, exps, y.view)
            assert np.array_equal(ref.f64(y.view), ref.decode(want_q, want_e, C))
            y.check()


def test_codes_at_the_edges_of_the_format():
    """Groups of zeros, of subnormals, of the largest values, at the rounding
    boundaries of the scale, and with infinities or NaN."""
    f = np.float32
    rows = [np.zeros(32), np.full(32, -0.0), np.full(32, 1e-45), np.linspace(-1e-38, 1e-38, 32),
            np.full(32, 3.4028234e38), np.full(32, 2.0 ** -126), np.full(32, 2.0 ** -127)]
    for k in (-120, -3, 0, 90):
        for m in (127.0, 127.25, 127.49999, 127.5, 127.50001, 128.0, 64.0, 63.75):
            r = np.zeros(32)
            r[5], r[6], r[7], r[8] = m, -m / 2, 0.5, 1.5
            rows.append(r * 2.0 ** k)
    x = np.array(rows, dtype=f)
    special = np.tile(np.linspace(-2, 2, 32, dtype=f), (4, 1))
    special[0, 3], special[1, 31], special[2, 0] = np.inf, -np.inf, np.nan
    x = np.concatenate([x, special])
    wide = np.concatenate([x, x[::-1]], 1)            # neighbouring groups keep their own scale
    want_q, want_e = ref.encode(wide.astype(np.float64))
    t = torch.from_numpy(wide).cuda()
    codes, exps = iabn.codes_empty(*wide.shape)
    iabn.iabn_codes_pack(t, codes, exps)
    assert np.array_equal(exps.cpu().numpy(), want_e)
    assert np.array_equal(codes.cpu().numpy(), want_q)
    y = torch.empty_like(t)
    iabn.iabn_codes_unpack(codes, exps, y)
    want = ref.decode(want_q, want_e, wide.shape[1])
    assert np.array_equal(y.cpu().numpy().astype(np.float64), want, equal_nan=True)
    assert np.isnan(want).sum() == 2 * 3 * 32


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
def test_unpack_with_scale_and_shift(dtype):
    T, C = 11, 333
    g = gen(5)
    codes, exps = (torch.from_numpy(a).cuda() for a in ref.encode(
        ref.f64(values(g, T, C, torch.float32))))
    v = ref.decode(codes.cpu().numpy(), exps.cpu().numpy(), C)
    a, b = torch.randn(C, generator=g), torch.randn(C, generator=g)
    for s, t in ((a, b), (a, None), (None, b)):
        y = torch.empty(T, C, device="cuda", dtype=dtype)
        iabn.iabn_codes_unpack(codes, exps, y, None if s is None else s.cuda(),
                               None if t is None else t.cuda())
        want = v * (1 if s is None else ref.f64(s)) + (0 if t is None else ref.f64(t))
        ref.within(y, want, U * np.abs(want) + ref.rounding(want, dtype))


def test_codes_past_32_bit_offsets():
    """A tensor of more than 2^31 elements, and rows past the first launch's 2^31
    vectors: the last rows come out as they do on their own."""
    T, C = 1050000, 16400
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GiB")
    x = torch.zeros(T, C, device="cuda", dtype=torch.bfloat16)
    assert T * iabn.code_cols(C) // 8 > 1 << 31
    tail = values(gen(1), 5000, C, torch.bfloat16).cuda()
    x[-5000:] = tail
    codes, exps = iabn.codes_empty(T, C)
    iabn.iabn_codes_pack(x, codes, exps)
    c2, e2 = iabn.codes_empty(5000, C)
    iabn.iabn_codes_pack(tail, c2, e2)
    assert torch.equal(codes[-5000:], c2) and torch.equal(exps[-5000:], e2)
    assert int(exps[:1000].max()) == 0
    x.fill_(1.0)
    iabn.iabn_codes_unpack(codes, exps, x)
    y = torch.empty_like(tail)
    iabn.iabn_codes_unpack(c2, e2, y)
    assert torch.equal(x[-5000:], y) and float(x[:1000].abs().max()) == 0.0


#: fp32 columns whose bytes pass 32 bits: whole vectors, and a ragged end
LONG = [(1 << 30) + 72, (1 << 30) + 75]


@pytest.mark.parametrize("cols", LONG)
def test_codes_of_a_row_past_32_bit_offsets(cols):
    """One fp32 row of more than 2^30 columns, as a flat tensor makes: its first and last
    groups come out as they do on their own."""
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GiB")
    n = 4096 + cols % 32                                    # whole groups and the ragged end
    head, tail = (values(gen(s), 1, n, torch.float32)[0].cuda() for s in (1, 2))
    x = torch.zeros(cols, device="cuda")
    x[:n], x[-n:] = head, tail
    codes, exps = iabn.codes_empty(1, cols)
    iabn.iabn_codes_pack(x, codes, exps)
    p = iabn.code_cols(n)
    ends = {}
    for name, v in (("head", head), ("tail", tail)):
        ends[name] = iabn.codes_empty(1, n)
        iabn.iabn_codes_pack(v, *ends[name])
    assert torch.equal(codes[0, -p:], ends["tail"][0][0])
    assert torch.equal(exps[0, -p // 32:], ends["tail"][1][0])
    assert torch.equal(codes[0, :n - n % 32], ends["head"][0][0, :n - n % 32])
    assert int(exps[0, 1 << 20:-(1 << 20)].max()) == 0
    # back, alone and with a scale and a shift, to fp32 and (the vectors' rows only are
    # long there) bf16
    vec = torch.ones(cols, device="cuda")
    vec[-n:] = torch.linspace(1, 2, n, device="cuda")
    for scale in (None, vec):
        for dtype in (torch.float32, torch.bfloat16):
            y = torch.full((cols,), 5.0, device="cuda", dtype=dtype)
            iabn.iabn_codes_unpack(codes, exps, y, scale, scale)
            for at, v in ((slice(0, 4096), "head"), (slice(cols - n, cols), "tail")):
                k = at.stop - at.start
                want = torch.empty(n, device="cuda", dtype=dtype)
                s = None if scale is None else scale[at][:k].contiguous()
                if s is not None and k < n:
                    s = torch.cat((s, s.new_ones(n - k)))
                iabn.iabn_codes_unpack(*ends[v], want, s, s)
                assert torch.equal(y[at], want[:k])
            mid = y[1 << 20:-(1 << 20)]
            assert float(mid.min()) == float(mid.max()) == (0.0 if scale is None else 1.0)


# ---------------------------------------------------------------------------
# gated activation

ACTS = ["silu", "gelu", "gelu_tanh"]


@pytest.mark.parametrize("gated", [True, False], ids=["gated", "plain"])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("T,F", [(1, 1), (3, 7), (2, 64), (5, 333), (33, 1024)])
def test_glu(T, F, dtype, act, gated):
    print("case:", T, F, dtype, act, gated, flush=True)
    g = gen(T + F)
    h = torch.randn(T, 2 * F, generator=g).mul(3).clamp(-12, 12).to(dtype).cuda()
    gate, up = h[:, :F], h[:, F:] if gated else None
    dout = torch.randn(T, F, generator=g).to(dtype).cuda()
    out = Slice(T, F, dtype)
    kept = [iabn.codes_empty(T, F), iabn.codes_empty(T, F) if gated else (None, None)]
    iabn.iabn_glu_forward(gate, up, out.view, act, *kept[0], *kept[1])
    out.check()
    x, u = ref.f64(gate), ref.f64(up) if gated else np.ones((T, F))
    f, _ = ref.act(x, act)
    scale = np.abs(x * u)
    ref.within(out.view, f * u, 40 * U * scale + ref.rounding(f * u, dtype), "out")
    # the kept codes
    cg, eg = ref.encode(x)
    assert np.array_equal(kept[0][0].cpu().numpy(), cg)
    assert np.array_equal(kept[0][1].cpu().numpy(), eg)
    xh, uh = ref.decode(cg, eg, F), np.ones((T, F))
    if gated:
        cu, eu = ref.encode(u)
        assert np.array_equal(kept[1][0].cpu().numpy(), cu)
        assert np.array_equal(kept[1][1].cpu().numpy(), eu)
        uh = ref.decode(cu, eu, F)
    # inference: no codes, the same output
    o2 = torch.empty(T, F, device="cuda", dtype=dtype)
    iabn.iabn_glu_forward(gate, up, o2, act)
    assert torch.equal(o2, out.view)
    dh, again = Slice(T, (2 if gated else 1) * F, dtype), Slice(T, F, dtype)
    dg, du = dh.view[:, :F], dh.view[:, F:] if gated else None
    iabn.iabn_glu_backward(*kept[0], *kept[1], dout, dg, du, act, out=again.view)
    dh.check()
    again.check()
    d = ref.f64(dout)
    f, s = ref.act(xh, act)
    want = d * uh * s
    ref.within(dg, want, 40 * U * np.abs(d * uh) * (1 + np.abs(xh)) + ref.rounding(want, dtype),
               "dgate")
    if gated:
        ref.within(du, d * f, 40 * U * np.abs(d * xh) + ref.rounding(d * f, dtype), "dup")
    ref.within(again.view, f * uh, 40 * U * np.abs(xh * uh) + ref.rounding(f * uh, dtype), "again")
    # over its own input: gate replaced by out, dout by dgate
    h2, d2 = h.clone(), dout.clone()
    iabn.iabn_glu_forward(h2[:, :F], h2[:, F:] if gated else None, h2[:, :F], act)
    assert torch.equal(h2[:, :F], o2)
    iabn.iabn_glu_backward(*kept[0], *kept[1], d2, d2, torch.empty_like(d2) if gated else None, act)
    assert torch.equal(d2, dg)


@pytest.mark.parametrize("cols", LONG)
def test_glu_of_a_row_past_32_bit_offsets(cols):
    """Gate and up of one fp32 row each of more than 2^30 columns: the last columns are those
    of a short row."""
    if torch.cuda.mem_get_info()[0] < 48 << 30:
        pytest.skip("needs 48 GiB")
    n = 4096 + cols % 32
    ends = [values(gen(s), 1, n, torch.float32)[0].cuda() for s in (3, 4, 5)]
    gate, up, dout = (torch.zeros(cols, device="cuda") for _ in range(3))
    for t, e in zip((gate, up, dout), ends):
        t[-n:] = e

    def passes(g, u, d):
        m = g.numel()
        kept = [*iabn.codes_empty(1, m), *iabn.codes_empty(1, m)]
        out, dg, du, again = (torch.full_like(g, 7.0) for _ in range(4))
        iabn.iabn_glu_forward(g, u, out, "silu", *kept)
        iabn.iabn_glu_backward(*kept, d, dg, du, "silu", out=again)
        return out, dg, du, again

    for got, want in zip(passes(gate, up, dout), passes(*ends)):
        assert torch.equal(got[-n:], want)
        assert float(got[:-n].abs().max()) == 0.0


@pytest.mark.parametrize("act", ACTS)
def test_glu_far_from_zero(act):
    """Saturated, huge and non-finite inputs: no NaN where the value has none."""
    x = torch.tensor([[-3e38, -1e20, -200.0, -40.0, -15.9, -0.0, 0.0, 15.9, 40.0, 200.0, 1e20,
                       3e38]]).cuda()
    out, dg = torch.empty_like(x), torch.empty_like(x)
    ones = torch.ones_like(x)
    for i in range(x.shape[1]):
        v = x[:, i:i + 1].contiguous()
        c = iabn.codes_empty(1, 1)
        o, d = torch.empty_like(v), torch.empty_like(v)
        iabn.iabn_glu_forward(v, None, o, act, *c)
        iabn.iabn_glu_backward(*c, None, None, ones[:, :1].contiguous(), d, None, act)
        out[:, i:i + 1], dg[:, i:i + 1] = o, d
    assert bool(torch.isfinite(out).all()) and bool(torch.isfinite(dg).all())
    v = ref.f64(x)
    f, _ = ref.act(v, act)
    ref.within(out, f, 40 * U * np.abs(v) + 1e-30, "out")
    kept = np.concatenate([ref.decode(*ref.encode(v[:, i:i + 1]), 1) for i in range(v.shape[1])], 1)
    _, s = ref.act(kept, act)
    ref.within(dg, s, 40 * U * (1 + np.minimum(np.abs(kept), 300)) + 1e-30, "dgate")
    bad = torch.full((1, 40), 0.5).cuda()
    bad[0, 2] = float("nan")
    c, o, d = iabn.codes_empty(1, 40), torch.empty_like(bad), torch.empty_like(bad)
    iabn.iabn_glu_forward(bad, None, o, act, *c)
    assert torch.isnan(o).nonzero().tolist() == [[0, 2]]
    iabn.iabn_glu_backward(*c, None, None, torch.ones_like(bad), d, None, act)
    assert bool(torch.isnan(d[0, :32]).all()) and bool(torch.isfinite(d[0, 32:]).all())


@pytest.mark.parametrize("act", ACTS)
def test_glu_gradient_against_differences(act):
    """Inputs that are codes already, so that the backward differentiates the
    forward itself: its directional derivative against central differences."""
    T, F, h = 4, 96, 2.0 ** -6
    g = gen(3)
    x, u = (torch.randint(-63, 64, (T, F), generator=g).float() / 32 for _ in range(2))
    x[:, ::32], u[:, ::32] = 127 / 32, 127 / 32
    v, w, dout = (torch.randn(T, F, generator=g) for _ in range(3))
    kept = [iabn.codes_empty(T, F), iabn.codes_empty(T, F)]
    o = torch.empty(T, F, device="cuda")

    def loss(s):
        iabn.iabn_glu_forward((x + s * v).cuda(), (u + s * w).cuda(), o, act)
        return float((o.double().cpu() * dout).sum())

    iabn.iabn_glu_forward(x.cuda(), u.cuda(), o, act, *kept[0], *kept[1])
    dg, du = torch.empty_like(o), torch.empty_like(o)
    iabn.iabn_glu_backward(*kept[0], *kept[1], dout.cuda(), dg, du, act)
    got = float((dg.double().cpu() * v + du.double().cpu() * w).sum())
    terms = float((dg.double().cpu() * v).abs().sum() + (du.double().cpu() * w).abs().sum())
    want = (loss(h) - loss(-h)) / (2 * h)
    # h^2/6 of third derivatives of order one, and 2^-24 of the loss over h
    assert abs(got - want) < 4 * h * h * terms


# ---------------------------------------------------------------------------
# weight gradient

@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("T,N,K", [(1, 1, 1), (3, 5, 7), (64, 128, 128), (65, 130, 33),
                                   (200, 129, 257), (1, 300, 64), (1000, 64, 100),
                                   (5000, 96, 40), (2048, 256, 512), (300, 1000, 777)])
@pytest.mark.parametrize("affine", ["none", "scale", "shift"])
def test_linear_wgrad(T, N, K, dtype, affine):
    print("case:", T, N, K, dtype, affine, flush=True)
    g = gen(T + N + K)
    dys = Slice(T, N, dtype)
    dys.view.copy_(values(g, T, N, dtype, 0.5))
    dy = dys.view
    codes, exps = ref.encode(ref.f64(values(g, T, K, torch.float32, 0.5)))
    x = ref.decode(codes, exps, K)
    s = torch.randn(K, generator=g) if affine != "none" else None
    t = torch.randn(K, generator=g) if affine == "shift" else None
    d = ref.f64(dy)
    sv, tv = (ref.f64(s) if s is not None else np.ones(K),
              ref.f64(t) if t is not None else np.zeros(K))
    want = (d.T @ x) * sv + np.outer(d.sum(0), tv)
    mag = (np.abs(d).T @ np.abs(x)) * np.abs(sv) + np.outer(np.abs(d).sum(0), np.abs(tv))
    steps = (T / 16 + 8) * 2 * U
    ws = iabn.linear_wgrad_workspace(T, N, K, dtype)
    args = dict(scale=None if s is None else s.cuda(), shift=None if t is None else t.cuda())
    cd, ed = torch.from_numpy(codes).cuda(), torch.from_numpy(exps).cuda()
    dw = Slice(N, K, torch.float32)
    db = torch.full((N,), 3.0, device="cuda")
    iabn.iabn_linear_wgrad(dy, cd, ed, dw.view, ws, dbias=db, **args)
    dw.check()
    ref.within(dw.view, want, steps * mag + 1e-30, "dw")
    ref.within(db, d.sum(0), steps * np.abs(d).sum(0) + 1e-30, "dbias")
    # the same bits without the bias, and on a second run
    dw2 = torch.empty(N, K, device="cuda")
    iabn.iabn_linear_wgrad(dy, cd, ed, dw2, ws, **args)
    assert torch.equal(dw2, dw.view)
    # added to what is there, and in 16 bits
    base = torch.randn(N, K, generator=g).cuda()
    acc, bacc = base.clone(), db.clone()
    iabn.iabn_linear_wgrad(dy, cd, ed, acc, ws, dbias=bacc, accumulate=True, **args)
    assert torch.equal(acc, base + dw2) and torch.equal(bacc, db + db)
    for dt in (torch.bfloat16, torch.float16):
        low = torch.empty(N, K, device="cuda", dtype=dt)
        iabn.iabn_linear_wgrad(dy, cd, ed, low, ws, **args)
        assert torch.equal(low, dw2.to(dt))


@pytest.mark.parametrize("T,N,K", [(70, 2048, 2048), (200, 2053, 2090), (64, 4096, 1030),
                                   (5, 1100, 4100)])
@pytest.mark.parametrize("affine", ["scale", "shift"])
def test_linear_wgrad_large_tiles(T, N, K, affine):
    """Outputs of many tiles, whole and ragged; the sum over t is short, so that the
    float64 form stays quick."""
    test_linear_wgrad(T, N, K, torch.bfloat16, affine)


@pytest.mark.parametrize("T,N,K", [(70, 4096, 2090), (130, 2053, 4100), (4200, 1030, 600)])
@pytest.mark.parametrize("dtype", [torch.float16, torch.float32], ids=str)
def test_linear_wgrad_large_tiles_of_several_parts(T, N, K, dtype):
    test_linear_wgrad(T, N, K, dtype, "shift")


@pytest.mark.parametrize("T,N,K,affine", [(1100, 2040, 2090, "shift"), (1152, 2053, 2048, "scale")])
def test_linear_wgrad_large_tiles_in_parts(T, N, K, affine):
    """256 x 256 tiles whose sum over t is cut, with ragged last tiles and columns."""
    assert iabn.iabn_linear_wgrad_workspace_size(T, N, K, torch.bfloat16) >= 2 * N * (K + 1) * 4
    test_linear_wgrad(T, N, K, torch.bfloat16, affine)


@pytest.mark.parametrize("low", [torch.bfloat16, torch.float16], ids=str)
@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("T,N,K", [(200, 129, 257), (5000, 96, 40), (70, 2048, 2048),
                                   (1100, 2040, 2090)])
def test_linear_wgrad_added_to_16_bits(T, N, K, dtype, low):
    """The sum in fp32 of what was there and the product, rounded once; in one part and in
    several."""
    g = gen(T + K)
    dy = torch.randn(T, N, generator=g).to(dtype).cuda()
    codes, exps = iabn.codes_empty(T, K)
    iabn.iabn_codes_pack(torch.randn(T, K, generator=g).cuda(), codes, exps)
    s, t = (torch.randn(K, generator=g).cuda() for _ in range(2))
    ws = iabn.linear_wgrad_workspace(T, N, K, dtype)
    full = torch.empty(N, K, device="cuda")
    iabn.iabn_linear_wgrad(dy, codes, exps, full, ws, scale=s, shift=t)
    base = (T ** 0.5 * torch.randn(N, K, generator=g)).to(low).cuda()
    dw = Slice(N, K, low)
    dw.view.copy_(base)
    iabn.iabn_linear_wgrad(dy, codes, exps, dw.view, ws, scale=s, shift=t, accumulate=True)
    dw.check()
    assert torch.equal(dw.view, (base.float() + full).to(low))


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
def test_linear_wgrad_of_no_rows(dtype):
    dy = torch.empty(0, 6, device="cuda", dtype=dtype)
    codes, exps = iabn.codes_empty(0, 9)
    dw, db = torch.ones(6, 9, device="cuda"), torch.ones(6, device="cuda")
    iabn.iabn_linear_wgrad(dy, codes, exps, dw, accumulate=True, dbias=db)
    assert float(dw.min()) == 1.0 and float(db.min()) == 1.0
    iabn.iabn_linear_wgrad(dy, codes, exps, dw, dbias=db, shift=torch.ones(9, device="cuda"))
    assert float(dw.abs().max()) == 0.0 and float(db.abs().max()) == 0.0


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("T,N", [(4, 6), (300, 200), (5000, 96), (0, 6)])
def test_linear_wgrad_of_no_columns(T, N, dtype):
    """The bias's gradient of a layer without inputs, in one part and in several."""
    dy = torch.randn(T, N, generator=gen(T)).to(dtype).cuda()
    codes, exps = iabn.codes_empty(T, 0)
    ws = iabn.linear_wgrad_workspace(T, N, 0, dtype)
    assert (ws is not None) == (T == 5000)
    dw, db = torch.empty(N, 0, device="cuda"), torch.full((N,), 3.0, device="cuda")
    iabn.iabn_linear_wgrad(dy, codes, exps, dw, ws, dbias=db)
    d = ref.f64(dy)
    ref.within(db, d.sum(0), (T / 16 + 8) * 2 * U * np.abs(d).sum(0) + 1e-30)
    twice = db.clone()
    iabn.iabn_linear_wgrad(dy, codes, exps, dw, ws, dbias=twice, accumulate=True)
    assert torch.equal(twice, db + db)


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
def test_linear_wgrad_keeps_non_finite_values_in_place(dtype):
    """An infinity in dy reaches its row of dW only, a group of NaN codes its
    columns; the padding of the last group reaches nothing."""
    T, N, K = 100, 70, 70
    g = gen(9)
    dy = torch.randn(T, N, generator=g).to(dtype)
    x = torch.rand(T, K, generator=g) + 0.5
    dy[13, 4] = float("inf")
    x[50, 65] = float("nan")
    c, e = iabn.codes_empty(T, K)
    iabn.iabn_codes_pack(x.cuda(), c, e)
    dw = torch.empty(N, K, device="cuda")
    iabn.iabn_linear_wgrad(dy.cuda(), c, e, dw, iabn.linear_wgrad_workspace(T, N, K, dtype))
    nan = torch.zeros(N, K, dtype=torch.bool)
    nan[:, 64:] = True
    assert torch.equal(torch.isnan(dw).cpu(), nan)
    assert bool((dw[4, :64] == float("inf")).all())
    rest = dw[:, :64].cpu()
    rest[4] = 0
    assert bool(torch.isfinite(rest).all())


def test_linear_wgrad_reads_extreme_values_exactly():
    """Values whose bf16 parts span fp32's and f16's whole mantissas and exponents:
    one row, so that every product is a single exact term."""
    N, K = 40, 33
    for dtype in (torch.float32, torch.float16):
        top = 3.4028234e38 / 64 if dtype == torch.float32 else 65504.0
        dy = torch.linspace(-1, 1, N, dtype=torch.float64).mul(top).to(dtype)[None]
        dy[0, :4] = torch.tensor([top, -top, 1.0 + 2.0 ** -10, 2.0 ** -14 * 1.0009765625]).to(dtype)
        x = torch.ones(1, K)
        c, e = iabn.codes_empty(1, K)
        iabn.iabn_codes_pack(x.cuda(), c, e)
        dw = torch.empty(N, K, device="cuda")
        iabn.iabn_linear_wgrad(dy.cuda(), c, e, dw)
        assert torch.equal(dw.cpu(), dy[0].float()[:, None].expand(N, K))


def test_linear_wgrad_past_32_bit_offsets():
    T, N, K, ld = 70000, 64, 64, 32768
    big = torch.zeros(T, ld, device="cuda", dtype=torch.bfloat16)
    assert T * ld > 1 << 31
    dy = big[:, ld - N:]
    dy[-3000:] = torch.randn(3000, N, generator=gen(2)).to(torch.bfloat16).cuda()
    x = torch.randn(T, K, generator=gen(4)).cuda()
    c, e = iabn.codes_empty(T, K)
    iabn.iabn_codes_pack(x, c, e)
    dw = torch.empty(N, K, device="cuda")
    iabn.iabn_linear_wgrad(dy, c, e, dw, iabn.linear_wgrad_workspace(T, N, K, torch.bfloat16))
    xs = ref.decode(c[-3000:].cpu().numpy(), e[-3000:].cpu().numpy(), K)
    d = ref.f64(dy[-3000:])
    ref.within(dw, d.T @ xs, (T / 16 + 8) * 2 * U * (np.abs(d).T @ np.abs(xs)))


# ---------------------------------------------------------------------------
# residual norms

def layer_of(g, C, post, pre, gate, T, R, dtype, affine=True):
    v = lambda a: (a + 0.3 * torch.randn(C, generator=g)) if affine else None   # noqa: E731
    p = dict(post=post, pre=pre, alpha=0.7, eps=1e-5,
             post_weight=v(1.0) if post != "none" else None,
             post_bias=v(0.0) if post == "layer" else None,
             pre_weight=v(1.0) if pre != "none" else None,
             pre_bias=v(0.0) if pre == "layer" else None, gate=None)
    if gate == "vector":
        p["gate"] = 0.5 + 0.3 * torch.randn(1, C, generator=g)
    elif gate != "none":
        p["gate"] = (0.5 + 0.3 * torch.randn(T // R, C, generator=g)).to(dtype)
    return p


def spec(p, C):
    dev = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in p.items()}
    gate = dev.pop("gate")
    return iabn.ResNormSpec(C, **dev), gate


def as64(p):
    # the library holds alpha and eps in fp32
    q = {k: ref.f64(v) if isinstance(v, torch.Tensor) else v for k, v in p.items()}
    q["alpha"], q["eps"] = float(np.float32(p["alpha"])), float(np.float32(p["eps"]))
    return q


KINDS = [("rms", "rms"), ("none", "rms"), ("layer", "layer"), ("rms", "layer"), ("none", "none"),
         ("layer", "none")]


def check_resnorm(T, C, dtype, post, pre, gate, R, codes, affine=True, seed=0, with_b=True):
    print("case:", T, C, dtype, post, pre, gate, R, "codes" if codes else "full", flush=True)
    g = gen(seed + T + C)
    r, b = values(g, T, C, dtype, 0.5), values(g, T, C, dtype, 0.5)
    p = layer_of(g, C, post, pre, gate, T, R, dtype, affine)
    layer, gt = spec(p, C)
    p64 = as64(p)
    o = ref.resnorm(ref.f64(r), ref.f64(b) if with_b else None, p64)
    new = lambda: Slice(T, C, dtype)                       # noqa: E731
    rs, bs, ro, n = new(), new(), new(), new()
    rs.view.copy_(r)
    bs.view.copy_(b)
    has_n = pre != "none"
    st = {k: torch.empty(T, 2, device="cuda") for k in ("post_stats", "pre_stats")}
    if post == "none" or not with_b:
        st["post_stats"] = None
    if not has_n:
        st["pre_stats"] = None
    cb, cn = iabn.codes_empty(T, C), iabn.codes_empty(T, C)
    kept = {}
    if codes:
        if with_b:
            kept.update(codes_b=cb[0], exps_b=cb[1])
        if has_n:
            kept.update(codes_n=cn[0], exps_n=cn[1])
    iabn.iabn_resnorm_forward(layer, rs.view, bs.view if with_b else None, ro.view,
                              n.view if has_n else None, gate=gt, **st, **kept)
    for s in (ro, n, rs, bs):
        s.check()

    amp = np.abs(ref.f64(r))
    if with_b:
        big = np.abs(o["branch"]) if post == "none" else \
            (np.abs(ref.f64(b)).max(1, keepdims=True) * o["rb"] *
             (1 if p64["post_weight"] is None else np.abs(p64["post_weight"])) +
             (0 if p64["post_bias"] is None else np.abs(p64["post_bias"])))
        amp = amp + abs(p64["alpha"]) * np.abs(ref.spread(p64["gate"], T, C)) * big
    ref.within(ro.view, o["r_out"], 32 * U * amp + ref.rounding(o["r_out"], dtype), "r_out")
    if has_n:
        w = 1 if p64["pre_weight"] is None else np.abs(p64["pre_weight"])
        lim = amp.max(1, keepdims=True) * o["rn"] * (1 + np.abs(o["xn"])) * w + \
            (0 if p64["pre_bias"] is None else np.abs(p64["pre_bias"]))
        ref.within(n.view, o["n"], 32 * U * lim + ref.rounding(o["n"], dtype), "n")
        rel = 32 * U * amp.max(1, keepdims=True) * o["rn"]
        ref.within(st["pre_stats"][:, 1:], o["rn"], (rel + 8 * U) * o["rn"], "pre rstd")
        ref.within(st["pre_stats"][:, :1], o["mn"],
                   32 * U * amp.max(1, keepdims=True) + 1e-30, "pre mean")
    if codes:
        # a code's value is within half a step of xhat (one more step's worth of slack
        # for the rounding of xhat itself is not needed: 1e-4 of a step is)
        for name, c, x in (("b", cb, o.get("xb")), ("n", cn, o.get("xn"))):
            if "codes_" + name not in kept:
                continue
            v = ref.decode(c[0].cpu().numpy(), c[1].cpu().numpy(), C)
            step = np.ldexp(1.0, np.repeat(c[1].cpu().numpy().astype(np.int32), 32, 1)[:, :C] - 127)
            slack = 32 * U * np.abs(x).max(1, keepdims=True) * \
                (1 + (amp.max(1, keepdims=True) * o["rn"] if name == "n" else
                      np.abs(ref.f64(b)).max(1, keepdims=True) * o["rb"]))
            assert (np.abs(v - x) <= 0.5 * step + slack).all(), name

    # backward
    dro, dn = (torch.randn(T, C, generator=g).to(dtype) for _ in range(2))
    dros, dns = new(), new()
    dros.view.copy_(dro)
    dns.view.copy_(dn)
    saved = {}
    f32 = lambda t: None if t is None else ref.f64(t)     # noqa: E731
    if codes:
        saved = kept
        dec = lambda c: ref.decode(c[0].cpu().numpy(), c[1].cpu().numpy(), C)   # noqa: E731
        xn, xb = dec(cn) if has_n else None, dec(cb) if with_b else None
    else:
        saved = dict(r_out=ro.view if has_n else None, b=bs.view if with_b else None)
        xn = (ref.f64(ro.view) - f32(st["pre_stats"])[:, :1]) * f32(st["pre_stats"])[:, 1:] \
            if has_n else None
        xb = ref.f64(b)
        if with_b and post != "none":
            xb = (xb - f32(st["post_stats"])[:, :1]) * f32(st["post_stats"])[:, 1:]
    rn = f32(st["pre_stats"])[:, 1:] if has_n else None
    rb = f32(st["post_stats"])[:, 1:] if with_b and post != "none" else np.ones((T, 1))
    if not with_b:
        xb = np.zeros((T, C))
    want, mag = ref.resnorm_grad(ref.f64(dro), ref.f64(dn) if has_n else None, xn, rn, xb, rb, p64,
                                 T // R if gate != "none" else 1)
    drs, dbs = new(), new()
    outs = dict(dr=drs.view)
    vec = lambda: torch.full((C,), 3.0, device="cuda")    # noqa: E731
    if has_n:
        outs["dpre_weight"] = vec()
        if pre == "layer":
            outs["dpre_bias"] = vec()
    if with_b:
        outs["db"] = dbs.view
        if post != "none":
            outs["dpost_weight"] = vec()
        if post == "layer":
            outs["dpost_bias"] = vec()
        if gt is not None:
            outs["dgate"] = torch.full_like(gt, 3.0)
    ws = iabn.resnorm_workspace(T, C, R)
    ws.fill_(255)                                         # its contents do not matter
    iabn.iabn_resnorm_backward(layer, dros.view, dns.view if has_n else None, ws, gate=gt, **st,
                               **saved, **outs)
    for s in (drs, dbs, dros, dns):
        s.check()
    for k, got in outs.items():
        dt = got.dtype
        rows = 1 if k in ("dr", "db") else R if k == "dgate" else T
        tol = (32 + rows) * U * mag[k] + ref.rounding(want[k], dt)
        ref.within(got.reshape(want[k].shape), want[k], tol, k)
    return layer, gt, st, saved, outs, (rs, bs, ro, n, dros, dns, ws)


@pytest.mark.parametrize("codes", [False, True], ids=["full", "codes"])
@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("T,C", [(1, 1), (3, 7), (2, 9), (5, 64), (4, 333), (3, 513), (130, 96),
                                 (3, 1000), (5, 1537), (2, 2055), (3, 4096)])
def test_resnorm_widths(T, C, dtype, codes):
    check_resnorm(T, C, dtype, "rms", "rms", "vector", T, codes)
    check_resnorm(T, C, dtype, "layer", "layer", "full", 1, codes)


@pytest.mark.parametrize("codes", [False, True], ids=["full", "codes"])
@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("C", [8192, 8200, 12289, 16384])
def test_resnorm_wide_rows(C, dtype, codes):
    check_resnorm(3, C, dtype, "rms", "rms", "none", 1, codes)
    check_resnorm(4, C, dtype, "layer", "layer", "rows", 2, codes)


@pytest.mark.parametrize("codes", [False, True], ids=["full", "codes"])
@pytest.mark.parametrize("gate", ["none", "vector", "rows", "full"])
@pytest.mark.parametrize("post,pre", KINDS)
def test_resnorm_kinds(post, pre, gate, codes):
    T = 12
    R = {"none": 1, "vector": T, "rows": 4, "full": 1}[gate]
    check_resnorm(T, 200, torch.bfloat16, post, pre, gate, R, codes)
    check_resnorm(T, 136, torch.float32, post, pre, gate, R, codes, affine=False)


@pytest.mark.parametrize("codes", [False, True], ids=["full", "codes"])
@pytest.mark.parametrize("T,R", [(6000, 6000), (6000, 3), (6000, 1), (6000, 2000), (6000, 12),
                                 (20000, 5000), (20000, 20)])
def test_resnorm_many_rows(T, R, codes):
    """Row blocks, gate groups inside and across workgroups."""
    gate = "vector" if T == R else "full" if R == 1 else "rows"
    check_resnorm(T, 72, torch.float32, "layer", "rms", gate, R, codes)


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
def test_resnorm_without_a_block(dtype):
    """b = None: the first norm of a network."""
    check_resnorm(5, 300, dtype, "none", "rms", "none", 1, False, with_b=False)
    check_resnorm(5, 300, dtype, "none", "layer", "none", 1, True, with_b=False)


@pytest.mark.parametrize("codes", [False, True], ids=["full", "codes"])
def test_resnorm_in_place(codes):
    """r' over r and n over b; dr over dr_out and db over dn: the same bits."""
    T, C = 9, 1000
    layer, gt, st, saved, outs, bufs = check_resnorm(T, C, torch.bfloat16, "rms", "rms", "vector",
                                                     T, codes)
    rs, bs, ro, n, dros, dns, ws = bufs
    want_dr, want_db = outs["dr"].clone(), outs["db"].clone()
    iabn.iabn_resnorm_backward(layer, dros.view, dns.view, ws, gate=gt, **st, **saved,
                               **dict(outs, dr=dros.view, db=dns.view))
    assert torch.equal(dros.view, want_dr) and torch.equal(dns.view, want_db)
    want_ro, want_n = ro.view.clone(), n.view.clone()
    iabn.iabn_resnorm_forward(layer, rs.view, bs.view, rs.view, bs.view, gate=gt)
    assert torch.equal(rs.view, want_ro) and torch.equal(bs.view, want_n)


@pytest.mark.parametrize("codes", [False, True], ids=["full", "codes"])
@pytest.mark.parametrize("T,C,R", [(9, 1000, 9), (8, 1001, 1), (8, 8200, 2), (4, 8200, 1),
                                   (600, 136, 2)])
def test_resnorm_gradients_over_what_they_are_of(T, C, R, codes):
    """dgate over the gate and the vectors' gradients over the vectors: the same bits."""
    gate = "vector" if R == T else "full" if R == 1 else "rows"
    layer, gt, st, saved, outs, bufs = check_resnorm(T, C, torch.bfloat16, "layer", "layer", gate,
                                                     R, codes)
    dros, dns, ws = bufs[4:]
    want = {k: v.clone() for k, v in outs.items()}
    outs = dict(outs, dgate=gt, **{"d" + k: getattr(layer, k) for k in
                                   ("post_weight", "post_bias", "pre_weight", "pre_bias")})
    iabn.iabn_resnorm_backward(layer, dros.view, dns.view, ws, gate=gt, **st, **saved, **outs)
    for k, v in outs.items():
        assert torch.equal(v, want[k]), k


def test_resnorm_rows_keep_to_themselves():
    """A row of zeros normalises to zeros, rows with an infinity or a NaN spoil
    themselves alone."""
    T, C = 6, 700
    g = gen(8)
    r, b = torch.randn(T, C, generator=g), torch.randn(T, C, generator=g)
    r[1], b[1] = 0.0, 0.0
    b[3, 17] = float("inf")
    r[4, 5] = float("nan")
    for kind in ("rms", "layer"):
        layer = iabn.ResNormSpec(C, post=kind, pre=kind)
        ro, n = torch.empty(T, C, device="cuda"), torch.empty(T, C, device="cuda")
        cn, cb = iabn.codes_empty(T, C), iabn.codes_empty(T, C)
        iabn.iabn_resnorm_forward(layer, r.cuda(), b.cuda(), ro, n, codes_b=cb[0], exps_b=cb[1],
                                  codes_n=cn[0], exps_n=cn[1])
        assert float(n[1].abs().max()) == 0.0 and float(ro[1].abs().max()) == 0.0
        assert int(cn[1][1].max()) == 0
        assert bool(torch.isfinite(n[[0, 1, 2, 5]]).all())
        assert bool(torch.isnan(n[4]).all()) and bool(torch.isnan(n[3]).any())
        assert int(cn[1][4].min()) == 255


@pytest.mark.parametrize("C", [1001, 1100, 1537, 4095])
def test_resnorm_gradients_that_overflowed(C):
    """An infinity in the last columns of dn or dr_out: the row's gradients are
    non-finite where the formula's are, other rows untouched."""
    T = 3
    g = gen(C)
    r, b, dro, dn = (torch.randn(T, C, generator=g) for _ in range(4))
    dn[1, C - 2] = float("inf")
    dro[2, C - 1] = float("-inf")
    p = dict(post="rms", pre="rms", alpha=1.0, eps=1e-5, post_weight=None, post_bias=None,
             pre_weight=None, pre_bias=None, gate=None)
    layer, _ = spec(p, C)
    ro, n = torch.empty(T, C, device="cuda"), torch.empty(T, C, device="cuda")
    st = dict(post_stats=torch.empty(T, 2, device="cuda"),
              pre_stats=torch.empty(T, 2, device="cuda"))
    iabn.iabn_resnorm_forward(layer, r.cuda(), b.cuda(), ro, n, **st)
    dr, db = torch.empty_like(ro), torch.empty_like(ro)
    iabn.iabn_resnorm_backward(layer, dro.cuda(), dn.cuda(), iabn.resnorm_workspace(T, C), r_out=ro,
                               b=b.cuda(), dr=dr, db=db, **st)
    pst, nst = ref.f64(st["post_stats"]), ref.f64(st["pre_stats"])
    with np.errstate(invalid="ignore"):
        want, mag = ref.resnorm_grad(ref.f64(dro), ref.f64(dn), ref.f64(ro) * nst[:, 1:], nst[:, 1:],
                                     ref.f64(b) * pst[:, 1:], pst[:, 1:], p, 1)
    for k, got in (("dr", dr), ("db", db)):
        assert np.array_equal(np.isnan(ref.f64(got)), np.isnan(want[k])), k
        assert np.array_equal(np.isinf(ref.f64(got)), np.isinf(want[k])), k
    assert np.isfinite(ref.f64(dr)[0]).all() and np.isinf(ref.f64(dr)[1]).any()


def test_resnorm_of_no_rows():
    C = 40
    w = torch.ones(C, device="cuda")
    layer = iabn.ResNormSpec(C, post="rms", pre="rms", pre_weight=w, post_weight=w)
    e = torch.empty(0, C, device="cuda")
    iabn.iabn_resnorm_forward(layer, e, e, torch.empty_like(e), torch.empty_like(e))
    dw = [torch.ones(C, device="cuda") for _ in range(2)]
    s = torch.empty(0, 2, device="cuda")
    iabn.iabn_resnorm_backward(layer, e, e, None, r_out=e, b=e, post_stats=s, pre_stats=s,
                               dr=torch.empty_like(e), db=torch.empty_like(e), dpre_weight=dw[0],
                               dpost_weight=dw[1])
    assert float(dw[0].abs().max()) == 0.0 and float(dw[1].abs().max()) == 0.0


@pytest.mark.parametrize("groups", [1, 3])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=str)
def test_resnorm_gate_gradient_of_no_rows(dtype, groups):
    """Zeros, also on another stream than the current one."""
    C = 40
    layer = iabn.ResNormSpec(C, post="rms", pre="rms")
    e, st = torch.empty(0, C, device="cuda", dtype=dtype), torch.empty(0, 2, device="cuda")
    gate = torch.ones(groups, C, device="cuda", dtype=dtype)
    for stream in (None, torch.cuda.Stream()):
        dgate = torch.full_like(gate, 3.0)
        torch.cuda.synchronize()
        iabn.iabn_resnorm_backward(layer, e, e, None, r_out=e, b=e, post_stats=st, pre_stats=st,
                                   gate=gate, dr=torch.empty_like(e), db=torch.empty_like(e),
                                   dgate=dgate, stream=stream)
        torch.cuda.synchronize()
        assert float(dgate.float().abs().max()) == 0.0


@pytest.mark.parametrize("post,pre,gate", [("rms", "rms", "vector"), ("layer", "layer", "full"),
                                           ("none", "layer", "none")])
def test_resnorm_gradient_against_differences(post, pre, gate):
    T, C, h = 6, 96, 2.0 ** -7
    g = gen(21)
    R = T if gate == "vector" else 1
    p = layer_of(g, C, post, pre, gate, T, R, torch.float32)
    names = [k for k in ("post_weight", "post_bias", "pre_weight", "pre_bias", "gate")
             if p[k] is not None]
    r, b, v, w, dro, dn = (torch.randn(T, C, generator=g) for _ in range(6))
    dirs = {k: torch.randn(p[k].shape, generator=g) for k in names}
    ro, n = torch.empty(T, C, device="cuda"), torch.empty(T, C, device="cuda")

    def forward(s, **kw):
        q = dict(p, **{k: p[k] + s * dirs[k] for k in names})
        layer, gt = spec(q, C)
        bd = (b + s * w).cuda()
        iabn.iabn_resnorm_forward(layer, (r + s * v).cuda(), bd, ro, n, gate=gt, **kw)
        return layer, gt, bd

    def loss(s):
        forward(s)
        return float((ro.double().cpu() * dro).sum() + (n.double().cpu() * dn).sum())

    want = (loss(h) - loss(-h)) / (2 * h)
    st = dict(pre_stats=torch.empty(T, 2, device="cuda"),
              post_stats=torch.empty(T, 2, device="cuda") if post != "none" else None)
    layer, gt, bd = forward(0.0, **st)
    outs = dict(dr=torch.empty_like(ro), db=torch.empty_like(ro))
    for k in names:
        outs["d" + k] = torch.empty_like(p[k], device="cuda")
    iabn.iabn_resnorm_backward(layer, dro.cuda(), dn.cuda(), iabn.resnorm_workspace(T, C, R),
                               r_out=ro, b=bd, gate=gt, **st, **outs)
    pairs = [(outs["dr"], v), (outs["db"], w)] + [(outs["d" + k], dirs[k]) for k in names]
    got = sum(float((a.double().cpu() * d).sum()) for a, d in pairs)
    terms = sum(float((a.double().cpu() * d).abs().sum()) for a, d in pairs)
    # h^2/6 of third derivatives of order a few, and 2^-24 of the loss over h
    assert abs(got - want) < 16 * h * h * terms


# ---------------------------------------------------------------------------
# streams, graphs, repeatability

def _step(T, C, N, bufs):
    """norm -> weight gradient -> gated unit on one set of buffers."""
    layer = bufs["layer"]
    iabn.iabn_resnorm_forward(layer, bufs["r"], bufs["b"], bufs["ro"], bufs["n"],
                              post_stats=bufs["ps"], pre_stats=bufs["ns"], codes_b=bufs["cb"],
                              exps_b=bufs["eb"], codes_n=bufs["cn"], exps_n=bufs["en"])
    iabn.iabn_glu_forward(bufs["ro"], bufs["n"], bufs["a"], "silu", bufs["cg"], bufs["eg"],
                          bufs["cu"], bufs["eu"])
    iabn.iabn_glu_backward(bufs["cg"], bufs["eg"], bufs["cu"], bufs["eu"], bufs["dy"], bufs["dg"],
                           bufs["du"], "silu", out=bufs["a2"])
    iabn.iabn_linear_wgrad(bufs["dg"], bufs["cn"], bufs["en"], bufs["dw"], bufs["wws"],
                           scale=layer.pre_weight, dbias=bufs["dbias"])
    iabn.iabn_resnorm_backward(layer, bufs["dg"], bufs["du"], bufs["ws"], codes_n=bufs["cn"],
                               exps_n=bufs["en"], codes_b=bufs["cb"], exps_b=bufs["eb"],
                               post_stats=bufs["ps"], pre_stats=bufs["ns"], dr=bufs["dr"],
                               db=bufs["db"], dpre_weight=bufs["dpw"], dpost_weight=bufs["dqw"])


OUTS = ("ro", "n", "a", "a2", "dg", "du", "dw", "dbias", "dr", "db", "dpw", "dqw")


def _buffers(T, C, seed):
    g = gen(seed)
    t = lambda: values(g, T, C, torch.bfloat16).cuda()       # noqa: E731
    e = lambda: torch.empty(T, C, device="cuda", dtype=torch.bfloat16)   # noqa: E731
    f = lambda *s: torch.empty(*s, device="cuda")            # noqa: E731
    b = dict(r=t(), b=t(), dy=t(), ro=e(), n=e(), a=e(), a2=e(), dg=e(), du=e(), dr=e(), db=e(),
             ps=f(T, 2), ns=f(T, 2), dw=f(C, C), dbias=f(C), dpw=f(C), dqw=f(C))
    for k in "bngu":
        b["c" + k], b["e" + k] = iabn.codes_empty(T, C)
    b["wws"] = iabn.linear_wgrad_workspace(T, C, C, torch.bfloat16)
    b["ws"] = iabn.resnorm_workspace(T, C)
    b["layer"] = iabn.ResNormSpec(C, post="rms", pre="rms",
                                  post_weight=torch.rand(C, generator=g).cuda(),
                                  pre_weight=torch.rand(C, generator=g).cuda())
    return b


def test_block_on_a_side_stream_and_in_a_graph():
    """Bits of the same step eagerly, again, on another stream, and in every replay of a
    captured graph, with new inputs and eager work between the replays."""
    T, C = 3000, 264
    b = _buffers(T, C, 3)
    _step(T, C, C, b)
    torch.cuda.synchronize()
    want = {k: b[k].clone() for k in OUTS}
    _step(T, C, C, b)
    torch.cuda.synchronize()
    for k in OUTS:
        assert torch.equal(b[k], want[k]), k
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for k in OUTS:
            b[k].zero_()
        _step(T, C, C, b)
    s.synchronize()
    for k in OUTS:
        assert torch.equal(b[k], want[k]), k
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _step(T, C, C, b)
    for i in range(4):
        other = _buffers(T, C, 50 + i)
        for k in ("r", "b", "dy"):
            b[k].copy_(other[k])
        other["layer"] = b["layer"]
        _step(T, C, C, other)
        graph.replay()
        torch.cuda.synchronize()
        for k in OUTS:
            assert torch.equal(b[k], other[k]), (i, k)
