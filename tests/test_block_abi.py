"""The residual-block entry points reject bad arguments before any HIP call (CPU
only: fake addresses, no call that would launch), and so does the binding."""
import ctypes

import pytest
import torch

iabn = pytest.importorskip("place_batchnorm_activation_amd")
lib = iabn.lib
from place_batchnorm_activation_amd import block  # noqa: E402

OK, INVALID, UNSUPPORTED, WS, MISALIGNED = 0, 1, 2, 3, 4
M = 1 << 24                    # fake device addresses M, 2M, ...: never dereferenced
F32, BF16, F16 = 0, 1, 2


def pack(x=M, ld=40, T=4, C=40, dt=BF16, codes=2 * M, exps=3 * M):
    return lib.iabn_codes_pack(x, ld, T, C, dt, codes, exps, None)


def unpack(codes=2 * M, exps=3 * M, T=4, C=40, scale=None, shift=None, y=M, ld=40, dt=BF16):
    return lib.iabn_codes_unpack(codes, exps, T, C, scale, shift, y, ld, dt, None)


def test_codes_validation():
    for f in (pack, unpack):
        assert f(T=0) == OK and f(C=0) == OK
        assert f(T=0, codes=None, exps=None) == OK
        assert f(T=-1) == INVALID and f(C=-1) == INVALID and f(dt=3) == INVALID
        assert f(T=1 << 31) == UNSUPPORTED and f(C=1 << 31, ld=1 << 31) == UNSUPPORTED
        assert f(ld=39) == INVALID
        assert f(codes=None) == INVALID and f(exps=None) == INVALID
        assert f(codes=2 * M + 8) == MISALIGNED
        # codes over the tensor: 4 rows of 64 bytes, and of 2 bytes of exponents
        assert f(codes=M + 16) == INVALID and f(exps=M) == INVALID
        assert f(T=(1 << 31) - 1, ld=1 << 40) == UNSUPPORTED
    assert pack(x=None) == INVALID and pack(x=M + 1) == MISALIGNED
    assert pack(dt=F32, x=M + 2) == MISALIGNED
    assert unpack(y=None) == INVALID and unpack(scale=M + 1) == MISALIGNED
    assert unpack(shift=M + 2) == MISALIGNED


def glu_f(g=M, ldg=80, u=M + 80, ldu=80, o=4 * M, ldo=40, T=4, F=40, dt=BF16, act=0, cg=5 * M,
          eg=6 * M, cu=7 * M, eu=8 * M):
    return lib.iabn_glu_forward(g, ldg, u, ldu, o, ldo, T, F, dt, act, cg, eg, cu, eu, None)


def glu_b(cg=5 * M, eg=6 * M, cu=7 * M, eu=8 * M, d=M, ldd=40, dg=2 * M, lddg=80, du=2 * M + 80,
          lddu=80, o=4 * M, ldo=40, T=4, F=40, dt=BF16, act=0):
    return lib.iabn_glu_backward(cg, eg, cu, eu, d, ldd, dg, lddg, du, lddu, o, ldo, T, F, dt,
                                 act, None)


def test_glu_validation():
    assert glu_f(T=0) == OK and glu_b(F=0) == OK
    assert glu_f(act=3) == INVALID and glu_b(act=-1) == INVALID
    assert glu_f(g=None) == INVALID and glu_f(o=None) == INVALID
    assert glu_f(ldg=39) == INVALID and glu_f(ldo=8) == INVALID
    # codes of both inputs or of none
    assert glu_f(cu=None, eu=None) == INVALID
    assert glu_f(cg=None, eg=None) == INVALID
    assert glu_f(eg=None) == INVALID and glu_f(u=None) == INVALID
    # out over gate only exactly; halves of one buffer are apart, shifted ones not
    assert glu_f(o=M + 2, ldo=80) == INVALID
    assert glu_f(o=M, ldo=40) == INVALID
    assert glu_f(o=M + 40, ldo=80) == INVALID
    assert glu_f(cg=M) == INVALID and glu_f(eu=4 * M) == INVALID
    assert glu_b(d=None) == INVALID and glu_b(dg=None) == INVALID
    assert glu_b(du=None) == INVALID and glu_b(cu=None, eu=None) == INVALID
    assert glu_b(dg=2 * M, du=2 * M + 40) == INVALID       # overlapping gradients
    assert glu_b(o=2 * M) == INVALID and glu_b(dg=M + 2, lddg=40) == INVALID
    assert glu_b(dg=5 * M) == INVALID                      # over the codes
    assert glu_b(dt=F32, d=M + 2) == MISALIGNED


def wgrad(dy=M, ldd=64, dt=BF16, c=2 * M, e=3 * M, s=None, t=None, dw=4 * M, ldw=48, wdt=F32,
          db=None, T=4, N=64, K=48, ws=None, wsb=0, acc=0):
    return lib.iabn_linear_wgrad(dy, ldd, dt, c, e, s, t, dw, ldw, wdt, db, acc, T, N, K, ws, wsb,
                                 None)


def test_wgrad_validation():
    assert wgrad(N=0) == OK and wgrad(K=0) == OK
    assert wgrad(N=-1) == INVALID and wgrad(K=-1) == INVALID and wgrad(T=-1) == INVALID
    assert wgrad(dt=5) == INVALID and wgrad(wdt=5) == INVALID
    assert wgrad(dy=None) == INVALID and wgrad(dw=None) == INVALID and wgrad(c=None) == INVALID
    assert wgrad(ldd=63) == INVALID and wgrad(ldw=47) == INVALID
    assert wgrad(dw=4 * M + 2) == MISALIGNED and wgrad(s=M + 1) == MISALIGNED
    assert wgrad(c=2 * M + 4) == MISALIGNED and wgrad(db=M + 2) == MISALIGNED
    assert wgrad(dw=M) == INVALID and wgrad(dw=2 * M) == INVALID
    assert wgrad(ldd=1 << 26) == UNSUPPORTED and wgrad(K=1 << 26, ldw=1 << 26) == UNSUPPORTED
    big = dict(T=100000, N=64, K=48)
    need = lib.iabn_linear_wgrad_workspace_size(100000, 64, 48, BF16)
    assert need > 0
    big = dict(T=100000, N=64, K=48, dy=1 << 40, c=1 << 41, e=1 << 42)
    assert wgrad(**big) == WS
    assert wgrad(ws=1 << 43, wsb=need - 1, **big) == WS
    assert wgrad(ws=(1 << 43) + 4, wsb=need, **big) == MISALIGNED
    assert lib.iabn_linear_wgrad_workspace_size(4, 64, 48, BF16) == 0
    assert lib.iabn_linear_wgrad_workspace_size(-1, 64, 48, BF16) == 0


def layer(T=4, C=40, dt=BF16, post=1, pre=1, alpha=1.0, eps=1e-5, gate=None, gd=0, R=1, pw=None):
    return block._Layer(T, C, dt, post, pre, pw, None, None, None, alpha, eps, gate, gd, R)


def rn_f(l=None, r=M, ldr=40, b=2 * M, ldb=40, ro=3 * M, ldro=40, n=4 * M, ldn=40, ps=None,
         ns=None, cb=None, eb=None, cn=None, en=None, **kw):
    l = l or layer(**kw)
    return lib.iabn_resnorm_forward(ctypes.byref(l), r, ldr, b, ldb, ro, ldro, n, ldn, ps, ns, cb,
                                    eb, cn, en, None)


def rn_b(l=None, dro=M, lddro=40, dn=2 * M, lddn=40, ro=3 * M, ldro=40, b=4 * M, ldb=40, cn=None,
         en=None, cb=None, eb=None, ps=5 * M, ns=6 * M, dr=7 * M, lddr=40, db=8 * M, lddb=40,
         dqw=None, dqb=None, dpw=None, dpb=None, dg=None, ws=9 * M, wsb=1 << 30, **kw):
    l = l or layer(**kw)
    return lib.iabn_resnorm_backward(ctypes.byref(l), dro, lddro, dn, lddn, ro, ldro, b, ldb, cn,
                                     en, cb, eb, ps, ns, dr, lddr, db, lddb, dqw, dqb, dpw, dpb,
                                     dg, ws, wsb, None)


def test_resnorm_validation():
    assert lib.iabn_resnorm_forward(None, M, 40, None, 0, M, 40, 2 * M, 40, *[None] * 7) == INVALID
    for f in (rn_f, rn_b):
        assert f(C=0) == OK
        assert f(T=-1) == INVALID and f(dt=3) == INVALID
        assert f(post=3) == INVALID and f(pre=-1) == INVALID
        assert f(alpha=float("nan")) == INVALID and f(eps=-1.0) == INVALID
        assert f(eps=float("inf")) == INVALID
        assert f(C=16385) == UNSUPPORTED
        assert f(pw=M + 1) == MISALIGNED
        # the gate: its type, whole groups of rows
        assert f(gate=10 * M, gd=F16, R=4) == INVALID
        assert f(gate=10 * M, R=3) == INVALID and f(gate=10 * M, R=0) == INVALID
        assert f(gate=10 * M + 2, R=4) == MISALIGNED
    assert rn_f(T=0) == OK
    assert rn_f(r=None) == INVALID and rn_f(n=None) == INVALID and rn_f(pre=0) == INVALID
    assert rn_f(pre=0, n=None, ro=None) == INVALID
    assert rn_f(ldr=39) == INVALID and rn_f(r=M + 1) == MISALIGNED
    assert rn_f(ro=4 * M) == INVALID                       # r_out over n
    assert rn_f(ro=M + 2) == INVALID and rn_f(n=2 * M + 2) == INVALID
    assert rn_f(cb=5 * M) == INVALID and rn_f(cn=5 * M + 8, en=6 * M) == MISALIGNED
    assert rn_f(b=None, cb=5 * M, eb=6 * M) == INVALID
    assert rn_f(cn=M, en=6 * M) == INVALID
    assert rn_b(pre=0) == INVALID                          # dn without a pre-norm
    assert rn_b(ns=None) == INVALID and rn_b(ps=None) == INVALID
    assert rn_b(ro=None) == INVALID and rn_b(b=None) == INVALID
    assert rn_b(cn=10 * M, en=11 * M) == INVALID           # codes and tensors mixed
    assert rn_b(db=None, dqw=12 * M) == INVALID
    assert rn_b(post=0, dqw=12 * M) == INVALID and rn_b(dg=12 * M) == INVALID
    assert rn_b(dr=8 * M) == INVALID                       # over db
    assert rn_b(dr=3 * M) == INVALID and rn_b(db=4 * M) == INVALID      # over what is saved
    assert rn_b(dr=M + 2) == INVALID
    assert rn_b(ws=None) == WS and rn_b(wsb=16) == WS and rn_b(ws=9 * M + 4) == MISALIGNED
    assert rn_b(dpw=12 * M + 1) == MISALIGNED


def test_resnorm_workspace_size_serves_every_gate():
    f = lib.iabn_resnorm_workspace_size
    assert f(0, 64, 1) == 0 and f(64, 0, 1) == 0 and f(64, 16385, 1) == 0 and f(64, 64, 0) == 0
    for T, C in ((1, 1), (4096, 512), (100000, 64), (7, 16384)):
        none = f(T, C, T)
        for R in (1, 2, T):
            assert f(T, C, R) >= none        # a call without a gate takes all rows as one


def test_binding_checks():
    t = lambda *s, dtype=torch.bfloat16: torch.empty(*s, dtype=dtype)     # noqa: E731
    codes, exps = iabn.codes_empty(4, 40, "cpu")
    assert codes.shape == (4, 64) and exps.shape == (4, 2)
    with pytest.raises(ValueError):
        iabn.iabn_codes_pack(t(5, 40), codes, exps, stream=0)             # other rows
    with pytest.raises(ValueError):
        iabn.iabn_codes_pack(t(40, 4).t(), codes, exps, stream=0)         # columns not contiguous
    with pytest.raises(ValueError):
        iabn.iabn_codes_pack(t(1, 40).expand(4, 40), codes, exps, stream=0)
    with pytest.raises(ValueError):
        iabn.iabn_codes_pack(t(2, 4, 40)[:, :2], codes, exps, stream=0)  # rows at two distances
    with pytest.raises(TypeError):
        iabn.iabn_codes_pack(t(4, 40, dtype=torch.float64), codes, exps, stream=0)
    with pytest.raises(TypeError):
        iabn.iabn_codes_pack(t(4, 40), codes.float(), exps, stream=0)
    with pytest.raises(ValueError):
        iabn.iabn_codes_pack(t(4, 40), codes, None, stream=0)
    with pytest.raises(TypeError):
        iabn.iabn_codes_unpack(codes, exps, t(4, 40), scale=t(40), stream=0)
    with pytest.raises(ValueError):
        iabn.iabn_glu_forward(t(4, 40), t(4, 41), t(4, 40), "silu", stream=0)
    with pytest.raises(TypeError):
        iabn.iabn_glu_forward(t(4, 40), None, t(4, 40, dtype=torch.float16), "silu", stream=0)
    with pytest.raises(ValueError):
        block._name("relu", block.GLU_ACTS, "act")
    with pytest.raises(ValueError):
        iabn.iabn_linear_wgrad(t(4, 6), codes, exps, t(7, 40, dtype=torch.float32), stream=0)
    with pytest.raises(ValueError):
        iabn.ResNormSpec(40, post="batch")
    layer = iabn.ResNormSpec(41)
    with pytest.raises(ValueError):
        iabn.iabn_resnorm_forward(layer, t(4, 40), None, None, t(4, 40), stream=0)
    layer = iabn.ResNormSpec(40)
    with pytest.raises(ValueError):
        iabn.iabn_resnorm_forward(layer, t(4, 40), t(4, 40), None, t(4, 40), gate=t(3, 40),
                                  stream=0)
    with pytest.raises(TypeError):
        iabn.iabn_resnorm_forward(layer, t(4, 40), t(4, 40), None, t(4, 40),
                                  gate=t(4, 40, dtype=torch.float16), stream=0)
    with pytest.raises(ValueError):
        iabn.iabn_resnorm_backward(layer, None, None, None)
    with pytest.raises(TypeError):                      # host tensors, all else being right
        iabn.iabn_resnorm_forward(layer, t(4, 40), None, None, t(4, 40), stream=0)


def test_tensors_of_no_rows_are_taken_with_any_strides():
    """An expanded gradient of an empty batch keeps strides of zero through contiguous()."""
    for shape in ((0, 40), (3, 0, 40), (0, 1)):
        t = torch.ones(()).expand(*shape)
        assert set(t.contiguous().stride()) <= {0, 1} and 0 in t.stride()
        ld, rows, cols = block._rows(t, "t")[1:]
        assert rows == 0 and cols == shape[-1] and ld >= cols
    with pytest.raises(ValueError):
        block._rows(torch.ones(()).expand(1, 40), "t")


def vectors(**kw):
    """A layer whose vectors lie at 20M .. 23M."""
    l = layer(**kw)
    l.post_weight, l.post_bias, l.pre_weight, l.pre_bias = (i * M for i in range(20, 24))
    return l


def test_outputs_keep_apart():
    """Outputs over one another, over vectors, statistics, codes and the workspace.  T = 4
    rows of 40: 320 bytes a tensor, 256 of codes, 8 of exponents, 160 a vector."""
    assert pack(exps=2 * M + 255) == INVALID and pack(codes=3 * M, exps=3 * M) == INVALID
    assert unpack(scale=M) == INVALID and unpack(shift=M + 316) == INVALID
    assert unpack(T=1, dt=F32, scale=M) == INVALID
    assert glu_f(cu=5 * M) == INVALID and glu_f(cu=5 * M + 240) == INVALID
    assert glu_f(eu=6 * M) == INVALID and glu_f(eg=5 * M + 255) == INVALID
    assert glu_f(eu=5 * M) == INVALID and glu_f(cu=6 * M) == INVALID

    for at in (M, 2 * M, 3 * M, 4 * M):                    # dy, codes, exps, dw
        assert wgrad(db=at) == INVALID
    assert wgrad(db=5 * M, s=5 * M) == INVALID and wgrad(db=5 * M, t=5 * M + 40) == INVALID
    assert wgrad(s=4 * M) == INVALID and wgrad(t=4 * M + 64) == INVALID       # dw over them
    big = dict(T=100000, dy=1 << 40, c=1 << 41, e=1 << 42, db=1 << 44)
    need = lib.iabn_linear_wgrad_workspace_size(100000, 64, 48, BF16)
    for at in (1 << 40, (1 << 41) + 16, 1 << 42, 4 * M, 1 << 44, (1 << 44) - need + 16):
        assert wgrad(ws=at, wsb=need, **big) == INVALID

    kept = dict(ps=5 * M, ns=6 * M, cb=7 * M, eb=8 * M, cn=9 * M, en=10 * M)
    for a in kept:
        for at in [M, 2 * M, 3 * M, 4 * M, 20 * M, 21 * M, 22 * M, 23 * M] + \
                [v for k, v in kept.items() if k != a]:
            assert rn_f(l=vectors(), **dict(kept, **{a: at})) == INVALID, (a, at)
    for at in (20 * M, 21 * M, 22 * M, 23 * M):
        assert rn_f(l=vectors(), ro=at) == INVALID and rn_f(l=vectors(), n=at) == INVALID
    gated = dict(gate=30 * M, gd=BF16)
    assert rn_f(l=vectors(R=2, **gated), n=30 * M) == INVALID
    assert rn_f(l=vectors(R=1, **gated), ro=30 * M + 2) == INVALID
    assert rn_f(l=vectors(R=1, **gated), ps=30 * M) == INVALID

    outs = dict(dr=7 * M, db=8 * M, dqw=12 * M, dqb=13 * M, dpw=14 * M, dpb=15 * M, dg=16 * M,
                ws=9 * M)
    def over(name, at, R=1, **kw):                         # noqa: E306
        return rn_b(l=vectors(R=R, **gated), **dict(outs, **{name: at}, **kw))
    for name in outs:
        ours = [v for k, v in outs.items() if k != name]
        for at in ours + [3 * M, 4 * M, 5 * M, 6 * M]:     # one another, and what was saved
            assert over(name, at) == INVALID, (name, at)
        if name[:2] not in ("dq", "dp"):
            for at in (20 * M, 21 * M, 22 * M):
                assert over(name, at) == INVALID, (name, at)
        if name not in ("dr", "db", "dg"):
            assert over(name, M) == INVALID and over(name, 2 * M) == INVALID
        if name != "dg":
            assert over(name, 30 * M) == INVALID, name
        coded = dict(ro=None, b=None, cn=40 * M, en=41 * M, cb=42 * M, eb=43 * M)
        for at in (40 * M, 41 * M, 42 * M, 43 * M):
            assert over(name, at, **coded) == INVALID, (name, at)
    assert over("dg", 30 * M, R=4, dr=30 * M) == INVALID
    assert over("dg", 30 * M + 2) == INVALID and over("dg", M + 2) == INVALID
