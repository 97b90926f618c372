"""The entry points of attention, rotary positions and group norm reject bad arguments before any HIP
call (CPU only: fake addresses, no call that would launch), and so does the binding."""
import ctypes

import pytest
import torch

iabn = pytest.importorskip("place_batchnorm_activation_amd")
lib = iabn.lib
from place_batchnorm_activation_amd import heads  # noqa: E402

OK, INVALID, UNSUPPORTED, WS, MISALIGNED = 0, 1, 2, 3, 4
M = 1 << 28                    # fake device addresses M, 2M, ...: never dereferenced
F32, BF16, F16 = 0, 1, 2


def problem(**kw):
    p = dict(batch=2, heads=4, kv_heads=2, head_dim=64, q_len=300, k_len=300, dtype=BF16,
             scale=0.125, left=-1, right=0, q_starts=None, k_starts=None, q_rows=0, k_rows=0,
             q_lens=None, k_lens=None)
    p.update(kw)
    return heads._Problem(**p)


class Heads(ctypes.Structure):
    """iabn_heads of include/iabn.h."""
    _fields_ = [("data", ctypes.c_void_p), ("batch", ctypes.c_int64), ("row", ctypes.c_int64),
                ("head", ctypes.c_int64)]


def place(data, B=2, S=300, H=4, D=64, layout="bshd", **kw):
    row, head = (H * D, D) if layout == "bshd" else (D, S * D)
    h = dict(data=data, batch=S * H * D, row=row, head=head)
    h.update(kw)
    return Heads(**h)


def ref(t):
    return None if t is None else ctypes.byref(t)


def forward(p=None, q=place(M), k=place(2 * M, H=2), v=place(3 * M, H=2), out=place(4 * M),
            lse=5 * M, ws=6 * M, wb=1 << 40):
    return lib.iabn_attention_forward(ref(problem() if p is None else p), ref(q), ref(k), ref(v),
                                      ref(out), lse, ws, wb, None)


def backward(p=None, q=place(M), k=place(2 * M, H=2), v=place(3 * M, H=2), out=place(4 * M),
             lse=5 * M, dout=place(7 * M), dq=place(8 * M), dk=place(9 * M, H=2),
             dv=place(10 * M, H=2), ws=6 * M, wb=1 << 40):
    return lib.iabn_attention_backward(ref(problem() if p is None else p), ref(q), ref(k), ref(v),
                                       ref(out), lse, ref(dout), ref(dq), ref(dk), ref(dv), ws, wb,
                                       None)


@pytest.mark.parametrize("call", (forward, backward))
def test_attention_problem(call):
    assert call(problem(batch=0)) == OK and call(problem(heads=0, kv_heads=0)) == OK
    for bad in (dict(batch=-1), dict(heads=-4), dict(kv_heads=0), dict(kv_heads=3),
                dict(heads=0), dict(head_dim=0), dict(q_len=-1), dict(k_len=-1), dict(dtype=3),
                dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
                dict(scale=float("inf")), dict(q_starts=M, q_lens=M, q_rows=600),
                dict(k_starts=M, k_lens=M, k_rows=600), dict(q_starts=M, q_rows=-1)):
        assert call(problem(**bad)) == INVALID, bad
    for far in (dict(head_dim=136), dict(head_dim=60), dict(q_len=(1 << 29) + 1),
                dict(k_len=(1 << 28) + 1), dict(batch=1 << 40), dict(heads=1 << 30, kv_heads=1),
                dict(q_starts=M, q_rows=1 << 31),
                dict(batch=1 << 15, q_len=1 << 16), dict(batch=1 << 15, k_len=1 << 16)):
        assert call(problem(**far)) == UNSUPPORTED, far
    for odd in (dict(q_lens=M + 2), dict(k_starts=M + 1, k_rows=600)):
        assert call(problem(**odd)) == MISALIGNED, odd
    assert lib.iabn_attention_forward(None, *[None] * 5, None, 0, None) == INVALID


@pytest.mark.parametrize("heads", (1 << 25, 1 << 26, 1 << 29))
def test_attention_of_one_token_and_the_most_heads(heads):
    """64 groups of rows pass 32 bits; the workspace holds a number a row all the same."""
    p = problem(batch=1, heads=heads, kv_heads=1, q_len=1, k_len=1)
    assert lib.iabn_attention_workspace_size(ctypes.byref(p), 1) >= 4 * heads


def test_attention_without_queries():
    assert forward(problem(q_len=0)) == OK


@pytest.mark.parametrize("call", (forward, backward))
def test_attention_tensors(call):
    assert call(q=None) == INVALID and call(q=place(None)) == INVALID
    assert call(k=place(2 * M, H=2, row=-1)) == INVALID
    assert call(v=place(3 * M + 1, H=2)) == MISALIGNED
    assert call(out=place(4 * M, batch=1 << 52)) == UNSUPPORTED
    assert call(lse=5 * M + 2) == MISALIGNED


def test_attention_outputs_apart():
    assert forward(out=place(M)) == INVALID                     # over q
    assert forward(out=place(2 * M + 64)) == INVALID            # over k
    assert forward(lse=M + 4096) == INVALID                     # over q
    assert forward(lse=4 * M) == INVALID                        # over out
    assert forward(out=place(4 * M, row=0)) == INVALID          # rows in one place
    assert forward(out=place(4 * M, row=4 * 64 - 1)) == INVALID
    # the keys are cut among workgroups: the workspace is needed (float32, since 16-bit types
    # part the keys of so short a cache inside one workgroup, which needs none)
    few = problem(q_len=1, dtype=F32)
    short = problem(q_len=1)
    assert lib.iabn_attention_workspace_size(ctypes.byref(short), 0) == 0
    one = dict(q=place(M, S=1), out=place(4 * M, S=1))
    assert forward(few, ws=None, **one) == WS and forward(few, wb=64, **one) == WS
    assert forward(few, ws=6 * M + 8, **one) == MISALIGNED
    assert forward(few, ws=4 * M, **one) == INVALID
    # lengths that an output would write
    assert forward(problem(q_lens=4 * M)) == INVALID
    assert forward(problem(k_starts=4 * M, k_rows=600)) == INVALID


def test_attention_gradients_apart():
    assert backward(dq=place(M)) == INVALID and backward(dq=place(7 * M)) == INVALID
    assert backward(dk=place(10 * M, H=2)) == INVALID           # over dv
    assert backward(dv=place(4 * M, H=2)) == INVALID            # over out
    assert backward(dk=place(9 * M, H=2, head=32)) == INVALID   # heads overlap
    assert backward(lse=None) == INVALID
    assert backward(ws=None) == WS and backward(wb=8) == WS
    assert backward(ws=8 * M) == INVALID


def meets(a, b):
    """Whether an attention forward refuses out = b beside q = a as sharing memory (only ever
    called where it does, or where another argument is refused after that check)."""
    return forward(q=a, out=b, lse=4 * M + 2)


def test_slices_of_one_buffer_are_apart():
    """dq, dk and dv as slices of one projection's gradient pass the overlap check: what is
    refused is the workspace, which is checked against them together."""
    H, KV, D, S = 4, 2, 64, 300
    row = (H + 2 * KV) * D
    at = lambda first, n: Heads(data=8 * M + 2 * first * D, batch=S * row, row=row,  # noqa: E731
                                       head=D)
    dq, dk, dv = at(0, H), at(H, KV), at(H + KV, KV)
    # every pair of them alone is apart; with the workspace over one of them, refused
    assert backward(dq=dq, dk=dk, dv=dv, ws=8 * M + 4096) == INVALID
    # one head further they meet
    assert backward(dq=at(1, H), dk=dk, dv=dv) == INVALID


def rotary(spec=None, q=place(M), qh=4, qo=place(2 * M), k=place(3 * M, H=2), kh=2,
           ko=place(4 * M, H=2), **kw):
    r = dict(batch=2, rows=300, head_dim=64, pairs=32, axes=2, dtype=BF16, interleaved=0,
             inv_freq=5 * M, axis=6 * M, positions=7 * M, pos_type=0, pos_batch=600, pos_row=2)
    r.update(kw)
    return lib.iabn_rotary(ref(heads._Rotary(**r)), ref(q), qh, ref(qo), ref(k), kh, ref(ko), 0,
                           None)


def test_rotary_validation():
    assert rotary(batch=0) == OK and rotary(rows=0) == OK
    assert rotary(qh=0, kh=0, q=None, qo=None, k=None, ko=None) == OK
    for bad in (dict(batch=-1), dict(rows=-1), dict(qh=-1), dict(pairs=0), dict(pairs=33),
                dict(axes=0), dict(dtype=7), dict(pos_type=3), dict(pos_batch=-1),
                dict(pos_row=-2), dict(inv_freq=None), dict(positions=None), dict(q=None),
                dict(ko=None), dict(q=place(None))):
        assert rotary(**bad) == INVALID, bad
    assert rotary(head_dim=1 << 17) == UNSUPPORTED and rotary(batch=1 << 40) == UNSUPPORTED
    assert rotary(axes=1 << 17) == UNSUPPORTED and rotary(qh=1 << 17) == UNSUPPORTED
    for odd in (dict(q=place(M + 1)), dict(inv_freq=5 * M + 4), dict(axis=6 * M + 2),
                dict(positions=7 * M + 2), dict(positions=7 * M + 4, pos_type=1)):
        assert rotary(**odd) == MISALIGNED, odd
    # outputs: exactly their input or apart from everything
    assert rotary(qo=place(M + 128)) == INVALID and rotary(qo=place(3 * M)) == INVALID
    assert rotary(ko=place(2 * M, H=2)) == INVALID
    assert rotary(qo=place(5 * M)) == INVALID and rotary(qo=place(7 * M - 64)) == INVALID
    assert rotary(qo=place(2 * M, row=0)) == INVALID
    assert rotary(qo=place(M, layout="bhsd")) == INVALID        # q's memory in another order


def gn(**kw):
    p = dict(n=2, hw=100, c=48, groups=6, dtype=BF16, weight=7 * M, bias=8 * M, act=0,
             act_param=0.0, eps=1e-5)
    p.update(kw)
    return heads._GroupNorm(**p)


def gn_forward(l=None, x=M, ldx=48, y=2 * M, ldy=48, stats=3 * M, ws=4 * M, wb=1 << 30, **kw):
    return lib.iabn_group_norm_forward(ref(l or gn(**kw)), x, ldx, y, ldy, stats, ws, wb, None)


def gn_backward(x=M, ldx=48, dy=2 * M, lddy=48, dx=5 * M, lddx=48, stats=3 * M, dw=9 * M,
                db=10 * M, ws=4 * M, wb=1 << 30, **kw):
    return lib.iabn_group_norm_backward(ref(gn(**kw)), x, ldx, dy, lddy, dx, lddx, stats, dw, db,
                                        ws, wb, None)


def test_group_norm_validation():
    assert gn_forward(n=0) == OK and gn_forward(hw=0) == OK and gn_forward(c=0) == OK
    for call in (gn_forward, gn_backward):
        for bad in (dict(n=-1), dict(hw=-1), dict(c=-48), dict(groups=0), dict(groups=5),
                    dict(dtype=5), dict(act=5), dict(act=-1), dict(act_param=float("nan")),
                    dict(eps=-1.0), dict(eps=float("inf")), dict(x=None), dict(ldx=47)):
            assert call(**bad) == INVALID, bad
        for far in (dict(n=1 << 20, hw=1 << 20), dict(c=6 << 25, ldx=6 << 25)):
            assert call(**far) == UNSUPPORTED, far
        for odd in (dict(x=M + 1), dict(weight=7 * M + 1), dict(bias=8 * M + 2),
                    dict(stats=3 * M + 4), dict(ws=4 * M + 8)):
            assert call(**odd) == MISALIGNED, odd
        assert call(ws=None) == WS and call(wb=16) == WS
        assert call(ws=M) == INVALID and call(ws=3 * M) == INVALID
    assert gn_forward(y=M + 96) == INVALID and gn_forward(y=None) == INVALID
    assert gn_forward(y=7 * M - 32) == INVALID and gn_forward(stats=M) == INVALID
    assert gn_backward(stats=None) == INVALID and gn_backward(dy=None) == INVALID
    assert gn_backward(dx=M + 2) == INVALID and gn_backward(dx=9 * M) == INVALID
    assert gn_backward(dw=10 * M) == INVALID and gn_backward(dw=M) == INVALID
    assert gn_backward(dw=8 * M) == INVALID and gn_backward(dx=7 * M) == INVALID
    assert gn_backward(dx=None, dw=None, db=None) == OK


@pytest.mark.parametrize("groups", (1 << 24, (1 << 24) + 1, 3 << 24))
def test_group_norm_of_too_many_groups(groups):
    """A workgroup a group passes a launch's 2^32 threads: refused, and not after the first of
    several kernels.  One group less goes on to the workspace."""
    for call in (gn_forward, gn_backward):
        wide = dict(n=1, hw=2, c=groups, groups=groups, weight=None, bias=None, ldx=groups)
        ld = dict(ldy=groups) if call is gn_forward else dict(lddy=groups, lddx=groups, dw=None,
                                                              db=None)
        assert call(ws=None, **wide, **ld) == UNSUPPORTED
        if groups == 1 << 24:
            less = {n: v - 1 if v == groups else v for n, v in dict(wide, **ld).items()}
            assert call(ws=None, **less) == WS
    assert lib.iabn_group_norm_workspace_size(ref(gn(n=1, hw=2, c=groups, groups=groups))) == 0


# ---------------------------------------------------------------------------
# the binding, before it looks for a GPU

def z(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


def test_binding_refuses_attention():
    spec = iabn.AttentionSpec()
    q, k = z(2, 30, 4, 64), z(2, 50, 2, 64)

    def fwd(q=q, k=k, v=k, out=q, **kw):
        return iabn.iabn_attention_forward(spec, q, k, v, out, **kw)

    with pytest.raises(ValueError, match="keys ahead"):
        iabn.AttentionSpec(causal=True, window=(-1, 5))
    with pytest.raises(ValueError, match=r"expected \[batch"):
        fwd(q=z(30, 4, 64))
    with pytest.raises(ValueError, match="k has 3|k 3"):
        fwd(k=z(3, 50, 2, 64))
    with pytest.raises(ValueError, match="no multiple"):
        fwd(k=z(2, 50, 3, 64))
    with pytest.raises(ValueError, match="v is"):
        fwd(v=z(2, 50, 2, 32))
    with pytest.raises(ValueError, match="out is"):
        fwd(out=z(2, 30, 4, 32))
    with pytest.raises(TypeError, match="k is"):
        fwd(k=k.float())
    with pytest.raises(ValueError, match="contiguous"):
        fwd(q=z(2, 30, 64, 4).transpose(2, 3))
    with pytest.raises(ValueError, match="max_q"):
        fwd(q=z(60, 4, 64), out=z(60, 4, 64), q_starts=torch.zeros(3, dtype=torch.int32))
    with pytest.raises(TypeError, match="q_lens"):
        fwd(q_lens=torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError, match="k_lens"):
        fwd(k_lens=torch.zeros(3, dtype=torch.int32))
    with pytest.raises(TypeError, match="storage dtype"):
        fwd(q=q.double(), k=k.double(), v=k.double(), out=q.double())
    with pytest.raises(TypeError, match="lse"):
        fwd(lse=z(2, 4, 30))
    with pytest.raises(TypeError, match="live on the GPU"):
        fwd(out=z(2, 30, 4, 64))
    with pytest.raises(ValueError, match="lse"):
        iabn.iabn_attention_backward(spec, q, k, k, q, None, q, q, k, k, None)


def test_binding_refuses_rotary():
    spec = iabn.RotarySpec(64, (8, 12, 12), device="cpu")
    q, pos = z(2, 30, 4, 64), torch.zeros(2, 30, 3, dtype=torch.int32)
    with pytest.raises(ValueError, match="sections"):
        iabn.RotarySpec(64, (), device="cpu")
    with pytest.raises(ValueError, match="pairs"):
        iabn.RotarySpec(64, (20, 20), device="cpu")
    with pytest.raises(ValueError, match="ramp"):
        iabn.RotarySpec(64, ramp="log", device="cpu")
    with pytest.raises(ValueError, match="heads of 64"):
        iabn.iabn_rotary(spec, pos, z(2, 30, 4, 32), z(2, 30, 4, 32))
    with pytest.raises(ValueError, match="positions are"):
        iabn.iabn_rotary(spec, pos[:, :, :2], q, q)
    with pytest.raises(TypeError, match="positions are"):
        iabn.iabn_rotary(spec, pos.half(), q, q)
    with pytest.raises(ValueError, match="go together"):
        iabn.iabn_rotary(spec, pos, q, q, k=q)
    with pytest.raises(ValueError, match="k is"):
        iabn.iabn_rotary(spec, pos, q, q, z(2, 31, 4, 64), q)
    with pytest.raises(ValueError, match="contiguous"):
        iabn.iabn_rotary(spec, pos.transpose(1, 2).contiguous().transpose(1, 2), q, q)
    with pytest.raises(TypeError, match="live on the GPU"):
        iabn.iabn_rotary(spec, pos, q, q)


def test_rotary_spec_tables():
    """Which axis and which frequency each pair takes."""
    s = iabn.RotarySpec(16, (2, 3, 3), base=100.0, device="cpu")
    assert s.axis.tolist() == [0, 0, 1, 1, 1, 2, 2, 2] and s.axes == 3 and s.pairs == 8
    want = 100.0 ** -(torch.arange(8, dtype=torch.float64) / 8)
    torch.testing.assert_close(s.inv_freq, want, rtol=1e-15, atol=0)
    s = iabn.RotarySpec(16, (2, 3), base=100.0, ramp="axis", device="cpu")
    want = 100.0 ** -torch.tensor([0, 1 / 2, 0, 1 / 3, 2 / 3], dtype=torch.float64)
    torch.testing.assert_close(s.inv_freq, want, rtol=1e-15, atol=0)
    s = iabn.RotarySpec(16, (4, 2, 2), mixed=True, device="cpu")
    assert s.axis.tolist() == [0, 1, 2, 0, 1, 2, 0, 0]
    assert iabn.RotarySpec(16, device="cpu").axis is None


def test_binding_refuses_group_norm():
    x = z(2, 5, 7, 48)
    w, ws = torch.ones(48), torch.empty(1 << 16, dtype=torch.uint8)

    def fwd(x=x, y=x, groups=6, weight=w, bias=w, act="silu", **kw):
        return iabn.iabn_group_norm_forward(x, y, groups, weight, bias, ws, act=act, **kw)

    with pytest.raises(ValueError, match="samples"):
        fwd(x=z(48))
    with pytest.raises(ValueError, match="divide"):
        fwd(groups=5)
    with pytest.raises(ValueError, match="divide"):
        fwd(groups=0)
    with pytest.raises(ValueError, match="act must be"):
        fwd(act="relu6")
    with pytest.raises(TypeError, match="weight"):
        fwd(weight=w.half())
    with pytest.raises(ValueError, match="bias"):
        fwd(bias=torch.ones(47))
    with pytest.raises(ValueError, match="y is"):
        fwd(y=z(2, 5, 7, 40))
    with pytest.raises(TypeError, match="y is"):
        fwd(y=x.float())
    with pytest.raises(ValueError, match="collapse"):
        fwd(x=z(2, 5, 48, 7).transpose(2, 3))
    with pytest.raises(ValueError, match="stats"):
        fwd(stats=torch.empty(2, 5, 2))
    with pytest.raises(TypeError, match="live on the GPU"):
        fwd()


def test_modules_refuse_head_sizes():
    """When they are made, not when they are called (and where no kernel would take them)."""
    from place_batchnorm_activation_amd import attention as A
    for channels, heads in ((512, 1), (48, 4), (160, 1), (24, 8)):
        with pytest.raises(ValueError, match="heads of %d elements" % (channels // heads)):
            A.MapAttention(channels, heads, groups=4, rotary=False)
        with pytest.raises(ValueError, match="heads of %d elements" % (channels // heads)):
            A.ResidualAttention(channels, heads)
    with pytest.raises(ValueError, match="heads of 192 elements"):
        A.ResidualAttention(256, 4, head_dim=192)
    assert A.ResidualAttention(256, 4, head_dim=128).head_dim == 128
    assert A.MapAttention(64, 8, rotary=False).heads == 8
