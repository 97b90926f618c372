"""Attention on the GPU against float64 with derived bounds (heads_ref.py): types, head
counts and sizes, masks, lengths, packed sequences, strides, and gradients."""
import math

import pytest
import torch

iabn = pytest.importorskip("place_batchnorm_activation_amd")
import heads_ref  # noqa: E402

pytestmark = pytest.mark.gpu
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
DT = pytest.mark.parametrize("dtype", (BF16, F16, F32), ids=("bf16", "f16", "f32"))


def make(seed, B, Sq, Sk, H, KV, D, dtype, size=1.0, dsize=1.0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    return [(f * t).to(dtype).cuda() for f, t in (
        (size, r(B, Sq, H, D)), (size, r(B, Sk, KV, D)), (1.0, r(B, Sk, KV, D)),
        (dsize, r(B, Sq, H, D)))]


def lens(v):
    return None if v is None else torch.tensor(v, dtype=torch.int32, device="cuda")


def both(q, k, v, dout, spec, **seq):
    """out, lse, dq, dk, dv of the library; outputs start as NaN."""
    nan = lambda t: torch.full_like(t, math.nan, memory_format=torch.contiguous_format)  # noqa: E731
    out, lse = nan(q), iabn.attention_lse(q).fill_(math.nan)
    iabn.iabn_attention_forward(spec, q, k, v, out, lse, iabn.attention_workspace(spec, q, k, **seq),
                                **seq)
    dq, dk, dv = nan(q), nan(k), nan(v)
    iabn.iabn_attention_backward(spec, q, k, v, out, lse, dout, dq, dk, dv,
                                 iabn.attention_workspace(spec, q, k, backward=True, **seq), **seq)
    return dict(out=out, lse=lse, dq=dq, dk=dk, dv=dv)


def check(got, val, bound):
    for name in got:
        heads_ref.within(got[name], val[name], bound[name], name)


@DT
@pytest.mark.parametrize("D", (8, 32, 40, 64, 72, 96, 104, 128))
def test_head_sizes(dtype, D):
    q, k, v, do = make(D, 2, 75, 141, 4, 2, D, dtype)
    spec = iabn.AttentionSpec(causal=True)
    check(both(q, k, v, do, spec), *heads_ref.attention(q, k, v, do, right=0))


@DT
@pytest.mark.parametrize("Sq,Sk", ((1, 1), (1, 2), (2, 1), (1, 700), (5, 33), (32, 32), (33, 64),
                                   (64, 65), (127, 129), (130, 1), (257, 385)))
@pytest.mark.parametrize("causal", (False, True))
def test_lengths(dtype, Sq, Sk, causal):
    q, k, v, do = make(Sq * 1000 + Sk, 1, Sq, Sk, 3, 3, 64, dtype)
    spec = iabn.AttentionSpec(causal=causal)
    check(both(q, k, v, do, spec), *heads_ref.attention(q, k, v, do, right=0 if causal else -1))


@DT
@pytest.mark.parametrize("H,KV", ((1, 1), (5, 1), (8, 2), (12, 4), (6, 6), (40, 1), (16, 8)))
def test_grouped_heads(dtype, H, KV):
    q, k, v, do = make(H * 100 + KV, 2, 21, 85, H, KV, 64, dtype)
    spec = iabn.AttentionSpec(causal=True)
    check(both(q, k, v, do, spec), *heads_ref.attention(q, k, v, do, right=0))


@DT
@pytest.mark.parametrize("left,right", ((0, 0), (7, -1), (-1, 9), (31, 0), (64, 64), (200, 3),
                                        (0, 5)))
@pytest.mark.parametrize("Sq,Sk", ((150, 150), (190, 100), (60, 210)))
def test_windows(dtype, left, right, Sq, Sk):
    """Rows that see no key (more queries than keys) among them."""
    q, k, v, do = make(left * 300 + right, 1, Sq, Sk, 4, 2, 40, dtype)
    spec = iabn.AttentionSpec(window=(left, right))
    got = both(q, k, v, do, spec)
    check(got, *heads_ref.attention(q, k, v, do, left=left, right=right))
    see = heads_ref.visible(Sq, Sk, left, right)
    blind = ~see.any(1).cuda()
    assert (got["out"][0][blind] == 0).all() and (got["dq"][0][blind] == 0).all()
    assert (got["lse"][0][:, blind] == -math.inf).all()
    unseen = ~see.any(0).cuda()
    assert (got["dk"][0][unseen] == 0).all() and (got["dv"][0][unseen] == 0).all()


@DT
@pytest.mark.parametrize("causal", (False, True))
def test_padded_batch(dtype, causal):
    """Lengths of zero, one and all; what lies behind a length is not read (NaN) and what
    belongs to it is written as zeros."""
    ql, kl = [0, 1, 70, 33, 130, 130, 7], [50, 0, 90, 1, 200, 130, 7]
    q, k, v, do = make(5, 7, 130, 200, 4, 2, 64, dtype)
    for b in range(7):
        for t in (q, do):
            t[b, ql[b]:] = math.nan
        for t in (k, v):
            t[b, kl[b]:] = math.nan
    spec = iabn.AttentionSpec(causal=causal)
    got = both(q, k, v, do, spec, q_lens=lens(ql), k_lens=lens(kl))
    check(got, *heads_ref.attention(q, k, v, do, right=0 if causal else -1, q_lens=ql, k_lens=kl))


def pack(t, ls, rows):
    """Sequences one behind another, and `rows` in all, the rest NaN."""
    out = torch.full((rows,) + t.shape[2:], math.nan, dtype=t.dtype, device=t.device)
    at = 0
    for b, n in enumerate(ls):
        out[at:at + n] = t[b, :n]
        at += n
    return out


def unpack(t, ls, most, fill=0.0):
    out = torch.full((len(ls), most) + t.shape[1:], fill, dtype=t.dtype, device=t.device)
    at = 0
    for b, n in enumerate(ls):
        out[b, :n] = t[at:at + n]
        at += n
    return out


def starts(ls):
    return lens([sum(ls[:i]) for i in range(len(ls) + 1)])


@DT
@pytest.mark.parametrize("H,KV", ((4, 2), (3, 3)))
def test_packed(dtype, H, KV):
    """Sequences one behind another, empty ones among them; rows behind the last stay."""
    ls = [17, 0, 1, 140, 64, 0, 33]
    q, k, v, do = make(9, len(ls), 140, 140, H, KV, 72, dtype)
    rows = sum(ls) + 5
    p = [pack(t, ls, rows) for t in (q, k, v, do)]
    seq = dict(q_starts=starts(ls), k_starts=starts(ls), max_q=140, max_k=140)
    got = both(*p, iabn.AttentionSpec(causal=True), **seq)
    for name in ("out", "dq", "dk", "dv"):
        assert got[name][sum(ls):].isnan().all() and not got[name][:sum(ls)].isnan().any()
    assert got["lse"][:, sum(ls):].isnan().all()
    un = {n: unpack(t, ls, 140) for n, t in got.items() if n != "lse"}
    un["lse"] = unpack(got["lse"].t().contiguous(), ls, 140, -math.inf).transpose(1, 2)
    check(un, *heads_ref.attention(q, k, v, do, right=0, q_lens=ls, k_lens=ls))


@DT
def test_packed_queries_over_padded_keys(dtype):
    """New tokens packed, caches padded: each side its own way."""
    ql, kl = [1, 5, 0, 2], [300, 77, 10, 513]
    q, k, v, do = make(11, 4, 5, 520, 8, 2, 128, dtype)
    rows = sum(ql)
    seq = dict(q_starts=starts(ql), max_q=5, k_lens=lens(kl))
    got = both(pack(q, ql, rows), k, v, pack(do, ql, rows), iabn.AttentionSpec(causal=True), **seq)
    got = dict(got, **{n: unpack(got[n], ql, 5) for n in ("out", "dq")},
               lse=unpack(got["lse"].t().contiguous(), ql, 5, -math.inf).transpose(1, 2))
    check(got, *heads_ref.attention(q, k, v, do, right=0, q_lens=ql, k_lens=kl))


@DT
def test_starts_and_lengths_outside_the_tensors(dtype):
    """Device values that no host check sees: cut to the tensors."""
    q, k, v, do = make(12, 2, 20, 40, 2, 2, 64, dtype)
    spec = iabn.AttentionSpec()
    got = both(q, k, v, do, spec, q_lens=lens([999, -5]), k_lens=lens([1 << 30, 40]))
    check(got, *heads_ref.attention(q, k, v, do, q_lens=[20, 0], k_lens=[40, 40]))
    p = [t.flatten(0, 1) for t in (q, k, v, do)]
    seq = dict(q_starts=lens([-7, 20, 90]), k_starts=lens([0, 40, 1 << 30]), max_q=20, max_k=40)
    got = both(*p, spec, **seq)
    # sequence 0: rows 0 .. 20 of -7 .. 20, cut to 20; sequence 1: all that is left
    got = {n: t.view(2, -1, *t.shape[1:]) for n, t in got.items() if n != "lse"}
    val, bound = heads_ref.attention(q, k, v, do)
    check(got, val, bound)


@DT
def test_one_token_over_a_long_cache(dtype):
    """The keys cut among workgroups: every length of a batch, one of them short."""
    kl = [4096, 1, 257, 0, 3001]
    q, k, v, _ = make(13, 5, 1, 4096, 8, 2, 128, dtype)
    for b, n in enumerate(kl):
        k[b, n:] = math.nan
        v[b, n:] = math.nan
    spec = iabn.AttentionSpec(causal=True)
    seq = dict(k_lens=lens(kl))
    assert iabn.iabn_attention_workspace_size(spec, q, k, **seq) > 0
    out, lse = torch.full_like(q, math.nan), iabn.attention_lse(q).fill_(math.nan)
    iabn.iabn_attention_forward(spec, q, k, v, out, lse,
                                iabn.attention_workspace(spec, q, k, **seq), **seq)
    val, bound = heads_ref.attention(q, k, v, right=0, k_lens=kl)
    check(dict(out=out, lse=lse), val, bound)


@DT
def test_a_very_long_cache(dtype):
    """Hundreds of parts, and a window that leaves all but the last few of them nothing."""
    q, k, v, _ = make(30, 1, 2, 150001, 2, 1, 64, dtype)
    for left in (-1, 700):
        spec = iabn.AttentionSpec(window=(left, 0))
        out, lse = torch.full_like(q, math.nan), iabn.attention_lse(q).fill_(math.nan)
        iabn.iabn_attention_forward(spec, q, k, v, out, lse, iabn.attention_workspace(spec, q, k))
        val, bound = heads_ref.attention(q, k, v, left=left, right=0)
        check(dict(out=out, lse=lse), val, bound)


@DT
@pytest.mark.parametrize("B,Sq,Sk,H,KV,D", ((32, 1, 900, 16, 8, 128), (70, 2, 300, 8, 8, 64),
                                            (66, 1, 1030, 16, 8, 40), (40, 1, 800, 16, 8, 96)))
def test_many_caches(dtype, B, Sq, Sk, H, KV, D):
    """One or two tokens for each of many caches: as many key heads as CUs, and more."""
    q, k, v, _ = make(37, B, Sq, Sk, H, KV, D, dtype)
    spec = iabn.AttentionSpec(causal=True)
    out, lse = torch.full_like(q, math.nan), iabn.attention_lse(q).fill_(math.nan)
    iabn.iabn_attention_forward(spec, q, k, v, out, lse, iabn.attention_workspace(spec, q, k))
    val, bound = heads_ref.attention(q, k, v, right=0)
    check(dict(out=out, lse=lse), val, bound)


@DT
@pytest.mark.parametrize("left,right", ((-1, 0), (40, 0), (3, 300)))
@pytest.mark.parametrize("D", (24, 64, 104))
def test_few_rows_over_short_keys(dtype, left, right, D):
    """Waves of one workgroup that part the keys: lengths of zero, one and all, windows that
    leave some waves, and some rows, nothing, and what lies behind a length."""
    ql, kl = [5, 0, 3, 5, 1, 5], [700, 33, 0, 1, 512, 3]
    q, k, v, _ = make(38, 6, 5, 700, 6, 2, D, dtype)
    for b in range(6):
        q[b, ql[b]:] = math.nan
        k[b, kl[b]:] = v[b, kl[b]:] = math.nan
    spec = iabn.AttentionSpec(window=(left, right))
    seq = dict(q_lens=lens(ql), k_lens=lens(kl))
    out, lse = torch.full_like(q, math.nan), iabn.attention_lse(q).fill_(math.nan)
    iabn.iabn_attention_forward(spec, q, k, v, out, lse,
                                iabn.attention_workspace(spec, q, k, **seq), **seq)
    val, bound = heads_ref.attention(q, k, v, left=left, right=right, q_lens=ql, k_lens=kl)
    check(dict(out=out, lse=lse), val, bound)


@DT
@pytest.mark.parametrize("padded", (False, True))
@pytest.mark.parametrize("Sq,left,right", ((1, 2000, 0), (6, 1500, 40), (300, 900, 130)))
def test_windows_over_long_keys(dtype, Sq, left, right, padded):
    """Parts of what a window shows: few rows and many, sequences of their own lengths."""
    ql, kl = [Sq, max(1, Sq // 2), Sq], [5000, 3100, 77]
    q, k, v, _ = make(39, 3, Sq, 5000, 4, 2, 72, dtype)
    seq, know = {}, {}
    if padded:
        seq, know = dict(q_lens=lens(ql), k_lens=lens(kl)), dict(q_lens=ql, k_lens=kl)
    spec = iabn.AttentionSpec(window=(left, right))
    out, lse = torch.full_like(q, math.nan), iabn.attention_lse(q).fill_(math.nan)
    iabn.iabn_attention_forward(spec, q, k, v, out, lse,
                                iabn.attention_workspace(spec, q, k, **seq), **seq)
    val, bound = heads_ref.attention(q, k, v, left=left, right=right, **know)
    check(dict(out=out, lse=lse), val, bound)


@DT
@pytest.mark.parametrize("Sq,Sk,H,KV", ((24, 9000, 4, 1), (3000, 40, 8, 2), (1500, 1500, 2, 1)))
def test_parted_gradients(dtype, Sq, Sk, H, KV):
    """Few row tiles over many keys, few key tiles under many rows: shares that are joined."""
    q, k, v, do = make(31, 1, Sq, Sk, H, KV, 64, dtype)
    for right in (-1, 0):
        spec = iabn.AttentionSpec(causal=right == 0)
        check(both(q, k, v, do, spec), *heads_ref.attention(q, k, v, do, right=right))


@DT
@pytest.mark.parametrize("left,right,H,KV", ((300, 20, 2, 1), (700, 0, 5, 1), (0, 400, 2, 2)))
def test_parted_gradients_under_windows(dtype, left, right, H, KV):
    """Parts of what a window shows of long sequences, the queries behind the keys and before."""
    for Sq, Sk in ((1900, 2200), (2100, 1500)):
        q, k, v, do = make(40, 1, Sq, Sk, H, KV, 40, dtype)
        spec = iabn.AttentionSpec(window=(left, right))
        check(both(q, k, v, do, spec), *heads_ref.attention(q, k, v, do, left=left, right=right))


@DT
def test_parted_padded_batch(dtype):
    """Joined shares under lengths: tiles that end inside a length, padded keys and rows."""
    ql, kl = [1400, 77, 0, 900], [1400, 500, 300, 0]
    q, k, v, do = make(32, 4, 1400, 1400, 2, 1, 40, dtype)
    for b in range(4):
        q[b, ql[b]:] = do[b, ql[b]:] = math.nan
        k[b, kl[b]:] = v[b, kl[b]:] = math.nan
    spec = iabn.AttentionSpec(window=(600, 100))
    got = both(q, k, v, do, spec, q_lens=lens(ql), k_lens=lens(kl))
    check(got, *heads_ref.attention(q, k, v, do, left=600, right=100, q_lens=ql, k_lens=kl))


@DT
@pytest.mark.parametrize("H,KV,D", ((3, 1, 128), (10, 2, 64), (40, 1, 40)))
def test_odd_groups_at_length(dtype, H, KV, D):
    """Groups that divide no pass of a tile, over many tiles."""
    q, k, v, do = make(33 + H, 1, 420, 640, H, KV, D, dtype)
    spec = iabn.AttentionSpec(causal=True)
    check(both(q, k, v, do, spec), *heads_ref.attention(q, k, v, do, right=0))


@DT
@pytest.mark.parametrize("shift", (1, 4))
def test_unaligned_at_length(dtype, shift):
    """Rows at no multiple of 16 bytes, over many tiles."""
    B, S, H, KV, D = 2, 500, 4, 2, 64
    wide = torch.randn(B, S, (H + 2 * KV) * D + shift, generator=torch.Generator().manual_seed(34))
    wide = wide.to(dtype).cuda()
    q, k, v = (t.unflatten(-1, (-1, D)) for t in
               wide[..., shift:].split((H * D, KV * D, KV * D), -1))
    do = make(35, B, S, S, H, KV, D, dtype)[3]
    spec = iabn.AttentionSpec()
    check(both(q, k, v, do, spec), *heads_ref.attention(q, k, v, do))


@DT
def test_packed_and_parted(dtype):
    """Long and short packed sequences whose gradients are made in shares."""
    ls, D = [1500, 0, 3, 800], 96
    q, k, v, do = make(36, 4, 1500, 1500, 2, 1, D, dtype)
    starts = lens([0, 1500, 1500, 1503, 2303])
    flat = [torch.cat([t[b, :n] for b, n in enumerate(ls)]) for t in (q, k, v, do)]
    spec = iabn.AttentionSpec(causal=True)
    got = both(*flat, spec, q_starts=starts, k_starts=starts, max_q=1500, max_k=1500)
    val, bound = heads_ref.attention(q, k, v, do, right=0, q_lens=ls, k_lens=ls)
    for name in ("out", "dq", "dk", "dv"):
        join = lambda t: torch.cat([t[b, :n] for b, n in enumerate(ls)])  # noqa: E731
        heads_ref.within(got[name], join(val[name]), join(bound[name]), name)


@DT
@pytest.mark.parametrize("Sq", (3, 40, 300))
def test_cut_keys_with_several_tokens(dtype, Sq):
    q, k, v, _ = make(14, 1, Sq, 2000, 4, 2, 96, dtype)
    spec = iabn.AttentionSpec(causal=True)
    ws = iabn.attention_workspace(spec, q, k)
    assert ws is not None
    out, lse = torch.full_like(q, math.nan), iabn.attention_lse(q).fill_(math.nan)
    iabn.iabn_attention_forward(spec, q, k, v, out, lse, ws)
    val, bound = heads_ref.attention(q, k, v, right=0)
    check(dict(out=out, lse=lse), val, bound)


@DT
def test_strides(dtype):
    """Slices of one projection (unaligned too), heads before rows, transposed gradients."""
    B, S, H, KV, D = 2, 70, 4, 2, 40
    g = torch.Generator().manual_seed(15)
    qkv = torch.randn(B, S, (H + 2 * KV) * D + 3, generator=g).to(dtype).cuda()[..., 3:]
    qkv = qkv.unflatten(-1, (H + 2 * KV, D))
    q, k, v = qkv.split((H, KV, KV), 2)
    do = torch.randn(B, H, S, D, generator=g).to(dtype).cuda().transpose(1, 2)
    spec = iabn.AttentionSpec(causal=True)
    val, bound = heads_ref.attention(q, k, v, do, right=0)
    out = torch.full((B, H, S, D), math.nan, dtype=dtype, device="cuda").transpose(1, 2)
    lse = iabn.attention_lse(q)
    iabn.iabn_attention_forward(spec, q, k, v, out, lse, iabn.attention_workspace(spec, q, k))
    grads = torch.full((B, S, (H + 2 * KV) * D + 1), math.nan, dtype=dtype, device="cuda")
    dq, dk, dv = grads[..., 1:].unflatten(-1, (H + 2 * KV, D)).split((H, KV, KV), 2)
    iabn.iabn_attention_backward(spec, q, k, v, out, lse, do, dq, dk, dv,
                                 iabn.attention_workspace(spec, q, k, backward=True))
    check(dict(out=out, lse=lse, dq=dq, dk=dk, dv=dv), val, bound)
    assert grads[..., 0].isnan().all()


@DT
def test_expanded_keys(dtype):
    """Keys and values shared by the batch, as a view without memory of its own."""
    q, k, v, do = make(16, 3, 50, 60, 2, 1, 64, dtype)
    k, v = k[:1].expand_as(k), v[:1].expand_as(v)
    got = both(q, k, v, do, iabn.AttentionSpec())
    check(got, *heads_ref.attention(q, k, v, do))


@DT
@pytest.mark.parametrize("Sq,Sk", ((0, 5), (5, 0), (0, 0)))
def test_no_rows_or_keys(dtype, Sq, Sk):
    q, k, v, do = make(17, 2, Sq, Sk, 4, 2, 64, dtype)
    got = both(q, k, v, do, iabn.AttentionSpec())
    assert all((t == 0).all() for n, t in got.items() if n != "lse")
    assert (got["lse"] == -math.inf).all()


@DT
@pytest.mark.parametrize("size,dsize", ((4.0, 1.0), (1.0, 1e-4), (0.02, 3.0)))
def test_sizes_of_values(dtype, size, dsize):
    """Scores of large spread; gradients near float16's smallest numbers; flat softmax."""
    q, k, v, do = make(18, 1, 160, 300, 2, 1, 64, dtype, size, dsize)
    got = both(q, k, v, do, iabn.AttentionSpec())
    check(got, *heads_ref.attention(q, k, v, do))


@DT
def test_growing_scores(dtype):
    """Each tile's scores above the last's: the running maximum moves with every tile, and in
    float16 the factor of dS too."""
    q, k, v, do = make(19, 1, 64, 1024, 2, 2, 64, dtype)
    k *= torch.linspace(0.05, 3.0, 1024, device="cuda")[None, :, None, None].to(dtype)
    v *= torch.linspace(0.01, 4.0, 1024, device="cuda")[None, :, None, None].to(dtype)
    got = both(q, k, v, do, iabn.AttentionSpec(scale=0.5))
    check(got, *heads_ref.attention(q, k, v, do, scale=0.5))


def test_scale():
    q, k, v, do = make(20, 1, 40, 40, 2, 2, 64, F32)
    got = both(q, k, v, do, iabn.AttentionSpec(scale=0.9))
    check(got, *heads_ref.attention(q, k, v, do, scale=0.9))


@DT
def test_nan_in_a_seen_key_reaches_its_row(dtype):
    q, k, v, do = make(21, 1, 4, 50, 1, 1, 64, dtype)
    q[0, 2] = math.nan
    out = torch.empty_like(q)
    spec = iabn.AttentionSpec()
    iabn.iabn_attention_forward(spec, q, k, v, out, None, iabn.attention_workspace(spec, q, k))
    assert out[0, 2].isnan().all() and not out[0, [0, 1, 3]].isnan().any()


@DT
def test_same_bits_every_time(dtype):
    q, k, v, do = make(22, 2, 200, 333, 8, 2, 128, dtype)
    spec = iabn.AttentionSpec(causal=True)
    a, b = both(q, k, v, do, spec), both(q, k, v, do, spec)
    for n in a:
        assert torch.equal(a[n], b[n]), n


def test_gradients_against_differences():
    """d/dt of sum(w * out(x + t u)) by central differences of the float32 forward, against the
    gradient's product with u.  The difference with step h is off by h^2/6 of the third
    derivative (|scale u| = O(1): a few units) and by the forward's rounding, 2^-24 sqrt(n) |w out| / h
    over n independent terms; with h = 2^-6 and n = 2 x 40 x 2 x 64 both stay below 1e-3 of
    |w out| = sqrt(n)."""
    g = torch.Generator().manual_seed(23)
    q, k, v, w = make(24, 1, 40, 56, 2, 1, 64, F32)
    spec = iabn.AttentionSpec(causal=True)

    def value(q, k, v):
        out = torch.empty_like(q)
        iabn.iabn_attention_forward(spec, q, k, v, out, None, iabn.attention_workspace(spec, q, k))
        return float((out.double() * w.double()).sum())

    got = both(q, k, v, w, spec)
    n = w.numel()
    for i, name in enumerate(("dq", "dk", "dv")):
        x = [q, k, v]
        u = torch.randn(x[i].shape, generator=g).cuda()
        u /= u.norm()
        h = 2.0 ** -6
        up, down = list(x), list(x)
        up[i], down[i] = x[i] + h * u, x[i] - h * u
        diff = (value(*up) - value(*down)) / (2 * h)
        want = float((got[name].double() * u.double()).sum())
        assert abs(diff - want) <= 1e-3 * math.sqrt(n), (name, diff, want)


def test_long_offsets():
    """A cache past 2^31 elements: rows beyond 32-bit offsets are read where they lie."""
    Sk, KV, D = 1 << 15, 8, 128
    B = 66                                   # 66 * 2^15 * 8 * 128 = 2.2e9 elements
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB")
    kv = torch.zeros(2, B, Sk, KV, D, dtype=BF16, device="cuda")
    q, k, v, _ = make(25, 1, 1, 300, 8, KV, D, BF16)
    b = B - 1
    kv[0, b, :300], kv[1, b, :300] = k[0], v[0]
    n = [1] * B
    n[b] = 300
    spec = iabn.AttentionSpec(causal=True)
    qs = q.expand(B, -1, -1, -1).contiguous()
    out = torch.empty_like(qs)
    seq = dict(k_lens=lens(n))
    iabn.iabn_attention_forward(spec, qs, kv[0], kv[1], out, None,
                                iabn.attention_workspace(spec, qs, kv[0], **seq), **seq)
    val, bound = heads_ref.attention(q, k, v, right=0)
    heads_ref.within(out[b:], val["out"], bound["out"], "out")
    assert (out[:b] == 0).all()


# ---------------------------------------------------------------------------
# one key far above all others, with a value of zero: the small probabilities are the result

def sink(dtype, n, gap, rows=1, heads=1, D=64):
    """q, k, v, dout of one sequence whose first key's score lies `gap` above the others', which are
    equal (exactly: scale 1, one element that counts)."""
    g = torch.Generator().manual_seed(n + int(10 * gap))
    q, k = torch.zeros(1, rows, heads, D), torch.zeros(1, n, heads, D)
    q[..., 0], k[:, 0, :, 0] = 1.0, gap
    v = 1 + 0.25 * torch.randn(1, n, heads, D, generator=g)
    v[:, 0] = 0
    do = torch.randn(1, rows, heads, D, generator=g)
    return [t.to(dtype).cuda() for t in (q, k, v, do)]


GAPS = pytest.mark.parametrize("gap", (12.5, 15.0, 16.5, 17.0, 17.5, 18.0))


@DT
@GAPS
@pytest.mark.parametrize("B,rows,n", ((1, 1, 517), (1, 1, 4096), (1, 1, 32768), (520, 1, 517),
                                      (520, 1, 4096), (520, 1, 32768), (1, 300, 517),
                                      (1, 300, 4096), (1, 300, 32768), (140, 200, 517),
                                      (140, 200, 4096)))
def test_small_probabilities_beside_a_large_one(dtype, gap, n, B, rows):
    """Parts among workgroups, waves of one workgroup (517 keys), and whole rows in one wave or
    four (as many sequences as fill the card, all of the same tensors)."""
    q, k, v, _ = sink(dtype, n, gap, rows)
    val, bound = heads_ref.attention(q, k, v, scale=1.0)
    q, k, v = (t.expand(B, -1, -1, -1) for t in (q, k, v))
    out = torch.full(q.shape, math.nan, dtype=dtype, device="cuda")
    lse = iabn.attention_lse(q).fill_(math.nan)
    spec = iabn.AttentionSpec(scale=1.0)
    iabn.iabn_attention_forward(spec, q, k, v, out, lse, iabn.attention_workspace(spec, q, k))
    for b in (0, B - 1):
        check(dict(out=out[b:b + 1], lse=lse[b:b + 1]), val, bound)
    assert (out == out[:1]).all() and (lse == lse[:1]).all()


@DT
@GAPS
@pytest.mark.parametrize("n", (517, 4096))
def test_gradients_of_small_probabilities(dtype, gap, n):
    """heads_ref's bounds take delta's own out as rounded by u |out|.  Here out is as small as 8e-6,
    among float16's subnormals, whose rounding is off by up to TINY = 2^-25 (u |out| is 4e-9): with
    |delta - exact| up to sum_d |dO| TINY more, dS is off by P times that, and dq and dk by its sums
    with |k| and |q|, doubled as the rest of the bound."""
    q, k, v, do = sink(dtype, n, gap, rows=200, heads=2)
    val, bound = heads_ref.attention(q, k, v, do, scale=1.0)
    q6, k6, do6 = (t[0].transpose(0, 1).double().cpu() for t in (q, k, do))      # [heads, rows, D]
    p = torch.softmax(q6 @ k6.transpose(1, 2), -1)
    off = p * do6.abs().sum(-1, keepdim=True) * 2 * heads_ref.TINY[dtype]
    bound["dq"] += (off @ k6.abs()).transpose(0, 1)
    bound["dk"] += (off.transpose(1, 2) @ q6.abs()).transpose(0, 1)
    check(both(q, k, v, do, iabn.AttentionSpec(scale=1.0)), val, bound)


@DT
@pytest.mark.parametrize("size", (2.0 ** 6, 2.0 ** 10, 2.0 ** 12, 1.1 * 2.0 ** 13))
@pytest.mark.parametrize("rows,n", ((1, 517), (1, 3000), (200, 300)))
def test_equal_scores_of_any_size(dtype, size, rows, n):
    """Scores of 2^12 to 2^26, all the same: whatever the scaled maximum's rounding makes of their
    exponentials (an order or two at 2^26), it is one value P and cancels: out is the values'
    mean, off by P's rounding to the type (u), the sums' (n e each) and its own (u), of sum |v| / n,
    doubled."""
    g = torch.Generator().manual_seed(41)
    q, k = torch.zeros(1, rows, 2, 64), torch.zeros(1, n, 2, 64)
    q[..., 3] = k[..., 3] = size
    v = torch.randn(1, n, 2, 64, generator=g)
    q, k, v = (t.to(dtype).cuda() for t in (q, k, v))
    out = torch.full_like(q, math.nan)
    spec = iabn.AttentionSpec(scale=1.0)
    iabn.iabn_attention_forward(spec, q, k, v, out, None, iabn.attention_workspace(spec, q, k))
    v6 = v.double().cpu()
    bound = 2 * (2 * heads_ref.HALF[dtype] + 2 * n * heads_ref.E) * v6.abs().mean(1, keepdim=True)
    heads_ref.within(out, v6.mean(1, keepdim=True).expand(1, rows, 2, 64),
                     bound.expand(1, rows, 2, 64))


@DT
@pytest.mark.parametrize("gap", (18.5, 18.8, 19.1, 19.4))
def test_value_gradients_of_small_probabilities(dtype, gap):
    """dv of keys far below another one, under gradients of one sign as large as a loss scale makes
    them: P of 2^-27 to
    2^-28 of the row's largest keeps its digits.  The bound is heads_ref's without what it allows
    float16 to lose there: u |dv| + sum P (u + x + m e) |dO|, m rows, doubled."""
    rows, n, D, u, e = 200, 517, 64, heads_ref.HALF[dtype], heads_ref.E
    q, k, v, do = sink(dtype, n, gap, rows)
    do = do.abs() * 256
    dv = both(q, k, v, do, iabn.AttentionSpec(scale=1.0))["dv"]
    q6, k6, do6 = (t[0, :, 0].double().cpu() for t in (q, k, do))
    s = q6 @ k6.T
    p = torch.softmax(s, -1)
    x = 2 * (D + 2) * e * s.abs().amax(1, keepdim=True) + 2.0 ** -22 + n * e
    want = p.T @ do6
    bound = 2 * (u * want.abs() + (p * (u + x + rows * e)).T @ do6.abs() + heads_ref.TINY[dtype])
    heads_ref.within(dv[0, :, 0], want, bound, "dv")
