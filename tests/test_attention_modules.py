"""The modules of attention.py and groupnorm.py on the GPU against float64, and runs of the
operators together: a block's forward and backward, generation through a cache, captured
graphs, other streams.

Bounds: the float32 operators by heads_ref.py's; whole blocks in float32, whose norm and
weight gradients read 8-bit codes, by the codes' rounding (tests/test_residual.py: 5% in the
2-norm for gradients; outputs do not see the codes: 1e-4 of their largest, for sums of up to
a thousand products of a few layers, each off by 2^-24 of its terms' sizes)."""
import importlib.util
import math
import os

import pytest
import torch

iabn = pytest.importorskip("place_batchnorm_activation_amd")
import heads_ref  # noqa: E402

pytestmark = pytest.mark.gpu
if torch.cuda.is_available():
    from place_batchnorm_activation_amd import attention as A
    from place_batchnorm_activation_amd.groupnorm import GroupNormAct
    from place_batchnorm_activation_amd.residual import ResidualMLP

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
DT = pytest.mark.parametrize("dtype", (BF16, F16, F32), ids=("bf16", "f16", "f32"))


def rnd(seed, *shape, dtype=F32):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


def off(got, want):
    want = want.detach().double().cpu()
    return float((got.detach().double().cpu() - want).norm() / (want.norm() + 1e-300))


# ---------------------------------------------------------------------------
# attention and rotary with autograd

@DT
def test_attention_function(dtype):
    q, k, v = (rnd(i, 2, 70, h, 64, dtype=dtype).requires_grad_() for i, h in ((1, 4), (2, 2), (3, 2)))
    w = rnd(4, 2, 70, 4, 64, dtype=dtype)
    out = A.attention(q, k, v, causal=True)
    out.backward(w)
    val, bound = heads_ref.attention(q, k, v, w, right=0)
    for got, name in ((out, "out"), (q.grad, "dq"), (k.grad, "dk"), (v.grad, "dv")):
        heads_ref.within(got, val[name], bound[name], name)


def test_attention_of_any_layout_and_gradient():
    """Heads before rows, a gradient without memory of its own, inputs without gradients."""
    q, k, v = (rnd(i, 2, 3, 40, 32).transpose(1, 2) for i in (5, 6, 7))
    k.requires_grad_()
    out = A.attention(q, k, v)
    out.sum().backward()
    val, bound = heads_ref.attention(q, k, v, torch.ones(2, 40, 3, 32))
    heads_ref.within(out, val["out"], bound["out"])
    heads_ref.within(k.grad, val["dk"], bound["dk"])
    t = rnd(8, 2, 40, 32, 3).transpose(2, 3)             # head elements apart
    torch.testing.assert_close(A.attention(t, k, v), A.attention(t.contiguous(), k, v), rtol=0,
                               atol=0)


def test_attention_types():
    q, k, v = rnd(9, 1, 20, 2, 64), rnd(10, 1, 20, 2, 64, dtype=BF16), rnd(11, 1, 20, 2, 64)
    assert A.attention(q, k, v).dtype == F32
    with torch.autocast("cuda", dtype=BF16):
        assert A.attention(q, k, v).dtype == BF16


def test_packed_rows_behind_the_last_are_zeros():
    q = rnd(12, 30, 2, 64).requires_grad_()
    s = torch.tensor([0, 10, 25], dtype=torch.int32, device="cuda")
    out = A.attention(q, q, q, causal=True, q_starts=s, k_starts=s, max_q=15, max_k=15)
    out.sum().backward()
    assert (out[25:] == 0).all() and (q.grad[25:] == 0).all() and not q.grad[:25].isnan().any()


@pytest.mark.parametrize("interleaved", (False, True))
def test_rotary_function(interleaved):
    spec = iabn.RotarySpec(64, (10, 11, 11), interleaved=interleaved)
    pos = torch.randint(0, 90, (2, 25, 3), dtype=torch.int32, device="cuda")
    q, k = rnd(13, 2, 25, 4, 64).requires_grad_(), rnd(14, 2, 25, 2, 64).requires_grad_()
    wq, wk = rnd(15, 2, 25, 4, 64), rnd(16, 2, 25, 2, 64)
    qo, ko = A.rotary(spec, pos, q, k)
    torch.autograd.backward((qo, ko), (wq, wk))
    for got, t, inverse in ((qo, q, False), (ko, k, False), (q.grad, wq, True), (k.grad, wk, True)):
        val, bound = heads_ref.rotary(t, pos, spec.inv_freq, spec.axis, interleaved, inverse)
        heads_ref.within(got, val, bound)
    assert torch.equal(A.rotary(spec, pos, q), qo)


# ---------------------------------------------------------------------------
# blocks

def turned64(t, spec, pos):
    n = spec.pairs
    axis = torch.zeros(n, dtype=torch.long) if spec.axis is None else spec.axis.long().cpu()
    angle = pos.double().cpu()[..., axis] * spec.inv_freq.cpu()
    co, si = angle.cos()[..., None, :], angle.sin()[..., None, :]
    a, b = t[..., :n], t[..., n:2 * n]
    return torch.cat((a * co - b * si, b * co + a * si, t[..., 2 * n:]), -1)


def attend64(q, k, v, see):
    G = q.shape[-2] // k.shape[-2]
    q, k, v = (t.transpose(-2, -3) for t in (q, k.repeat_interleave(G, -2),
                                             v.repeat_interleave(G, -2)))
    s = (q @ k.transpose(-1, -2)) * q.shape[-1] ** -0.5
    p = torch.softmax(s.masked_fill(~see, -math.inf), -1)
    return (p @ v).transpose(-2, -3)


def block64(block, r, b, pos, leaves):
    """The block in float64 on leaves (float64 copies of its parameters)."""
    def rms(x, w):
        return x / torch.sqrt(x.square().mean(-1, keepdim=True) + block.norm.eps) * w

    if b is not None:
        r = r + block.norm.alpha * rms(b, leaves["norm.post_weight"])
    n = rms(r, leaves["norm.pre_weight"])
    H, KV, D = block.heads, block.kv_heads, block.head_dim
    qkv = (n @ leaves["qkv.weight"].T).unflatten(-1, (H + 2 * KV, D))
    q, k, v = qkv.split((H, KV, KV), -2)
    q, k = turned64(q, block.rotary, pos), turned64(k, block.rotary, pos)
    S = r.shape[1]
    a = attend64(q, k, v, torch.ones(S, S, dtype=torch.bool).tril())
    return r, a.flatten(-2) @ leaves["out.weight"].T


def make_block(cols=96, heads=4, kv=2, sections=None, **kw):
    torch.manual_seed(3)
    turn = iabn.RotarySpec(cols // heads, sections)
    block = A.ResidualAttention(cols, heads, kv, rotary=turn, alpha=0.8, device="cuda", **kw)
    with torch.no_grad():
        for p in (block.norm.post_weight, block.norm.pre_weight):
            p.add_(0.2 * torch.randn_like(p))
    return block


def test_residual_attention():
    block = make_block()
    r, b = rnd(20, 2, 50, 96).requires_grad_(), rnd(21, 2, 50, 96).requires_grad_()
    wr, wb = rnd(22, 2, 50, 96), rnd(23, 2, 50, 96)
    ro, bo = block(r, b)
    torch.autograd.backward((ro, bo), (wr, wb))
    leaf = lambda t: t.detach().double().cpu().requires_grad_()  # noqa: E731
    leaves = {n: leaf(p) for n, p in block.named_parameters()}
    r6, b6 = leaf(r), leaf(b)
    pos = torch.arange(50)[None, :, None].expand(2, 50, 1)
    ro6, bo6 = block64(block, r6, b6, pos, leaves)
    torch.autograd.backward((ro6, bo6), (wr.double().cpu(), wb.double().cpu()))
    for got, want in ((ro, ro6), (bo, bo6)):
        assert float((got.double().cpu() - want).detach().abs().max()) <= \
            1e-4 * float(want.detach().abs().max())
    assert off(r.grad, r6.grad) < 0.05 and off(b.grad, b6.grad) < 0.05
    for n, p in block.named_parameters():
        assert off(p.grad, leaves[n].grad) < 0.05, n
    # the path that no code enters: the output projection reads the attention's own output
    assert off(block.out.weight.grad, leaves["out.weight"].grad) < 1e-4


def plainly(block, x, keeps):
    """The block's branch with its projection through `keeps`, by operations that turn nothing
    in place."""
    _, n, kept = block.norm(x)
    H, KV = block.heads, block.kv_heads
    qkv = keeps(block.qkv(n, kept)).unflatten(-1, (H + 2 * KV, block.head_dim))
    q, k, v = qkv.split((H, KV, KV), -2)
    pos = torch.arange(x.shape[1], dtype=torch.int32, device="cuda")
    return block.out(A.attention(*A.rotary(block.rotary, pos, q, k), v, causal=True).flatten(-2))


@pytest.mark.parametrize("everywhere", (False, True))
def test_hooks_that_keep_the_projection(everywhere):
    """A hook may record the projection, or replace it by an operation that keeps its result for
    its own backward: neither finds it turned.  (The same kernels on the same values, in one
    buffer or three: sums in one order, 2^-20 for torch's own products.)"""
    block, x, g = make_block(), rnd(34, 2, 30, 96).requires_grad_(), rnd(35, 2, 30, 96)
    with torch.no_grad():
        want = block.qkv(block.norm(x)[1])
    seen = []

    def hook(layer, args, out):
        if layer is not block.qkv:
            return None
        seen.append(out.detach())
        return out.tanh()

    def grads(out):
        out.backward(g)
        got = [x.grad] + [p.grad for p in (block.qkv.weight, block.out.weight)]
        x.grad = None
        block.zero_grad()
        return [out, *got]

    handle = torch.nn.modules.module.register_module_forward_hook(hook) if everywhere else \
        block.qkv.register_forward_hook(hook)
    try:
        got = grads(block(x)[1])
        with torch.no_grad():
            block(x, cache=A.KVCache(2, 30, 2, 24, F32))
    finally:
        handle.remove()
    for t in seen:
        assert off(t, want) < 2.0 ** -20
    assert len(seen) == 2
    for a, b in zip(got, grads(plainly(block, x, torch.tanh))):
        assert off(a, b) < 2.0 ** -20


def test_a_hook_that_keeps_a_maps_projection():
    torch.manual_seed(7)
    m, x = A.MapAttention(48, 2, groups=4, device="cuda"), rnd(36, 2, 48, 6, 5)
    seen = []
    with m.qkv.register_forward_hook(lambda layer, args, out: seen.append(out)):
        want = m(x)
    assert off(seen[0], m.qkv(m.norm(x).movedim(1, -1).flatten(1, -2))) < 2.0 ** -20
    assert off(m(x), want) < 2.0 ** -20


def test_a_kept_projection_is_refused():
    """Turned in place behind an operation that keeps its result, or over a leaf."""
    turn = iabn.RotarySpec(24)
    pos = torch.arange(9, dtype=torch.int32, device="cuda")
    x = rnd(37, 1, 9, 8, 24).requires_grad_()
    apply = lambda t: A.QKVAttentionFunction.apply(t, pos, 4, 2, turn, iabn.AttentionSpec(),  # noqa: E731
                                                   {})
    with pytest.raises(RuntimeError, match="inplace operation"):
        apply(x.tanh()).sum().backward()
    before = x.detach().clone()
    with pytest.raises(RuntimeError, match="leaf"):
        apply(x)
    assert torch.equal(x, before)
    out = apply(x * 1)                             # an intermediate, twice through its graph
    out.sum().backward(retain_graph=True)
    once = x.grad.clone()
    out.sum().backward()
    assert torch.equal(x.grad, 2 * once)


def test_packed_equals_padded():
    block = make_block(sections=(5, 7))
    ls = [13, 30, 1]
    x = rnd(24, 3, 30, 96)
    pos = torch.randint(0, 60, (3, 30, 2), dtype=torch.int32, device="cuda")
    lens = torch.tensor(ls, dtype=torch.int32, device="cuda")
    _, want = block(x, positions=pos, lens=lens)
    starts = torch.tensor([0, 13, 43, 44], dtype=torch.int32, device="cuda")
    rows = torch.cat([x[i, :n] for i, n in enumerate(ls)])
    p = torch.cat([pos[i, :n] for i, n in enumerate(ls)])
    _, got = block(rows, positions=p, starts=starts, max_len=30)
    # the same rows in other tiles: float32 sums in another order
    for i, n in enumerate(ls):
        torch.testing.assert_close(got[starts[i]:starts[i + 1]], want[i, :n], rtol=1e-4, atol=1e-4)
        assert (want[i, n:] == 0).all()


@pytest.mark.parametrize("chunk", (1, 7))
def test_generation_through_a_cache(chunk):
    """Rows a few at a time over the cache give what they give together."""
    block, mlp = make_block(), None
    torch.manual_seed(4)
    mlp = ResidualMLP(96, 128, device="cuda")
    x = rnd(25, 2, 21, 96)
    with torch.no_grad():
        want = mlp(*block(x))[1]
        cache = A.KVCache(2, 40, 2, 24, F32)
        got = torch.cat([mlp(*block(x[:, i:i + chunk], cache=cache))[1]
                         for i in range(0, 21, chunk)], 1)
    assert cache.lens.tolist() == [21, 21] and cache.used == 21
    assert float((got - want).abs().max()) <= 1e-4 * float(want.abs().max())


def test_cache_of_sequences_of_their_own_length():
    block = make_block()
    ls = [5, 9]
    x, y = rnd(26, 2, 9, 96), rnd(27, 2, 1, 96)
    with torch.no_grad():
        cache = A.KVCache(2, 16, 2, 24, F32)
        block(x, cache=cache, lens=torch.tensor(ls, dtype=torch.int32, device="cuda"))
        assert cache.lens.tolist() == ls
        got = block(y, cache=cache)[1]
        for i, n in enumerate(ls):
            whole = torch.cat((x[i:i + 1, :n], y[i:i + 1]), 1)
            want = block(whole)[1][:, -1:]
            assert float((got[i:i + 1] - want).abs().max()) <= 1e-4 * float(want.abs().max())


def test_cache_refuses():
    cache = A.KVCache(1, 4, 2, 8, F32)
    k = rnd(28, 1, 3, 2, 8)
    cache.append(k, k)
    with pytest.raises(ValueError, match="do not fit"):
        cache.append(k, k)
    with pytest.raises(ValueError, match="expected"):
        cache.append(k[:, :1, :1], k[:, :1, :1])
    block = make_block()
    with pytest.raises(RuntimeError, match="no_grad"):
        block(rnd(29, 1, 1, 96), cache=A.KVCache(1, 4, 2, 24, F32))
    with torch.no_grad(), pytest.raises(TypeError, match="cache is"):
        block(rnd(29, 1, 1, 96), cache=A.KVCache(1, 4, 2, 24, BF16))
    with pytest.raises(ValueError, match="positions"):
        block(rnd(29, 4, 96), starts=torch.zeros(2, dtype=torch.int32, device="cuda"), max_len=4)
    with pytest.raises(ValueError, match="expected"):
        block(rnd(29, 4, 96))
    with pytest.raises(ValueError, match="no multiple"):
        A.ResidualAttention(96, 4, 3)
    with pytest.raises(ValueError, match="heads of"):
        A.ResidualAttention(96, 4, rotary=iabn.RotarySpec(32))


def test_a_cache_keeps_no_graph():
    """Rows that need a gradient are stored, and nothing of how they were made."""
    cache = A.KVCache(1, 8, 2, 8, BF16)
    k = rnd(38, 1, 3, 2, 8).requires_grad_()
    cache.append(k * 2, k * 3)
    assert not cache.k.requires_grad and not cache.v.requires_grad
    assert torch.equal(cache.k[:, :3], (k.detach() * 2).to(BF16))
    assert torch.equal(cache.v[:, :3], (k.detach() * 3).to(BF16))


def test_a_refused_call_leaves_the_cache_as_it_was():
    """Of another type, with lengths that the attention refuses, with a spec that the library
    does: what the cache counts is what it held, and the call made right then gives what it gives
    on a fresh cache."""
    x, y = rnd(32, 2, 5, 96), rnd(33, 2, 3, 96)
    lens = torch.tensor([2, 3], dtype=torch.int32, device="cuda")

    def state(cache):
        return cache.used, cache.lens.tolist()

    block = make_block()
    with torch.no_grad():
        other = A.KVCache(2, 16, 2, 24, BF16)
        with pytest.raises(TypeError, match="cache is"):
            block(x, cache=other)
        assert state(other) == (0, [0, 0]) and not other.k.any() and not other.v.any()
        cache, fresh = A.KVCache(2, 16, 2, 24, F32), A.KVCache(2, 16, 2, 24, F32)
        block(x, cache=cache), block(x, cache=fresh)
        for bad, error in ((lens.long(), TypeError), (lens.cpu(), (TypeError, RuntimeError)),
                           (lens[:1], ValueError)):
            with pytest.raises(error):
                block(y, cache=cache, lens=bad)
            assert state(cache) == (5, [5, 5]), bad
        right, block.spec = block.spec, iabn.AttentionSpec(scale=-1.0, causal=True)
        with pytest.raises((ValueError, RuntimeError)):
            block(y, cache=cache, lens=lens)
        assert state(cache) == (5, [5, 5])
        block.spec = right
        got, want = (block(y, cache=c, lens=lens)[1] for c in (cache, fresh))
        assert torch.equal(got, want) and state(cache) == state(fresh) == (8, [7, 8])


def test_block_with_16_bit_layers_and_autocast():
    """float32 stream, bf16 layers; and autocast over float32 ones: against the float32 block to
    the rounding of a few bf16 layers (2^-8 each of five: 2% in the 2-norm)."""
    block = make_block()
    x = rnd(30, 2, 33, 96).requires_grad_()
    _, want = block(x)
    g = rnd(31, 2, 33, 96)
    want.backward(g)
    gw, gx = block.qkv.weight.grad.clone(), x.grad.clone()
    block.zero_grad(), setattr(x, "grad", None)
    with torch.autocast("cuda", dtype=BF16):
        _, got = block(x)
    assert off(got, want) < 0.02
    got.backward(g.to(got.dtype))
    assert off(block.qkv.weight.grad, gw) < 0.05 and off(x.grad, gx) < 0.05
    block.zero_grad(), setattr(x, "grad", None)
    block.qkv.to(BF16), block.out.to(BF16)
    _, got = block(x)
    assert got.dtype == BF16 and off(got, want) < 0.02
    got.backward(g.to(BF16))
    assert off(block.qkv.weight.grad, gw) < 0.05 and off(x.grad, gx) < 0.05


# ---------------------------------------------------------------------------
# maps

@pytest.mark.parametrize("shape", ((2, 24, 9, 7), (3, 24), (2, 24, 11), (1, 24, 3, 4, 5)))
@pytest.mark.parametrize("act", ("silu", "identity", "leaky_relu"))
def test_group_norm_act(shape, act):
    layer = GroupNormAct(6, 24, activation=act, act_param=0.1, device="cuda")
    with torch.no_grad():
        layer.weight.copy_(rnd(40, 24)), layer.bias.copy_(rnd(41, 24))
    x = rnd(42, *shape)
    if x.dim() == 4:
        x = x.to(memory_format=torch.channels_last)
    x.requires_grad_()
    y = layer(x)
    g = rnd(43, *shape)
    y.backward(g)
    x6, w6, b6 = (t.detach().double().cpu().requires_grad_() for t in (x, layer.weight, layer.bias))
    z = torch.nn.functional.group_norm(x6, 6, w6, b6, layer.eps)
    y6 = {"silu": torch.nn.functional.silu, "identity": lambda t: t,
          "leaky_relu": lambda t: torch.nn.functional.leaky_relu(t, 0.1)}[act](z)
    y6.backward(g.double().cpu())
    # float32 throughout: some roundings of sums of up to a thousand terms
    assert off(y, y6) < 1e-5
    for got, want in ((x.grad, x6.grad), (layer.weight.grad, w6.grad), (layer.bias.grad, b6.grad)):
        assert off(got, want) < 1e-4
    assert layer.state_dict().keys() == torch.nn.GroupNorm(6, 24).state_dict().keys()


def test_group_norm_act_layouts():
    layer = GroupNormAct(4, 16, device="cuda")
    x = rnd(44, 2, 16, 6, 5)
    want = layer(x)
    cl = x.to(memory_format=torch.channels_last)
    assert torch.equal(layer(cl), want)
    assert layer(cl).is_contiguous(memory_format=torch.channels_last)
    wide = torch.empty(2, 40, 6, 5, device="cuda").to(memory_format=torch.channels_last)
    wide[:, 8:24] = x
    assert torch.equal(layer(wide[:, 8:24]), want)               # a slice of its channels
    x1 = cl.clone().requires_grad_()
    layer(x1).sum().backward()                                   # a gradient of one value
    x2 = cl.clone().requires_grad_()
    layer(x2).backward(torch.ones_like(cl))
    assert torch.equal(x1.grad, x2.grad)
    assert layer(torch.empty(0, 16, 6, 5, device="cuda")).shape == (0, 16, 6, 5)
    half = layer.to(BF16)
    assert half(x.to(BF16)).dtype == BF16
    with pytest.raises(ValueError, match="expects"):
        layer(x[:, :8])
    with pytest.raises(ValueError, match="divide"):
        GroupNormAct(5, 16)


def test_map_attention():
    """Group norm, projection, rotary over rows and columns, attention: a map's block."""
    torch.manual_seed(5)
    m = A.MapAttention(48, 2, groups=4, device="cuda")
    with torch.no_grad():
        m.norm.weight.add_(0.2 * torch.randn_like(m.norm.weight))
    x = rnd(45, 2, 48, 6, 5).to(memory_format=torch.channels_last).requires_grad_()
    y = m(x)
    g = rnd(46, 2, 48, 6, 5)
    y.backward(g)
    p6 = {n: p.detach().double().cpu().requires_grad_() for n, p in m.named_parameters()}
    x6 = x.detach().double().cpu().requires_grad_()
    n = torch.nn.functional.group_norm(x6, 4, p6["norm.weight"], p6["norm.bias"], m.norm.eps)
    n = n.flatten(2).transpose(1, 2)
    q, k, v = (n @ p6["qkv.weight"].T + p6["qkv.bias"]).unflatten(-1, (6, 24)).split(2, -2)
    i, j = torch.meshgrid(torch.arange(6), torch.arange(5), indexing="ij")
    pos = torch.stack((i, j), -1).flatten(0, 1)[None].expand(2, 30, 2)
    q, k = turned64(q, m.rotary, pos), turned64(k, m.rotary, pos)
    a = attend64(q, k, v, torch.ones(30, 30, dtype=torch.bool))
    o = a.flatten(-2) @ p6["out.weight"].T + p6["out.bias"]
    y6 = x6 + o.transpose(1, 2).unflatten(2, (6, 5))
    y6.backward(g.double().cpu())
    assert off(y, y6) < 1e-5 and y.is_contiguous(memory_format=torch.channels_last)
    # the projection's weight gradient reads codes of the norm's output
    for name, p in m.named_parameters():
        assert off(p.grad, p6[name].grad) < (0.05 if name == "qkv.weight" else 1e-4), name
    assert off(x.grad, x6.grad) < 1e-4
    video = A.MapAttention(48, 2, groups=4, axes=3, device="cuda")
    assert video(rnd(47, 1, 48, 2, 3, 4)).shape == (1, 48, 2, 3, 4)
    with pytest.raises(ValueError, match="extents"):
        video(x)


# ---------------------------------------------------------------------------
# the operators together: graphs, streams, an example

def run_all(t, ws):
    """Rotary, attention (its keys cut, its gradients' parts joined) and group norm, forward
    and backward, into t's buffers."""
    iabn.iabn_rotary(t["turn"], t["pos"], t["q"], t["qt"], t["k"], t["kt"])
    iabn.iabn_attention_forward(t["spec"], t["qt"], t["kt"], t["v"], t["out"], t["lse"], ws["f"])
    iabn.iabn_attention_backward(t["spec"], t["qt"], t["kt"], t["v"], t["out"], t["lse"], t["do"],
                                 t["dq"], t["dk"], t["dv"], ws["b"])
    iabn.iabn_rotary(t["turn"], t["pos"], t["dq"], t["dq"], t["dk"], t["dk"], inverse=True)
    iabn.iabn_group_norm_forward(t["x"], t["y"], 4, t["w"], t["bias"], ws["g"], act="silu",
                                 stats=t["stats"])
    iabn.iabn_group_norm_backward(t["x"], t["dy"], t["dx"], 4, t["w"], t["bias"], t["stats"],
                                  ws["g"], act="silu", dweight=t["dw"], dbias=t["db"])


OUTS = ("out", "lse", "dq", "dk", "dv", "y", "dx", "dw", "db")


def buffers(seed):
    t = dict(turn=iabn.RotarySpec(64), pos=torch.arange(600, dtype=torch.int32, device="cuda"),
             spec=iabn.AttentionSpec(causal=True))
    for i, (n, h) in enumerate((("q", 4), ("k", 2), ("v", 2), ("do", 4))):
        t[n] = rnd(seed + i, 1, 600, h, 64, dtype=BF16)
    for n, like in (("qt", "q"), ("kt", "k"), ("out", "q"), ("dq", "q"), ("dk", "k"), ("dv", "v")):
        t[n] = torch.empty_like(t[like])
    t["lse"] = iabn.attention_lse(t["q"])
    t["x"], t["dy"] = rnd(seed + 5, 2, 500, 32, dtype=BF16), rnd(seed + 6, 2, 500, 32, dtype=BF16)
    t["y"], t["dx"] = torch.empty_like(t["x"]), torch.empty_like(t["x"])
    t["w"], t["bias"] = rnd(seed + 7, 32), rnd(seed + 8, 32)
    t["dw"], t["db"], t["stats"] = (torch.empty(*s, device="cuda") for s in ((32,), (32,), (2, 4, 2)))
    return t


def spaces(t):
    return dict(f=iabn.attention_workspace(t["spec"], t["q"], t["k"]),
                b=iabn.attention_workspace(t["spec"], t["q"], t["k"], backward=True),
                g=iabn.group_norm_workspace(t["x"], 4))


def test_graph_replays():
    """Two captured graphs that share their workspaces, replayed in turn with new inputs and
    eager work between: each replay is the eager result."""
    a, b, eager = buffers(50), buffers(60), buffers(70)
    ws = spaces(a)
    assert ws["f"] is not None
    graphs = []
    for t in (a, b):
        run_all(t, ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run_all(t, ws)
        graphs.append(g)
    for i in range(4):
        for t, g in zip((a, b), graphs):
            for n in ("q", "k", "v", "do", "x", "dy"):
                fresh = rnd(100 + 7 * i + ord(n[0]), *t[n].shape, dtype=BF16)
                t[n].copy_(fresh)
                eager[n].copy_(fresh)
            for n in ("w", "bias"):
                eager[n].copy_(t[n])
            g.replay()
            got = {n: t[n].clone() for n in OUTS}
            run_all(eager, ws)
            torch.cuda.synchronize()
            for n in OUTS:
                assert torch.equal(got[n], eager[n]), (i, n)


def test_other_streams():
    """The current stream, and one given by name; two at once with workspaces of their own."""
    a, b, want = buffers(80), buffers(90), None
    wa, wb = spaces(a), spaces(b)
    run_all(a, wa), run_all(b, wb)
    torch.cuda.synchronize()
    want = [{n: t[n].clone() for n in OUTS} for t in (a, b)]
    for t in (a, b):
        for n in OUTS:
            t[n].fill_(math.nan)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(s1):
        run_all(a, wa)
    with torch.cuda.stream(s2):
        run_all(b, wb)
    torch.cuda.synchronize()
    for t, w in zip((a, b), want):
        for n in OUTS:
            assert torch.equal(t[n], w[n]), n
    out = torch.full_like(a["out"], math.nan)
    iabn.iabn_attention_forward(a["spec"], a["qt"], a["kt"], a["v"], out, None, wa["f"], stream=s1)
    s1.synchronize()
    assert torch.equal(out, want[0]["out"])


def test_host_tensors_are_refused_in_place_of_gpu_ones():
    t = buffers(95)
    with pytest.raises(TypeError, match="lse is"):
        iabn.iabn_attention_forward(t["spec"], t["q"], t["k"], t["v"], t["out"],
                                    torch.empty(1, 4, 600), None)
    with pytest.raises(TypeError, match="k is"):
        iabn.iabn_attention_forward(t["spec"], t["q"], t["k"].cpu(), t["v"], t["out"])
    with pytest.raises(TypeError, match="positions are on"):
        iabn.iabn_rotary(t["turn"], t["pos"].cpu(), t["q"], t["qt"])
    with pytest.raises(TypeError, match="inv_freq"):
        iabn.iabn_rotary(iabn.RotarySpec(64, device="cpu"), t["pos"], t["q"], t["qt"])
    with pytest.raises(ValueError, match="workspace"):
        iabn.iabn_group_norm_forward(t["x"], t["y"], 4, None, None,
                                     torch.empty(1 << 20, dtype=torch.uint8))


def load_example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "attention_block.py")
    spec = importlib.util.spec_from_file_location("attention_block", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_example_runs_and_its_gradients():
    ex = load_example()
    ex.main(["--rows", "64", "--cols", "64", "--heads", "4", "--steps", "2", "--tokens", "5",
             "--layers", "1", "--dtype", "f32"])
    torch.manual_seed(6)
    model = ex.Stack(64, 4, 2, 1, F32, "cuda")
    x, g = rnd(110, 2, 40, 64), rnd(111, 2, 40, 64)
    model(x).backward(g)
    # the first norm has no branch before it
    got = {n: p.grad.clone() for n, p in model.named_parameters() if p.grad is not None}
    model.zero_grad()
    model.plain(x).backward(g)
    for n, p in model.named_parameters():
        if p.grad is not None:
            assert off(got[n], p.grad) < 0.05, n
    assert len(got) == len(list(model.parameters())) - 1
