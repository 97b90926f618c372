"""The residual modules (place_batchnorm_activation_amd.residual) on the GPU against
torch's autograd of the same functions in float64 on the CPU.

With stored tensors (keep="full") in float32 the gradients are torch's up to fp32
rounding.  With codes they differ by the codes' own rounding: a value is off by at most
half a step, and a step is at most 1/63.5 of its group's largest magnitude; for rows of
normal values (largest of 32: 2 to 3 sigma) that is an rms error of 3/63.5/sqrt(12) = 1.4%
of sigma at the most, in each operand of a gradient that codes enter.  A gradient here
has at most three such factors: 5% in the 2-norm."""
import pytest
import torch

pytest.importorskip("place_batchnorm_activation_amd")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from place_batchnorm_activation_amd import residual
    from place_batchnorm_activation_amd.residual import (GLULinear, KeptLinear, ResidualMLP,
                                                         ResNorm)


def norm64(x, kind, w, b, eps):
    if kind == "none":
        return x
    if kind == "layer":
        x = x - x.mean(-1, keepdim=True)
    x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps)
    x = x * w
    return x if b is None else x + b


def off(got, want):
    want = want.double().cpu()
    got, want = got.detach().double().cpu(), want.detach()
    return float((got - want).norm() / (want.norm() + 1e-300))


def leaf(t):
    return t.detach().double().cpu().requires_grad_()


@pytest.mark.parametrize("keep,tol", [("full", 2e-5), ("codes", 0.05)])
@pytest.mark.parametrize("post,pre,gate", [("rms", "rms", "vector"), ("layer", "layer", "rows"),
                                           ("none", "rms", "none"), ("none", "layer", "vector"),
                                           ("rms", "none", "rows")])
def test_resnorm_module(post, pre, gate, keep, tol):
    torch.manual_seed(3)
    B, S, C = 3, 40, 96
    m = ResNorm(C, post, pre, alpha=0.5, gate=gate == "vector", keep=keep, device="cuda")
    with torch.no_grad():
        for p in m.parameters():
            p.add_(0.2 * torch.randn_like(p))
    r, b = (torch.randn(B, S, C, device="cuda", requires_grad=True) for _ in range(2))
    g = torch.randn(B, C, device="cuda", requires_grad=True) if gate == "rows" else None
    r_out, n, kept = m(r, b, g)
    assert (kept is None) == (keep == "full" or pre == "none")
    vr, vn = torch.randn_like(r), torch.randn_like(r)
    loss = (r_out * vr).sum() + ((n * vn).sum() if n is not None else 0.0)
    loss.backward()
    p = {k: leaf(v) for k, v in m.named_parameters()}
    r64, b64 = leaf(r), leaf(b)
    g64 = leaf(g) if g is not None else p.get("gate")
    br = norm64(b64, post, p.get("post_weight"), p.get("post_bias"), m.eps)
    if g64 is not None:
        br = br * (g64[:, None] if gate == "rows" else g64)
    ro = r64 + 0.5 * br
    loss64 = (ro * vr.double().cpu()).sum()
    assert off(r_out, ro) < 1e-6
    if pre != "none":
        n64 = norm64(ro, pre, p["pre_weight"], p.get("pre_bias"), m.eps)
        assert off(n, n64) < 1e-6
        loss64 = loss64 + (n64 * vn.double().cpu()).sum()
    loss64.backward()
    assert off(r.grad, r64.grad) < tol and off(b.grad, b64.grad) < tol
    if g is not None:
        assert off(g.grad, g64.grad) < tol
    for k, v in m.named_parameters():
        assert off(v.grad, p[k].grad) < tol, k


@pytest.mark.parametrize("dtype,rounding", [(torch.float32, 1e-6), (torch.bfloat16, 0.01)])
def test_linear_and_glu_modules(dtype, rounding):
    torch.manual_seed(5)
    T, C, F = 300, 160, 104
    norm = ResNorm(C, pre="layer", device="cuda")
    up = KeptLinear(C, 2 * F, device="cuda", dtype=dtype)
    alone = KeptLinear(C, 2 * F, device="cuda", dtype=dtype)
    alone.load_state_dict(up.state_dict())
    down = GLULinear(F, C, device="cuda", dtype=dtype, act="gelu")
    x = torch.randn(T, C, device="cuda").to(dtype).requires_grad_()
    _, n, kept = norm(x)
    dy = torch.randn(T, C, device="cuda").to(dtype)
    y = down(up(n, kept))
    y.backward(dy)
    p = {k: leaf(v) for k, v in [("uw", up.weight), ("ub", up.bias), ("dw", down.weight),
                                 ("db", down.bias), ("nw", norm.pre_weight),
                                 ("nb", norm.pre_bias)]}
    x64 = leaf(x)
    n64 = norm64(x64, "layer", p["nw"], p["nb"], norm.eps)
    g, u = (n64 @ p["uw"].t() + p["ub"]).chunk(2, -1)
    y64 = (torch.nn.functional.gelu(g) * u) @ p["dw"].t() + p["db"]
    assert off(y, y64) < max(rounding, 1e-5)
    y64.backward(dy.double().cpu())
    tol = 0.05 + 3 * rounding
    for got, want in ((x, x64), (up.weight, p["uw"]), (up.bias, p["ub"]), (down.weight, p["dw"]),
                      (down.bias, p["db"]), (norm.pre_weight, p["nw"]), (norm.pre_bias, p["nb"])):
        assert off(got.grad, want.grad) < tol
    # the layer's own codes of n serve as well as the norm's of xhat
    z = alone(n.detach())
    z.backward(torch.randn_like(z))
    dz = torch.randn_like(z)
    alone.weight.grad = None
    alone(n.detach()).backward(dz)
    assert off(alone.weight.grad, dz.double().t() @ n.detach().double()) < tol


def test_inference_keeps_nothing():
    m = ResidualMLP(64, 32, device="cuda", dtype=torch.bfloat16)
    x = torch.randn(5, 64, device="cuda", dtype=torch.bfloat16)
    r, b = m(x)
    with torch.no_grad():
        r2, b2 = m(x)
        assert m.norm(x)[2] is None
    assert torch.equal(r, r2) and torch.equal(b, b2)
    one, _ = m(x[:1])
    assert torch.equal(one, r[:1])


def test_unused_outputs_and_strided_gradients():
    """dn or dr_out missing, gradients that are expanded or transposed views."""
    m = ResNorm(48, post="rms", pre="rms", device="cuda")
    r, b = (torch.randn(6, 48, device="cuda", requires_grad=True) for _ in range(2))
    r_out, n, _ = m(r, b)
    n.sum().backward()                                  # an expanded gradient, dr_out None
    want = [t.grad.clone() for t in (r, b)]
    r.grad = b.grad = None
    r_out, n, _ = m(r, b)
    (n.t().contiguous().t() * torch.ones(48, 6, device="cuda").t()).sum().backward()
    assert torch.equal(r.grad, want[0]) and torch.equal(b.grad, want[1])
    r.grad = b.grad = None
    m(r, b)[0].sum().backward()                         # dn None
    assert torch.equal(r.grad, torch.ones_like(r)) and bool(torch.isfinite(b.grad).all())
    with pytest.raises(ValueError):
        m(r, b[:3])
    with pytest.raises(ValueError):
        ResNorm(48, keep="some")
    with pytest.raises(ValueError):
        GLULinear(10, 48, device="cuda")(r)


def test_example_trains_like_plain_torch_with_less_memory(capsys):
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "residual_mlp.py")
    spec = importlib.util.spec_from_file_location("residual_mlp_example", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    kept, plain = mod.main(["--rows", "4096", "--cols", "512", "--hidden", "1024", "--layers", "4",
                            "--steps", "6"])
    assert plain[0][-1] < plain[0][0] and kept[0][-1] < kept[0][0]
    for a, b in zip(kept[0], plain[0]):
        assert abs(a - b) < 0.01 * abs(b)
    assert kept[2] < 0.6 * plain[2]


def test_an_empty_batch_has_gradients():
    """Expanded gradients of no rows, through every module of a block."""
    m = ResidualMLP(64, 32, device="cuda")
    r = torch.empty(0, 64, device="cuda", requires_grad=True)
    b = torch.empty(0, 64, device="cuda", requires_grad=True)
    r_out, n, _ = m.norm(r, b)
    (r_out.sum() + n.sum()).backward()
    r_out, out = m(r, b)
    out.sum().backward()
    assert r.grad.shape == b.grad.shape == (0, 64)
    for k, p in m.named_parameters():
        assert float(p.grad.abs().max()) == 0.0, k


def test_an_empty_batch_leaves_a_gate_no_gradient():
    m = ResNorm(64, post="rms", pre="rms", gate=True, device="cuda")
    r, b = (torch.empty(0, 64, device="cuda", requires_grad=True) for _ in range(2))
    own = torch.ones(5, 64, device="cuda", requires_grad=True)
    for gate, leaf_ in ((None, m.gate), (own, own)):
        dirt = [torch.full((5, 64), 9.0, device="cuda") for _ in range(16)]
        dirt += [torch.full((64,), 9.0, device="cuda") for _ in range(16)]
        r_out, n, _ = m(r, b, gate)
        del dirt                       # what the next allocations find in memory
        torch.autograd.backward([r_out, n], [torch.empty_like(r_out), torch.empty_like(n)])
        assert float(leaf_.grad.abs().max()) == 0.0


def test_kept_codes_serve_their_own_tensor_only():
    torch.manual_seed(11)
    norm, other = (ResNorm(64, device="cuda") for _ in range(2))
    lin = KeptLinear(64, 32, device="cuda")
    x = torch.randn(4, 6, 64, device="cuda")
    _, n, kept = norm(x)
    for bad in (2.0 * n, n.clone(), n.transpose(0, 1), other(x)[1], n[:, :3], n.reshape(48, 32)):
        with pytest.raises(ValueError):
            lin(bad, kept)
    # its rows in any shape, cut from the graph, and cast to the weight's type
    dy = torch.randn(24, 32, device="cuda")
    want = dy.double().t() @ n.detach().double().view(24, 64)
    for good in (n, n.view(24, 64), n.flatten(0, 1)[None], n.detach()):
        lin.weight.grad = None
        lin(good, kept).backward(dy.view(*good.shape[:-1], 32), retain_graph=True)
        assert off(lin.weight.grad, want) < 0.05
    low = KeptLinear(64, 32, device="cuda", dtype=torch.bfloat16)
    y = low(n, kept)
    assert y.dtype == torch.bfloat16
    y.backward(dy.view(4, 6, 32).bfloat16())
    assert off(low.weight.grad, want) < 0.08
    with torch.no_grad():
        n.mul_(2.0)                                   # written since
    with pytest.raises(ValueError):
        lin(n, kept)
    assert residual.Kept(*kept[:4]).fits(n)               # without a mark only the shape counts


def test_gates_are_broadcast_or_refused():
    """Whatever shape of gate is taken means what broadcasting makes of it."""
    torch.manual_seed(13)
    B, S, C = 4, 64, 64
    m = ResNorm(C, pre="none", keep="full", device="cuda")
    r, b = torch.zeros(B, S, C, device="cuda"), torch.randn(B, S, C, device="cuda")
    for shape in ((C,), (1, C), (1, 1, C), (B, 1, C), (B, S, C)):
        g = torch.randn(*shape, device="cuda", requires_grad=True)
        out = m(r, b, g)[0]
        assert torch.equal(out, g.detach() * b)
        out.sum().backward()
        assert off(g.grad, b.double().sum_to_size(shape)) < 1e-6
    # rows without a batch: runs of them, or one each
    g = torch.randn(B, 1, C, device="cuda")
    assert torch.equal(m(r.view(-1, C), b.view(-1, C), g)[0], (g * b).view(-1, C))
    g = torch.randn(B, S, C, device="cuda")
    assert torch.equal(m(r.view(-1, C), b.view(-1, C), g)[0], (g * b).view(-1, C))
    # one value a row, a vector of another length, a gate for each position, batch and
    # position in the other order
    for shape in ((B, S, 1), (B * S, 1), (2 * C,), (C // 2,), (1, S, C), (S, B, C), (S, 1, C), ()):
        with pytest.raises(ValueError):
            m(r, b, torch.ones(shape, device="cuda"))


@pytest.mark.parametrize("low", [torch.bfloat16, torch.float16], ids=str)
@pytest.mark.parametrize("with_kept", [False, True], ids=["own", "kept"])
def test_linear_and_glu_modules_under_autocast(low, with_kept):
    """Parameters in float32, products in 16 bits, gradients in float32 (the bounds of
    test_linear_and_glu_modules in bf16)."""
    torch.manual_seed(17)
    T, C, F = 300, 160, 104
    norm = ResNorm(C, pre="layer", device="cuda")
    up, down = KeptLinear(C, 2 * F, device="cuda"), GLULinear(F, C, device="cuda")
    x = torch.randn(T, C, device="cuda", requires_grad=True)
    with torch.autocast("cuda", dtype=low):
        _, n, kept = norm(x)
        h = up(n, kept if with_kept else None)
        y = down(h)
    assert n.dtype == torch.float32 and h.dtype == y.dtype == low
    dy = torch.randn(T, C, device="cuda").to(low)
    y.backward(dy)
    p = {k: leaf(v) for k, v in [("uw", up.weight), ("ub", up.bias), ("dw", down.weight),
                                 ("db", down.bias), ("nw", norm.pre_weight),
                                 ("nb", norm.pre_bias)]}
    x64 = leaf(x)
    n64 = norm64(x64, "layer", p["nw"], p["nb"], norm.eps)
    g, u = (n64 @ p["uw"].t() + p["ub"]).chunk(2, -1)
    y64 = (torch.nn.functional.silu(g) * u) @ p["dw"].t() + p["db"]
    assert off(y, y64) < 0.01
    y64.backward(dy.double().cpu())
    for got, want in ((x, x64), (up.weight, p["uw"]), (up.bias, p["ub"]), (down.weight, p["dw"]),
                      (down.bias, p["db"]), (norm.pre_weight, p["nw"]), (norm.pre_bias, p["nb"])):
        assert got.grad.dtype == torch.float32
        assert off(got.grad, want.grad) < 0.08


def block64(m, r, b):
    """ResidualMLP in float64 on leaves of its parameters: (r', b', leaves)."""
    p = {k: leaf(v) for k, v in m.named_parameters()}
    if b is not None:
        br = norm64(b, "rms", p["norm.post_weight"], None, m.norm.eps)
        r = r + m.norm.alpha * (br if m.norm.gate is None else br * p["norm.gate"])
    n = norm64(r, "rms", p["norm.pre_weight"], None, m.norm.eps)
    g, u = (n @ p["up.weight"].t()).chunk(2, -1)
    return r, (torch.nn.functional.silu(g) * u) @ p["down.weight"].t(), p


@pytest.mark.parametrize("how", ["autocast", "stream", "cast"])
def test_blocks_of_mixed_types(how):
    """A float32 stream with 16-bit branches (under autocast, and with 16-bit layers), and a
    block whose parameters .to() made 16-bit.  Bounds: those of 8 bits and of bf16, 5 of its
    roundings deep."""
    torch.manual_seed(19)
    T, C, F, low = 200, 96, 64, torch.bfloat16
    first, second = (ResidualMLP(C, F, gate=True, device="cuda",
                                 dtype=low if how == "stream" else None) for _ in range(2))
    if how == "cast":
        first, second = first.to(low), second.to(low)
    x = torch.randn(T, C, device="cuda", dtype=low if how == "cast" else torch.float32)
    x.requires_grad_()
    b0 = torch.randn(T, C, device="cuda").to(low).requires_grad_()
    with torch.autocast("cuda", dtype=low, enabled=how == "autocast"):
        r, b = first(x, b0)
        r, b = second(r, b)
    assert r.dtype == x.dtype and b.dtype == low
    vr, vb = torch.randn(T, C, device="cuda"), torch.randn(T, C, device="cuda").to(low)
    torch.autograd.backward([r, b], [vr.to(r.dtype), vb])
    x64, b64 = leaf(x), leaf(b0)
    r1, out, p1 = block64(first, x64, b64)
    r2, out, p2 = block64(second, r1, out)
    assert off(r, r2) < 0.02 and off(b, out) < 0.04
    with torch.no_grad(), torch.autocast("cuda", dtype=low, enabled=how == "autocast"):
        assert torch.equal(second(*first(x, b0))[1], b)
    torch.autograd.backward([r2, out], [vr.to(r.dtype).double().cpu(), vb.double().cpu()])
    for got, want in [(x, x64), (b0, b64)] + [(v, p[k]) for m, p in ((first, p1), (second, p2))
                                              for k, v in m.named_parameters()]:
        assert got.grad.dtype == got.dtype and off(got.grad, want.grad) < 0.1


def test_norms_promote_and_cast():
    """A 16-bit stream with a float32 branch, 16-bit gates with float32 rows."""
    m = ResNorm(64, post="rms", pre="layer", keep="full", device="cuda")
    r, b = torch.randn(8, 64, device="cuda"), torch.randn(8, 64, device="cuda")
    r_out, n, _ = m(r.half(), b)
    want = m(r.half().float(), b)
    assert r_out.dtype == n.dtype == torch.float32
    assert torch.equal(r_out, want[0]) and torch.equal(n, want[1])
    g = torch.rand(8, 64, device="cuda").bfloat16()
    assert torch.equal(m(r, b, g)[1], m(r, b, g.float())[1])
    want = m(r.half(), b.half(), g.float())[1]
    assert want.dtype == torch.float16 and torch.equal(m(r.half(), b.half(), g)[1], want)


def test_a_weight_may_be_a_transposed_view():
    torch.manual_seed(23)
    lin = KeptLinear(64, 48, bias=False, device="cuda")
    lin.weight = torch.nn.Parameter(torch.randn(64, 48, device="cuda").t())
    x = torch.randn(30, 64, device="cuda", requires_grad=True)
    dy = torch.randn(30, 48, device="cuda")
    lin(x).backward(dy)
    assert off(lin.weight.grad, dy.double().t() @ x.detach().double()) < 0.05
    assert off(x.grad, dy.double() @ lin.weight.detach().double()) < 1e-5


def test_overlapping_windows_are_taken():
    """Windows of one sequence, as unfold makes them, into every module."""
    torch.manual_seed(29)
    x = torch.randn(100, device="cuda").unfold(0, 64, 1)
    own = x.contiguous()
    for m in (KeptLinear(64, 32, device="cuda"), GLULinear(32, 16, device="cuda")):
        dy = torch.randn(len(x), m.out_features, device="cuda")
        grads = []
        for v in (x, own):
            m.weight.grad = None
            m(v).backward(dy)
            grads.append(m.weight.grad)
        assert torch.equal(*grads)
    m = ResNorm(64, post="rms", pre="rms", device="cuda")
    assert torch.equal(m(x, x)[1], m(own, own)[1])


@pytest.mark.parametrize("shape", [(0, 64), (0, 1, 64), (0, 5, 64)])
def test_gates_of_an_empty_batch(shape):
    """A gate for each of no samples, or of their rows."""
    m = ResNorm(64, post="rms", pre="layer", device="cuda")
    r, b = (torch.empty(0, 5, 64, device="cuda", requires_grad=True) for _ in range(2))
    g = torch.empty(shape, device="cuda", requires_grad=True)
    r_out, n, _ = m(r, b, g)
    (r_out.sum() + n.sum()).backward()
    assert r_out.shape == n.shape == r.grad.shape == (0, 5, 64) and g.grad.shape == shape
    for p in m.parameters():
        assert float(p.grad.abs().max()) == 0.0
    with pytest.raises(ValueError):
        m(torch.ones(2, 64, device="cuda"), torch.ones(2, 64, device="cuda"), g)
