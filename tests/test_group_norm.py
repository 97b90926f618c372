"""Group norm with an activation on the GPU against float64 with derived bounds
(heads_ref.py)."""
import math

import pytest
import torch

iabn = pytest.importorskip("place_batchnorm_activation_amd")
import heads_ref  # noqa: E402

pytestmark = pytest.mark.gpu
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
DT = pytest.mark.parametrize("dtype", (BF16, F16, F32), ids=("bf16", "f16", "f32"))
ACTS = ("identity", "silu", "gelu", "gelu_tanh", "leaky_relu")


def make(seed, N, HW, C, dtype, mean=0.5, affine=True):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x = (r(N, HW, C) * (0.5 + torch.rand(C, generator=g)) + mean * r(C)).to(dtype).cuda()
    dy = r(N, HW, C).to(dtype).cuda()
    if not affine:
        return x, dy, None, None
    return x, dy, (1 + 0.2 * r(C)).cuda(), (0.3 * r(C)).cuda()


def both(x, dy, G, w, b, act, param=0.01, eps=1e-5):
    nan = lambda t: torch.full_like(t, math.nan)  # noqa: E731
    C = x.shape[-1]
    y, dx = nan(x), nan(x)
    stats = torch.full((x.shape[0], G, 2), math.nan, device="cuda")
    dw, db = torch.full((C,), math.nan, device="cuda"), torch.full((C,), math.nan, device="cuda")
    ws = iabn.group_norm_workspace(x, G)
    iabn.iabn_group_norm_forward(x, y, G, w, b, ws, act=act, act_param=param, eps=eps, stats=stats)
    iabn.iabn_group_norm_backward(x, dy, dx, G, w, b, stats, ws, act=act, act_param=param,
                                  dweight=dw, dbias=db)
    return dict(y=y, stats=stats, dx=dx, dweight=dw, dbias=db)


def check(got, val, bound):
    for name in got:
        heads_ref.within(got[name], val[name], bound[name], name)


@DT
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("N,HW,C,G", ((2, 100, 64, 8), (3, 37, 150, 10), (1, 700, 320, 32)))
def test_activations(dtype, act, N, HW, C, G):
    x, dy, w, b = make(1, N, HW, C, dtype)
    check(both(x, dy, G, w, b, act, 0.2),
          *heads_ref.group_norm(x, dy, G, w, b, act, 0.2, 1e-5))


@DT
@pytest.mark.parametrize("N,HW,C,G", ((1, 1, 8, 1), (1, 1, 7, 7), (2, 3, 5, 1), (5, 1, 96, 3),
                                      (1, 9, 1, 1), (2, 2, 2056, 8), (1, 20, 4100, 2),
                                      (1, 5000, 24, 3), (2, 4099, 40, 40), (1, 64, 2048, 1)))
def test_sizes(dtype, N, HW, C, G):
    x, dy, w, b = make(2, N, HW, C, dtype)
    check(both(x, dy, G, w, b, "silu"), *heads_ref.group_norm(x, dy, G, w, b, "silu", 0, 1e-5))


@DT
def test_without_affine(dtype):
    x, dy, _, _ = make(3, 2, 50, 48, dtype, affine=False)
    check(both(x, dy, 4, None, None, "silu"),
          *heads_ref.group_norm(x, dy, 4, None, None, "silu", 0, 1e-5))


@DT
def test_slices(dtype):
    """Channels of a wider tensor, at odd offsets."""
    x, dy, w, b = make(4, 2, 60, 48, dtype)
    wide = torch.full((2, 60, 101), math.nan, dtype=dtype, device="cuda")
    wide[..., 3:51], wide[..., 52:100] = x, dy
    val, bound = heads_ref.group_norm(x, dy, 6, w, b, "silu", 0, 1e-5)
    out = torch.full((2, 60, 99), math.nan, dtype=dtype, device="cuda")
    y, dx = out[..., 1:49], out[..., 50:98]
    stats, ws = torch.empty(2, 6, 2, device="cuda"), iabn.group_norm_workspace(x, 6)
    iabn.iabn_group_norm_forward(wide[..., 3:51], y, 6, w, b, ws, act="silu", stats=stats)
    iabn.iabn_group_norm_backward(wide[..., 3:51], wide[..., 52:100], dx, 6, w, b, stats, ws,
                                  act="silu")
    check(dict(y=y, dx=dx), val, bound)
    for c in (0, 49, 98):
        assert out[..., c].isnan().all()


@DT
@pytest.mark.parametrize("HW", (50, 3000))
def test_far_means(dtype, HW):
    """A mean a thousand times the spread (exact in the type: steps of 8 about 4096 in bf16 are
    too coarse, so the spread there is of whole steps)."""
    g = torch.Generator().manual_seed(5)
    step = {BF16: 16.0, F16: 2.0, F32: 1.0}[dtype]
    x = (4096 + step * torch.randint(-3, 4, (2, HW, 32), generator=g)).to(dtype).cuda()
    dy = torch.randn(2, HW, 32, generator=g).to(dtype).cuda()
    check(both(x, dy, 4, None, None, "identity"),
          *heads_ref.group_norm(x, dy, 4, None, None, "identity", 0, 1e-5))


@DT
def test_constant_and_huge_groups(dtype):
    """A group of one value: xhat 0, rstd 1/sqrt(eps)."""
    x, dy, w, b = make(6, 2, 40, 32, dtype)
    x[0, :, :8] = 3.0
    got = both(x, dy, 4, w, b, "identity", eps=1e-3)
    assert torch.equal(got["y"][0, :, :8], b[:8].to(dtype).expand(40, 8))
    check(got, *heads_ref.group_norm(x, dy, 4, w, b, "identity", 0, 1e-3))


@DT
def test_nan_stays_in_its_group(dtype):
    x, dy, w, b = make(7, 2, 40, 32, dtype)
    x[1, 5, 9] = math.nan
    got = both(x, dy, 4, w, b, "silu")
    bad = got["y"].isnan()
    assert bad[1, :, 8:16].all() and int(bad.sum()) == 40 * 8


@DT
def test_in_place(dtype):
    x, dy, w, b = make(8, 2, 300, 72, dtype)
    want = both(x, dy, 6, w, b, "silu")
    stats, ws = torch.empty(2, 6, 2, device="cuda"), iabn.group_norm_workspace(x, 6)
    iabn.iabn_group_norm_backward(x, dy, dy, 6, w, b, want["stats"], ws, act="silu")
    assert torch.equal(dy, want["dx"])
    iabn.iabn_group_norm_forward(x, x, 6, w, b, ws, act="silu", stats=stats)
    assert torch.equal(x, want["y"]) and torch.equal(stats, want["stats"])


@DT
@pytest.mark.parametrize("N,HW,C,G", ((2, 300, 4104, 3), (1, 40, 2056, 257), (3, 9, 5000, 1)))
def test_wide(dtype, N, HW, C, G):
    """More channels than a workgroup has, groups across two workgroups' channels."""
    x, dy, w, b = make(14, N, HW, C, dtype)
    check(both(x, dy, G, w, b, "silu"), *heads_ref.group_norm(x, dy, G, w, b, "silu", 0, 1e-5))


@DT
@pytest.mark.parametrize("HW", (20, 5000))
def test_gradients_in_place_of_the_parameters(dtype, HW):
    x, dy, w, b = make(15, 2, HW, 64, dtype)
    want = both(x, dy, 4, w, b, "silu")
    for same in ("weight", "bias", "both"):
        weight, bias, dx = w.clone(), b.clone(), torch.empty_like(x)
        dw = torch.empty_like(w) if same == "bias" else weight
        db = torch.empty_like(b) if same == "weight" else bias
        iabn.iabn_group_norm_backward(x, dy, dx, 4, weight, bias, want["stats"],
                                      iabn.group_norm_workspace(x, 4), act="silu", dweight=dw,
                                      dbias=db)
        for name, t in (("dx", dx), ("dweight", dw), ("dbias", db)):
            assert torch.equal(t, want[name]), name


def test_statistics_are_optional():
    x, dy, w, b = make(9, 3, 300, 64, F32)
    ws = iabn.group_norm_workspace(x, 8)
    y = torch.empty_like(x)
    iabn.iabn_group_norm_forward(x, y, 8, w, b, ws, act="silu")
    assert torch.equal(y, both(x, dy, 8, w, b, "silu")["y"])


@pytest.mark.parametrize("shape", ((0, 5, 24), (3, 0, 24)))
def test_empty(shape):
    x = torch.empty(*shape, device="cuda")
    got = both(x, x, 3, None, None, "silu")
    assert (got["dweight"] == 0).all() and (got["dbias"] == 0).all()


def test_many_samples():
    """More samples than a grid's second extent."""
    x, dy, w, b = make(10, 70000, 1, 16, BF16)
    check(both(x, dy, 2, w, b, "silu"), *heads_ref.group_norm(x, dy, 2, w, b, "silu", 0, 1e-5))


@DT
def test_same_bits_every_time(dtype):
    x, dy, w, b = make(11, 2, 5000, 96, dtype)
    one, two = both(x, dy, 8, w, b, "gelu"), both(x, dy, 8, w, b, "gelu")
    for n in one:
        assert torch.equal(one[n], two[n]), n


def test_gradients_against_differences():
    """d/dt of sum(g * y(x + t u)) by central differences of the float32 forward: off by h^2/6 of
    a third derivative of order one, and by 2^-24 sqrt(n) |g y| / h; with h = 2^-6 and |u| = 1
    both are below 1e-3 sqrt(n)."""
    x, g, w, b = make(12, 2, 30, 24, F32)
    got = both(x, g, 3, w, b, "gelu")
    ws = iabn.group_norm_workspace(x, 3)

    def value(x, w, b):
        y = torch.empty_like(x)
        iabn.iabn_group_norm_forward(x, y, 3, w, b, ws, act="gelu")
        return float((y.double() * g.double()).sum())

    h = 2.0 ** -6
    for i, name in enumerate(("dx", "dweight", "dbias")):
        p = [x, w, b]
        u = torch.randn(p[i].shape, generator=torch.Generator().manual_seed(i)).cuda()
        u /= u.norm()
        up, down = list(p), list(p)
        up[i], down[i] = p[i] + h * u, p[i] - h * u
        diff = (value(*up) - value(*down)) / (2 * h)
        want = float((got[name].double() * u.double()).sum())
        assert abs(diff - want) <= 1e-3 * math.sqrt(x.numel()), (name, diff, want)


def test_the_most_groups():
    """2^24 - 1 groups of one channel and two rows: every one is written.  With d half the pair's
    difference, xhat = +-d rstd and rstd = 1/sqrt(d^2 + eps), to a few roundings of float32 (2^-20
    of it); the gradients are those of that function."""
    G, eps = (1 << 24) - 1, 0.1
    x, dy = (torch.randn(1, 2, G, generator=torch.Generator(device="cuda").manual_seed(s),
                         device="cuda") for s in (16, 17))
    got = both(x, dy, G, None, None, "identity", eps=eps)
    x6, dy6 = x.double(), dy.double()
    half = (x6[:, 0] - x6[:, 1]) / 2
    rstd = (half.square() + eps).rsqrt()
    xhat = torch.stack((half * rstd, -half * rstd), 1)
    m, mx = dy6.mean(1, keepdim=True), (dy6 * xhat).mean(1, keepdim=True)
    dx = rstd[:, None] * (dy6 - m - xhat * mx)
    for name, want, size in (("y", xhat, xhat.abs() + 1), ("stats", torch.stack((x6.mean(1), rstd), -1),
                                                           rstd[..., None] + x6.abs().amax(1)[..., None]),
                             ("dx", dx, rstd[:, None] * (dy6.abs().sum(1, keepdim=True) + 1)),
                             ("dbias", dy6.sum((0, 1)), dy6.abs().sum((0, 1))),
                             ("dweight", (dy6 * xhat).sum((0, 1)), dy6.abs().sum((0, 1)) + 1)):
        off = (got[name].double() - want).abs()
        assert bool((off <= 2.0 ** -20 * size).all()), (name, float((off / size).max()))
