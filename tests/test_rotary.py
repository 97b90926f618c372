"""Rotary positions on the GPU against float64 with derived bounds (heads_ref.py)."""
import math

import pytest
import torch

iabn = pytest.importorskip("place_batchnorm_activation_amd")
import heads_ref  # noqa: E402

pytestmark = pytest.mark.gpu
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
DT = pytest.mark.parametrize("dtype", (BF16, F16, F32), ids=("bf16", "f16", "f32"))


def rnd(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed))


def positions(seed, kind, *shape):
    g = torch.Generator().manual_seed(seed)
    if kind == "f32":
        return 40 * torch.rand(*shape, generator=g).cuda() - 20
    return torch.randint(0, 5000, shape, generator=g).to(
        torch.int32 if kind == "i32" else torch.int64).cuda()


def axis_of(spec):
    return torch.zeros(spec.pairs, dtype=torch.int32) if spec.axis is None else spec.axis


def check(spec, pos, x, y, inverse=False):
    pos = pos.expand(x.shape[0], *pos.shape[-2:])
    val, bound = heads_ref.rotary(x, pos, spec.inv_freq, axis_of(spec), spec.interleaved, inverse)
    heads_ref.within(y, val, bound)


@DT
@pytest.mark.parametrize("kind", ("i32", "i64", "f32"))
@pytest.mark.parametrize("interleaved", (False, True))
@pytest.mark.parametrize("D,sections", ((64, (32,)), (128, (16, 24, 24)), (72, (15, 15)),
                                        (10, (3, 2)), (7, (1, 1)), (40, (3, 1, 4, 2)),
                                        (64, (8, 8))))
def test_turns(dtype, kind, interleaved, D, sections):
    spec = iabn.RotarySpec(D, sections, interleaved=interleaved)
    pos = positions(D, kind, 2, 19, len(sections))
    q, k = rnd(1, 2, 19, 5, D).to(dtype).cuda(), rnd(2, 2, 19, 2, D).to(dtype).cuda()
    qo, ko = torch.full_like(q, math.nan), torch.full_like(k, math.nan)
    for inverse in (False, True):
        iabn.iabn_rotary(spec, pos, q, qo, k, ko, inverse=inverse)
        check(spec, pos, q, qo, inverse)
        check(spec, pos, k, ko, inverse)


@DT
@pytest.mark.parametrize("interleaved", (False, True))
@pytest.mark.parametrize("sections", ((32,), (11, 10)))
def test_in_place_equals_out_of_place(dtype, interleaved, sections):
    spec = iabn.RotarySpec(72, sections, interleaved=interleaved)
    pos = positions(3, "i32", 333, len(sections))
    q, k = rnd(4, 1, 333, 12, 72).to(dtype).cuda(), rnd(5, 1, 333, 4, 72).to(dtype).cuda()
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    iabn.iabn_rotary(spec, pos, q, qo, k, ko)
    iabn.iabn_rotary(spec, pos, q, q, k, k)
    assert torch.equal(q, qo) and torch.equal(k, ko)


@DT
@pytest.mark.parametrize("tokens", (1, 3, 2000))
def test_slices_packed_and_one_axis(dtype, tokens):
    """Slices of a projection at odd offsets, packed rows, positions without an axis."""
    spec = iabn.RotarySpec(64)
    qkv = rnd(6, tokens, 8 * 64 + 1).to(dtype).cuda()[:, 1:].unflatten(-1, (8, 64))
    q, k = qkv[:, :4], qkv[:, 4:6]
    pos = positions(7, "i64", tokens)
    want, kwant = q.clone(), k.clone()
    iabn.iabn_rotary(spec, pos, q, want, k, kwant)
    check(spec, pos[:, None], q[None], want[None])
    check(spec, pos[:, None], k[None], kwant[None])
    rest = qkv[:, 6:].clone()
    iabn.iabn_rotary(spec, pos, q, q, k, k)
    assert torch.equal(q, want) and torch.equal(k, kwant) and torch.equal(qkv[:, 6:], rest)


@DT
def test_heads_before_rows_and_q_alone(dtype):
    spec = iabn.RotarySpec(64, (16, 16), ramp="axis", mixed=True)
    pos = positions(8, "f32", 2, 37, 2)
    q = rnd(9, 2, 3, 37, 64).to(dtype).cuda().transpose(1, 2)
    out = torch.full((2, 3, 37, 64), math.nan, dtype=dtype, device="cuda").transpose(1, 2)
    iabn.iabn_rotary(spec, pos, q, out)
    check(spec, pos, q, out)


def test_far_positions():
    """Positions to 2^31: the angle keeps its digits."""
    spec = iabn.RotarySpec(64)
    pos = torch.tensor([0, 1, 1 << 20, (1 << 31) - 1, -(1 << 31)], dtype=torch.int32).cuda()
    q = rnd(10, 1, 5, 2, 64).cuda()
    out = torch.empty_like(q)
    iabn.iabn_rotary(spec, pos, q, out)
    check(spec, pos[:, None], q, out)


def test_axis_values_outside_are_cut():
    axis = torch.tensor([-3, 0, 1, 99], dtype=torch.int32).cuda()
    inv = torch.tensor([1.0, 0.5, 0.25, 0.125], dtype=torch.float64).cuda()
    spec = iabn.RotarySpec(8, inv_freq=inv, axis=axis, axes=2)
    pos = positions(11, "i32", 1, 6, 2)
    q = rnd(12, 1, 6, 2, 8).cuda()
    out = torch.empty_like(q)
    iabn.iabn_rotary(spec, pos, q, out)
    val, bound = heads_ref.rotary(q, pos, inv, axis.clamp(0, 1))
    heads_ref.within(out, val, bound)


@DT
def test_inverse_returns(dtype):
    """Turning there and back: two roundings of each value's pair."""
    spec = iabn.RotarySpec(128, (32, 32))
    pos = positions(13, "i32", 2, 50, 2)
    q = rnd(14, 2, 50, 4, 128).to(dtype).cuda()
    there, back = torch.empty_like(q), torch.empty_like(q)
    iabn.iabn_rotary(spec, pos, q, there)
    iabn.iabn_rotary(spec, pos, there, back, inverse=True)
    x = q.double().cpu()
    m = (x[..., :64].abs() + x[..., 64:].abs()).repeat(1, 1, 1, 2)
    # each turn rounds both of a pair by u of its size, and is off by 40 e of it
    heads_ref.within(back, x, m * (4 * heads_ref.HALF[dtype] + 80 * heads_ref.E))


def test_no_tokens():
    spec = iabn.RotarySpec(64)
    q = torch.empty(2, 0, 4, 64, device="cuda")
    iabn.iabn_rotary(spec, torch.empty(2, 0, dtype=torch.int32, device="cuda"), q, q)
    q = torch.empty(0, 5, 4, 64, device="cuda")
    iabn.iabn_rotary(spec, torch.empty(5, dtype=torch.int32, device="cuda"), q, q)
