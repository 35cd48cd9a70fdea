"""Rotary positions on the GPU against their definition in 64 bits."""
import math

import pytest
import torch

from block_reference import DEV, TYPES, check_rotary, normal

pytestmark = pytest.mark.gpu
# tokens, heads, columns, rotated columns
SHAPES = [(1, 1, 2, 2), (1, 64, 128, 128), (3, 5, 64, 64), (17, 3, 80, 20), (5, 25, 80, 80), (9, 7, 100, 50), (4, 2, 96, 6),
          (1000, 12, 64, 32), (2, 3, 1024, 1024), (2, 2, 1000, 998), (33, 1, 36, 34), (1, 300, 40, 40), (64, 40, 128, 128),
          (5, 4, 7, 2), (6, 3, 33, 16), (129, 2, 256, 128)]


@pytest.fixture(scope="module")
def bfo():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from bf16_numerics_amd import binding
    torch.cuda.set_device(0)
    return binding


def inputs(seed, tokens, heads, dim, t, reach=4096):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return normal(g, tokens, heads, dim).to(t), torch.randint(-reach, reach, (tokens,), generator=g, device=DEV).to(torch.int32)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("half", [True, False])
@pytest.mark.parametrize("backward", [False, True])
def test_sizes(bfo, dt, half, backward):
    for k, (tokens, heads, dim, rotated) in enumerate(SHAPES):
        print(tokens, heads, dim, rotated, flush=True)
        x, positions = inputs(k, tokens, heads, dim, TYPES[dt])
        f = bfo.rotary_frequencies(rotated, device=DEV)
        out = torch.full_like(x, float("nan"))
        layout = bfo.ROTARY_HALF if half else bfo.ROTARY_INTERLEAVED
        bfo.rotary_apply(x, f, out, positions=positions, layout=layout, backward=backward, amplitude=1.0 + 0.25 * (k % 2))
        check_rotary(out, x, positions, f, half, 1.0 + 0.25 * (k % 2), backward)
        # in place, the columns behind stay
        y = x.clone()
        bfo.rotary_apply(y, f, y, positions=positions, layout=layout, backward=backward, amplitude=1.0 + 0.25 * (k % 2))
        assert torch.equal(y, out)


@pytest.mark.parametrize("half", [True, False])
def test_far_positions(bfo, half):
    for t in (torch.float32, torch.bfloat16):
        x, _ = inputs(3, 40, 3, 64, t)
        g = torch.Generator(device=DEV).manual_seed(4)
        positions = torch.randint(0, 1 << 31, (40,), generator=g, device=DEV).to(torch.int32)
        positions[0], positions[1], positions[2], positions[3] = 0, 2 ** 31 - 1, -2 ** 31, 10 ** 6
        f = bfo.rotary_frequencies(64, device=DEV)
        out = torch.empty_like(x)
        bfo.rotary_apply(x, f, out, positions=positions, layout=0 if half else 1)
        check_rotary(out, x, positions, f, half)
        assert torch.equal(out[0], x[0])


def test_positions_by_index_and_period(bfo):
    x, _ = inputs(5, 100, 4, 48, torch.float32)
    f = bfo.rotary_frequencies(48, device=DEV)
    out = torch.empty_like(x)
    index = torch.arange(100, device=DEV)
    bfo.rotary_apply(x, f, out)
    check_rotary(out, x, index, f, True)
    bfo.rotary_apply(x, f, out, period=32)
    check_rotary(out, x, index % 32, f, True)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("half", [True, False])
def test_strides(bfo, dt, half):
    """Queries and keys of one buffer that holds values too; heads outside, tokens inside; odd starts."""
    t, layout = TYPES[dt], 0 if half else 1
    f = bfo.rotary_frequencies(64, device=DEV)
    qkv, positions = inputs(6, 50, 16 + 4 + 4, 72, t)
    y = qkv.clone()
    bfo.rotary_apply(y[:, :20], f, y[:, :20], positions=positions, layout=layout)
    check_rotary(y[:, :20], qkv[:, :20], positions, f, half)
    assert torch.equal(y[:, 20:], qkv[:, 20:])
    out = torch.full((24, 50, 72), 7.0, dtype=t, device=DEV)          # heads x tokens x columns
    bfo.rotary_apply(qkv[:, :20], f, out[:20].transpose(0, 1), positions=positions, layout=layout)
    check_rotary(out[:20].transpose(0, 1), qkv[:, :20], positions, f, half)
    assert (out[20:] == 7).all()
    back = torch.empty(50, 20, 72, dtype=t, device=DEV)
    turned = out[:20].clone().transpose(0, 1)
    bfo.rotary_apply(turned, f, back, positions=positions, layout=layout, backward=True)
    check_rotary(back, turned, positions, f, half, backward=True)
    flat = torch.zeros(50 * 24 * 75 + 1, dtype=t, device=DEV)
    odd = flat[1:].view(50, 24, 75)[:, :, :72]
    odd.copy_(qkv)
    bfo.rotary_apply(odd, f, odd, positions=positions, layout=layout)
    check_rotary(odd, qkv, positions, f, half)
    assert (flat[1:].view(50, 24, 75)[:, :, 72:] == 0).all() and flat[0] == 0
    empty = torch.empty(0, 5, 72, dtype=t, device=DEV)
    bfo.rotary_apply(empty, f, empty)


def test_tokens_past_32_bit_offsets(bfo):
    tokens = (1 << 32) // 4096 + 10
    x = torch.zeros(tokens, 32, 128, dtype=torch.bfloat16, device=DEV)
    last, _ = inputs(7, 10, 32, 128, torch.bfloat16)
    x[-10:] = last
    f = bfo.rotary_frequencies(128, device=DEV)
    bfo.rotary_apply(x, f, x)
    check_rotary(x[-10:], last, torch.arange(tokens - 10, tokens, device=DEV), f, True)
    assert not x[:-10].any()
    del x
    torch.cuda.empty_cache()


def test_turning_back_is_the_inverse_and_the_transpose(bfo):
    """<turn(x), y> = <x, turn back(y)>, and turning back undoes turning."""
    x, positions = inputs(8, 30, 6, 64, torch.float32)
    y, _ = inputs(9, 30, 6, 64, torch.float32)
    f = bfo.rotary_frequencies(40, device=DEV)
    for layout in (0, 1):
        turned, back, again = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
        bfo.rotary_apply(x, f, turned, positions=positions, layout=layout)
        bfo.rotary_apply(y, f, back, positions=positions, layout=layout, backward=True)
        a, b = (turned.double() * y.double()).sum(), (x.double() * back.double()).sum()
        assert abs(a - b) <= 30 * 2.0 ** -24 * (turned.double() * y.double()).abs().sum()
        bfo.rotary_apply(turned, f, again, positions=positions, layout=layout, backward=True)
        assert (again - x).abs().max() <= 40 * 2.0 ** -24 * x.abs().max() * 2


@pytest.mark.parametrize("half", [True, False])
def test_large_calls(bfo, half):
    """Calls that pass through the caches are loaded and stored another way."""
    for t, dim, rotated in ((torch.bfloat16, 128, 128), (torch.float32, 80, 60), (torch.bfloat16, 100, 50)):
        x, positions = inputs(dim, 5000, 80, dim, t)
        f = bfo.rotary_frequencies(rotated, device=DEV)
        out = torch.empty_like(x)
        bfo.rotary_apply(x, f, out, positions=positions, layout=0 if half else 1)
        check_rotary(out, x, positions, f, half)
        bfo.rotary_apply(x, f, x, positions=positions, layout=0 if half else 1)
        assert torch.equal(x, out)


def test_more_work_than_workgroups(bfo):
    """Above 2^22 pieces of work the workgroups take several turns."""
    tokens = (1 << 26) + 50
    x = torch.zeros(tokens, 1, 256, dtype=torch.bfloat16, device=DEV)
    last, _ = inputs(11, 50, 1, 256, torch.bfloat16)
    x[-50:] = last
    f = bfo.rotary_frequencies(256, device=DEV)
    bfo.rotary_apply(x, f, x, period=1 << 20)
    check_rotary(x[-50:], last, torch.arange(tokens - 50, tokens, device=DEV) % (1 << 20), f, True)
    assert not x[:-50].any()                      # zeros of either sign
    del x
    torch.cuda.empty_cache()


@pytest.mark.parametrize("backward", [False, True])
def test_small_sines_and_cosines_keep_their_digits(bfo, backward):
    """Near whole quarters of a turn, relative to themselves: sine or cosine is off by two steps (four roundings), the
    sum with what the turn's rounding left by one, and that part, below 2^-23, by a few roundings of its own; the
    angle's two roundings in 64 bits are below 2^-50."""
    g = torch.Generator(device=DEV).manual_seed(14)
    off = 10.0 ** (-7.5 + 5.5 * torch.rand(512, generator=g, device=DEV, dtype=torch.float64))
    quarter = 0.25 * (1 + torch.arange(512, device=DEV) % 3)
    f = 2 * math.pi * (quarter + off * (1 - 2 * (torch.arange(512, device=DEV) // 3 % 2)))
    x = torch.zeros(2, 1, 1024, device=DEV)
    x[:, :, :512] = 1.0                                    # pairs (1, 0) become (cos, sin)
    out = torch.empty_like(x)
    positions = torch.tensor([1, -1], dtype=torch.int32, device=DEV)
    bfo.rotary_apply(x, f, out, positions=positions, backward=backward)
    angle = positions.double()[:, None] * f * (-1 if backward else 1)
    ref = torch.cat([torch.cos(angle), torch.sin(angle)], 1)[:, None]
    assert ((out.double() - ref).abs() <= 6 * 2.0 ** -24 * ref.abs() + 1e-13).all()


def test_periods_past_64_bits_are_not_their_low_words(bfo):
    x, _ = inputs(15, 100, 2, 16, torch.float32)
    f = bfo.rotary_frequencies(16, device=DEV)
    want, out = torch.empty_like(x), torch.empty_like(x)
    bfo.rotary_apply(x, f, want)
    for period in (101, (1 << 64) - 1, 1 << 64, (1 << 64) + 5):
        bfo.rotary_apply(x, f, out, period=period)
        assert torch.equal(out, want), period
