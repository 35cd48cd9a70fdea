"""The feed-forward's activation on the GPU, its inputs kept in 8 bits, and
codes by themselves, against their definitions in 64 bits."""
import pytest
import torch

from block_reference import CODES, DEV, SMALLEST, TOP, TYPES, U, activation, check, \
    check_activation_backward, check_activation_forward, check_codes, check_rounded, empty, matrix, normal, untouched, values

pytestmark = pytest.mark.gpu
SHAPES = [(1, 1), (3, 1), (1, 11008), (7, 2), (5, 15), (33, 16), (17, 31), (40, 127), (16, 128), (19, 129), (9, 511),
          (1003, 801), (5, 1025), (37, 1600), (3, 2049), (11, 4096), (2, 8200), (2, 33000), (4099, 40)]


@pytest.fixture(scope="module")
def bfo():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from bf16_numerics_amd import binding
    torch.cuda.set_device(0)
    return binding


def generator(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def codes_for(bfo, rows, cols, kind, pad=0):
    scales = bfo.new_codes(rows, cols, DEV, CODES[kind])[1].fill_(float("nan"))
    return empty(rows, cols, CODES[kind], pad), scales


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("gated", [True, False])
@pytest.mark.parametrize("keep", [None, "i8", "e4m3"])
def test_forward_and_backward_sizes(bfo, dt, kind, gated, keep):
    for k, (rows, cols) in enumerate(SHAPES):
        print(rows, cols, flush=True)
        g, t, pad = generator(100 + k), TYPES[dt], k % 4
        gate = matrix(g, rows, cols, t, pad, size=2.0)
        up = matrix(g, rows, cols, t, k % 3) if gated else None
        out, kept = empty(rows, cols, t, pad), {}
        if keep:
            kept["gate_codes"], kept["gate_scales"] = codes_for(bfo, rows, cols, keep, pad)
            if gated:
                kept["up_codes"], kept["up_scales"] = codes_for(bfo, rows, cols, keep, k % 3)
        bfo.activation_forward(gate, up, out, kind=kind, **kept)
        check_activation_forward(kind, gate, up, out)
        assert untouched(out)
        G, H, off = gate.double(), up.double() if gated else None, 0
        if keep:
            check_codes(kept["gate_codes"], kept["gate_scales"], G, 0, "gate")
            assert untouched(kept["gate_codes"])
            G, off = values(kept["gate_codes"], kept["gate_scales"]), 1
            if gated:
                check_codes(kept["up_codes"], kept["up_scales"], H, 0, "up")
                assert untouched(kept["up_codes"])
                H = values(kept["up_codes"], kept["up_scales"])
        d = matrix(g, rows, cols, t, pad, size=0.01)
        dgate, dup = empty(rows, cols, t, pad), empty(rows, cols, t, pad) if gated else None
        again = empty(rows, cols, t, pad) if k % 2 else None
        bfo.activation_backward(d, None if keep else gate, None if keep else up, dgate, dup, kind=kind, out=again, **kept)
        check_activation_backward(kind, d, G, H, dgate, dup, again, off)
        assert all(x is None or untouched(x) for x in (dgate, dup, again))


@pytest.mark.parametrize("kind", [0, 1])
def test_outputs_may_be_inputs(bfo, kind):
    """Columns of one fused buffer, gradients over the inputs, the output over the incoming gradient."""
    g, t, F = generator(3), torch.bfloat16, 1111
    both, d = matrix(g, 50, 2 * F, t), matrix(g, 50, F, t)
    gate, up = both[:, :F], both[:, F:]
    for place in ("gate", "up"):
        b = both.clone()
        bfo.activation_forward(b[:, :F], b[:, F:], b[:, :F] if place == "gate" else b[:, F:], kind=kind)
        check_activation_forward(kind, gate, up, b[:, :F] if place == "gate" else b[:, F:])
        assert torch.equal(b[:, F:], up) if place == "gate" else torch.equal(b[:, :F], gate)
    b, over = both.clone(), d.clone()
    bfo.activation_backward(over, b[:, :F], b[:, F:], b[:, :F], b[:, F:], kind=kind, out=over)
    check_activation_backward(kind, d, gate.double(), up.double(), b[:, :F], b[:, F:], over)
    b, over = both.clone(), d.clone()
    bfo.activation_backward(over, b[:, :F], b[:, F:], over, b[:, :F], kind=kind, out=b[:, F:])
    check_activation_backward(kind, d, gate.double(), up.double(), over, b[:, :F], b[:, F:])


@pytest.mark.parametrize("kind", [0, 1])
def test_far_and_special_values(bfo, kind):
    """Where sigma is 0 or 1 the activation is 0 or g and its derivative 0 or 1, however far g is; NaN stays in place."""
    g = torch.tensor([[0.0, -0.0, 1e-30, -1e-30, 30.0, -30.0, 88.0, -88.0, 200.0, -200.0, 1e10, -1e10, 3e19, -3e19, 3e38,
                       -3e38, float("inf"), float("nan"), 1.0, 2.0]], device=DEV)
    out, dg = torch.empty_like(g), torch.empty_like(g)
    one = torch.ones_like(g)
    bfo.activation_forward(g, None, out, kind=kind)
    bfo.activation_backward(one, g, None, dg, None, kind=kind)
    for k, v in enumerate(g[0].tolist()):
        if v != v:
            assert out[0, k].isnan() and dg[0, k].isnan()
        elif v == float("inf"):
            assert out[0, k] == v
        elif abs(v) >= 200:
            assert out[0, k] == (v if v > 0 else 0) and dg[0, k] == (1 if v > 0 else 0), v
    near = [k for k, v in enumerate(g[0].tolist()) if abs(v) < 200]
    check_activation_forward(kind, g[:, near], None, out[:, near])
    check_activation_backward(kind, one[:, near], g[:, near].double(), None, dg[:, near], None)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["i8", "e4m3"])
def test_pack_and_unpack(bfo, dt, kind):
    for k, (rows, cols) in enumerate(SHAPES):
        g, t, pad = generator(500 + k), TYPES[dt], k % 4
        x = matrix(g, rows, cols, t, pad)
        codes, scales = codes_for(bfo, rows, cols, kind, pad)
        bfo.activation_pack(x, codes, scales)
        check_codes(codes, scales, x.double(), 0, "pack")
        out = empty(rows, cols, t, pad)
        bfo.activation_unpack(codes, scales, out)
        check_rounded(out, values(codes, scales), U * values(codes, scales).abs(), "unpack")
        assert untouched(codes) and untouched(out)
        whole = torch.rand(rows, 1, generator=g, device=DEV) + 0.5
        if cols > 128:
            bfo.activation_unpack(codes, whole, out)
            ref = codes.double() * whole.double()
            check_rounded(out, ref, U * ref.abs(), "unpack by rows")


@pytest.mark.parametrize("kind", ["i8", "e4m3"])
def test_codes_of_extremes(bfo, kind):
    """Zeros, the smallest and largest numbers, ties, NaN and infinities; each group is its own."""
    top = TOP[CODES[kind]]
    x = torch.zeros(10, 256, device=DEV)
    x[1, :128] = 2.0 ** -140 * torch.arange(128, device=DEV)
    x[2, :128] = 3.4e38 * torch.linspace(-1, 1, 128, device=DEV)
    x[3, 3], x[3, 7] = float("nan"), 5.0
    x[4, 3], x[4, 7] = float("inf"), 5.0
    x[5, 130] = -float("inf")
    x[6, :128] = torch.arange(-63, 65, device=DEV) + 0.5      # int8 steps of 64.5 / 127
    x[7, 0], x[7, 1] = top, 2.5                               # a scale of 1: a tie of the integers
    x[8, 5] = -1e-45
    x[9] = 1.0
    codes, scales = codes_for(bfo, 10, 256, kind)
    bfo.activation_pack(x, codes, scales)
    keep = [0, 1, 2, 6, 7, 8, 9]
    a = x.double()[keep] / scales.double()[keep].repeat_interleave(128, 1)
    half = 0.5 if kind == "i8" else (a.abs() * 2.0 ** -4).clamp(min=2.0 ** -10)
    assert ((codes.double()[keep] - a).abs() <= half + a.abs() * 3 * U).all()
    assert (scales[0] == SMALLEST).all() and (codes[0].float() == 0).all()
    assert scales[1, 0] == SMALLEST and scales[8, 0] == SMALLEST
    v = values(codes, scales)
    assert v[3, :128].isnan().all() and (v[3, 128:] == 0).all()
    assert v[4, :128].isnan().all() and v[5, 128:].isnan().all() and (v[5, :128] == 0).all()
    assert (codes[9].float() == top).all()
    out = torch.empty_like(x)
    bfo.activation_unpack(codes, scales, out)
    assert torch.equal(out.isnan(), v.isnan())
    assert out[2].isfinite().all()
    check_rounded(out.nan_to_num(), v.nan_to_num(), U * v.nan_to_num().abs(), "unpack")
    bf = torch.full((1, 128), torch.finfo(torch.bfloat16).max, dtype=torch.bfloat16, device=DEV)
    codes, scales = codes_for(bfo, 1, 128, kind)
    bfo.activation_pack(bf, codes, scales)
    back = torch.empty_like(bf)
    bfo.activation_unpack(codes, scales, back)
    assert (back == bf).all()


def test_codes_do_not_depend_on_the_start(bfo):
    """The same rows at every byte of a line, in the buffers of both sides."""
    g = generator(21)
    x = matrix(g, 6, 300, torch.bfloat16)
    want, scales = bfo.new_codes(6, 300, DEV)
    bfo.activation_pack(x, want, scales)
    for at in range(9):
        wide = torch.zeros(6, 320, dtype=torch.bfloat16, device=DEV)
        wide[:, at:at + 300] = x
        room = torch.full((6, 317), 77, dtype=torch.int8, device=DEV)
        s = torch.empty_like(scales)
        bfo.activation_pack(wide[:, at:at + 300], room[:, at:at + 300], s)
        assert torch.equal(room[:, at:at + 300], want) and torch.equal(s, scales)
        assert (room[:, :at] == 77).all() and (room[:, at + 300:] == 77).all()
        out = torch.empty(6, 300, dtype=torch.bfloat16, device=DEV)
        bfo.activation_unpack(room[:, at:at + 300], s, out)
        check_rounded(out, values(want, scales), U * values(want, scales).abs(), "unpack")


def test_rows_past_32_bit_offsets(bfo):
    """The last rows of matrices whose element offsets pass 2^32."""
    cols, t = 4096, torch.bfloat16
    rows = (1 << 32) // cols + 100
    g = generator(62)
    x, d = matrix(g, 100, cols, t), matrix(g, 100, cols, t, size=0.01)
    big = torch.zeros(rows, cols, dtype=t, device=DEV)
    big[-100:] = x
    out = torch.empty_like(big)
    codes, scales = bfo.new_codes(rows, cols, DEV)
    bfo.activation_forward(big, None, out, kind=bfo.GELU, gate_codes=codes, gate_scales=scales)
    check_activation_forward(1, x, None, out[-100:])
    check_codes(codes[-100:], scales[-100:], x.double(), 0, "gate")
    assert not out[:-100].any() and not codes[:-100].any()
    big.zero_()
    big[-100:] = d
    bfo.activation_backward(big, None, None, out, None, kind=bfo.GELU, gate_codes=codes, gate_scales=scales)
    check_activation_backward(1, d, values(codes[-100:], scales[-100:]), None, out[-100:], None, off=1)
    assert not out[:-100].any()
    del big, out, codes, scales
    torch.cuda.empty_cache()


@pytest.mark.parametrize("kind", [0, 1])
def test_gradient_against_differences(bfo, kind):
    g = generator(8)
    gate, up, d = (matrix(g, 4, 500, torch.float32, size=1.5) for _ in range(3))
    dg, du = torch.empty_like(gate), torch.empty_like(gate)
    bfo.activation_backward(d, gate, up, dg, du, kind=kind)

    def out(a, b):
        return activation(kind, a)[0] * b
    h, G, H, D = 1e-4, gate.double(), up.double(), d.double()
    # third derivatives of the activations are below 4
    tol = 4 * h * h * (D * H).abs() + 40 * U * (D * H).abs() * (1 + G.abs()) ** 3 + 1e-10
    assert ((dg.double() - D * (out(G + h, H) - out(G - h, H)) / (2 * h)).abs() <= tol).all()
    assert ((du.double() - D * (out(G, H + h) - out(G, H - h)) / (2 * h)).abs() <= 40 * U * (D * G).abs() + 1e-10).all()


def test_codes_kept_for_the_backward_pass_cost_what_their_step_is(bfo):
    """Gradients from codes against those from the inputs: a code moves an input by half a step at most, and the
    derivative moves by at most 1.2 times that (SiLU's second derivative is at most 1/2, GELU's 0.8 and 1.2)."""
    g = generator(12)
    gate, d = matrix(g, 64, 1024, torch.float32), normal(g, 64, 1024)
    codes, scales = bfo.new_codes(64, 1024, DEV)
    out, dg = torch.empty_like(gate), torch.empty_like(gate)
    for kind in (0, 1):
        bfo.activation_forward(gate, None, out, kind=kind, gate_codes=codes, gate_scales=scales)
        bfo.activation_backward(d, None, None, dg, None, kind=kind, gate_codes=codes, gate_scales=scales)
        exact = d.double() * activation(kind, gate.double())[1]
        half = scales.double().repeat_interleave(128, 1) / 2
        assert ((dg.double() - exact).abs() <= d.double().abs() * (1.2 * half * (1 + 1e-5) + 60 * U)).all()


@pytest.mark.parametrize("cols", [1, 128])
def test_more_groups_than_workgroups(bfo, cols):
    """Above 2^26 groups the workgroups take several turns."""
    rows = (1 << 26) + 40 if cols == 1 else 1 << 20
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device=DEV)
    x[-64:] = matrix(generator(2), 64, cols, torch.bfloat16)
    codes, scales = bfo.new_codes(rows, cols, DEV)
    out = torch.empty_like(x)
    bfo.activation_forward(x, None, out, gate_codes=codes, gate_scales=scales)
    check_activation_forward(0, x[-64:], None, out[-64:])
    check_codes(codes[-64:], scales[-64:], x[-64:].double(), 0, "gate")
    assert not out[:-64].any() and not codes[:-64].any() and (scales[:-64] == SMALLEST).all()
    del x, codes, scales, out
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("gated", [True, False])
def test_large_calls(bfo, dt, gated):
    """Calls that pass through the caches are loaded and stored another way; widths of whole chunks and others."""
    for cols in (4096, 4100, 4099):
        rows = 6000 if dt == "bf16" else 3000
        g, t = generator(cols), TYPES[dt]
        gate, d = matrix(g, rows, cols, t, size=2.0), matrix(g, rows, cols, t, size=0.01)
        up = matrix(g, rows, cols, t) if gated else None
        out = torch.empty_like(gate)
        kept = {}
        kept["gate_codes"], kept["gate_scales"] = codes_for(bfo, rows, cols, "i8")
        if gated:
            kept["up_codes"], kept["up_scales"] = codes_for(bfo, rows, cols, "i8")
        bfo.activation_forward(gate, up, out, **kept)
        check_activation_forward(0, gate, up, out)
        G = values(kept["gate_codes"], kept["gate_scales"])
        H = values(kept["up_codes"], kept["up_scales"]) if gated else None
        check_codes(kept["gate_codes"], kept["gate_scales"], gate.double(), 0, "gate")
        dgate, dup, again = torch.empty_like(gate), torch.empty_like(gate) if gated else None, torch.empty_like(gate)
        bfo.activation_backward(d, None, None, dgate, dup, out=again, **kept)
        check_activation_backward(0, d, G, H, dgate, dup, again, 1)
        bfo.activation_backward(d, gate, up, dgate, dup, out=again)
        check_activation_backward(0, d, gate.double(), up.double() if gated else None, dgate, dup, again)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["i8", "e4m3"])
def test_codes_of_a_matrix_as_it_is_are_the_definition_bit_for_bit(bfo, dt, kind):
    """Every step of the definition is one binary32 operation, so there is nothing to tolerate."""
    for rows, cols in ((300, 1000), (64, 4096), (7, 129), (5, 3)):
        x = matrix(generator(cols), rows, cols, TYPES[dt])
        codes, scales = codes_for(bfo, rows, cols, kind)
        bfo.activation_pack(x, codes, scales)
        wide = torch.nn.functional.pad(x.float(), (0, -cols % 128)).view(rows, -1, 128)
        want = (wide.abs().amax(2) * torch.tensor(1 / TOP[CODES[kind]], device=DEV)).clamp(min=SMALLEST)
        v = (wide * (1 / want)[:, :, None]).view(rows, -1)[:, :cols]
        assert torch.equal(scales, want)
        assert torch.equal(codes.float(), (v.round() if kind == "i8" else v.to(CODES[kind]).float()))


@pytest.mark.parametrize("kind", [0, 1])
def test_negative_gates_keep_their_digits(bfo, kind):
    """fp32 results relative to themselves, however small: z's exponential is off by two roundings and the one
    that takes in what its exponent's rounding left, their sum by one, the reciprocal by two and the product with
    the gate by one; none of them grows with |z|.  (Down to z = -85 nothing is below 2^-126.)"""
    g, low = generator(77), (80.0, 9.8)[kind]
    gate = -low * torch.rand(64, 1000, generator=g, device=DEV)
    gate[0] = -torch.linspace(0, low, 1000, device=DEV)
    up, d = (normal(g, 64, 1000) for _ in range(2))
    out, dg, du, plain = (torch.empty_like(gate) for _ in range(4))
    G, H, D = gate.double(), up.double(), d.double()
    act, slope, s, t, z, dz = activation(kind, G)
    rel = (3 * t + 4) * U
    # the derivative: sigma, act * (1 - sigma) * dz with five roundings of dz and two products, and their sum
    off = s * rel + (act * t * dz).abs() * (rel + 9 * U) + (act * dz).abs() * (s * rel + U) + U * slope.abs()
    bfo.activation_forward(gate, None, plain, kind=kind)
    check(plain, act, act.abs() * (rel + U), "out")
    bfo.activation_forward(gate, up, out, kind=kind)
    check(out, act * H, (act * H).abs() * (rel + 2 * U), "gated out")
    bfo.activation_backward(d, gate, up, dg, du, kind=kind, out=out)
    check(dg, D * H * slope, (D * H).abs() * (off + 2 * U * slope.abs()), "dgate")
    check(du, D * act, (D * act).abs() * (rel + 2 * U), "dup")
    check(out, act * H, (act * H).abs() * (rel + 2 * U), "out again")
    bfo.activation_backward(d, gate, None, dg, None, kind=kind)
    check(dg, D * slope, D.abs() * (off + U * slope.abs()), "dgate without up")


@pytest.mark.parametrize("cols", [8, 9])
def test_more_groups_than_workgroups_of_whole_and_ragged_rows(bfo, cols):
    """Above 2^26 groups the workgroups take several turns: rows of one group, of whole chunks and not, forward,
    backward from the codes and from the inputs, and the codes' values."""
    rows, t, g = (1 << 26) + 40, torch.bfloat16, generator(4)
    x = torch.zeros(rows, cols, dtype=t, device=DEV)
    x[-64:] = matrix(g, 64, cols, t)
    d = torch.zeros(rows, cols, dtype=t, device=DEV)
    d[-64:] = matrix(g, 64, cols, t, size=0.01)
    codes, scales = bfo.new_codes(rows, cols, DEV)
    out = torch.full_like(x, 3.0)
    bfo.activation_forward(x, None, out, gate_codes=codes, gate_scales=scales)
    check_activation_forward(0, x[-64:], None, out[-64:])
    check_codes(codes[-64:], scales[-64:], x[-64:].double(), 0, "gate")
    assert not out[:-64].any() and not codes[:-64].any() and (scales[:-64] == SMALLEST).all()
    kept = values(codes[-64:], scales[-64:])
    for coded in (True, False):
        out.fill_(3.0)
        bfo.activation_backward(d, None if coded else x, None, out, None, gate_codes=codes if coded else None,
                                gate_scales=scales if coded else None)
        check_activation_backward(0, d[-64:], kept if coded else x[-64:].double(), None, out[-64:], None, off=int(coded))
        assert not out[:-64].any()
    out.fill_(3.0)
    bfo.activation_unpack(codes, scales, out)
    check_rounded(out[-64:], kept, U * kept.abs(), "unpack")
    assert not out[:-64].any()
    del x, d, codes, scales, out
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("gated", [True, False])
@pytest.mark.parametrize("keep", ["i8", "e4m3"])
def test_large_calls_of_every_kind(bfo, dt, kind, gated, keep):
    """128 MB and more forward and backward, whole chunks (nontemporal) and not; packed and unpacked too."""
    for cols in (4096, 4099):
        rows = 8200 if dt == "bf16" else 4200
        g, t = generator(cols), TYPES[dt]
        gate, d = matrix(g, rows, cols, t, size=2.0), matrix(g, rows, cols, t, size=0.01)
        up = matrix(g, rows, cols, t) if gated else None
        out, kept = torch.empty_like(gate), {}
        kept["gate_codes"], kept["gate_scales"] = codes_for(bfo, rows, cols, keep)
        if gated:
            kept["up_codes"], kept["up_scales"] = codes_for(bfo, rows, cols, keep)
        bfo.activation_forward(gate, up, out, kind=kind, **kept)
        check_activation_forward(kind, gate, up, out)
        check_codes(kept["gate_codes"], kept["gate_scales"], gate.double(), 0, "gate")
        G, H = values(kept["gate_codes"], kept["gate_scales"]), None
        if gated:
            check_codes(kept["up_codes"], kept["up_scales"], up.double(), 0, "up")
            H = values(kept["up_codes"], kept["up_scales"])
        dgate, dup, again = torch.empty_like(gate), torch.empty_like(gate) if gated else None, torch.empty_like(gate)
        bfo.activation_backward(d, None, None, dgate, dup, kind=kind, out=again, **kept)
        check_activation_backward(kind, d, G, H, dgate, dup, again, 1)
        codes, scales = codes_for(bfo, rows, cols, keep)
        bfo.activation_pack(gate, codes, scales)
        assert torch.equal(codes.view(torch.int8), kept["gate_codes"].view(torch.int8))
        assert torch.equal(scales, kept["gate_scales"])
        bfo.activation_unpack(codes, scales, again)
        check_rounded(again, G, U * G.abs(), "unpack")
