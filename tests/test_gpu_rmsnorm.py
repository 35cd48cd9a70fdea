"""RMS norm on the GPU, with the residual's addition and 8-bit codes, against its
definition in 64 bits."""
import pytest
import torch

from block_reference import CODES, DEV, TYPES, U, check_rms_backward, check_rms_forward, empty, matrix, normal, untouched, \
    values

pytestmark = pytest.mark.gpu
COMBOS = [("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16"), ("f32", "f32")]
SHAPES = [(1, 1), (3, 1), (1, 768), (7, 2), (5, 15), (33, 16), (17, 31), (64, 32), (40, 127), (16, 128), (19, 129), (9, 511),
          (8, 512), (21, 513), (1003, 801), (12, 1024), (5, 1025), (37, 1600), (6, 2047), (4, 2048), (3, 2049),
          (11, 4096), (2, 4099), (5, 8191), (3, 8192), (2, 8200), (3, 16383), (2, 16384), (4099, 40)]


@pytest.fixture(scope="module")
def bfo():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from bf16_numerics_amd import binding
    torch.cuda.set_device(0)
    return binding


def generator(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def weights(g, cols, pdt):
    return (1 + 0.2 * normal(g, cols)).to(pdt)


def codes_for(bfo, rows, cols, kind, per_row=False, pad=0):
    codes, scales = bfo.new_codes(rows, cols, DEV, CODES[kind], per_row)
    scales.fill_(float("nan"))
    return empty(rows, cols, CODES[kind], pad), scales


@pytest.mark.parametrize("dt,pdt", COMBOS)
def test_forward_sizes(bfo, dt, pdt):
    for k, (rows, cols) in enumerate(SHAPES):
        print(dt, pdt, rows, cols, flush=True)
        g, t, pad = generator(100 + k), TYPES[dt], k % 3
        x, w = matrix(g, rows, cols, t, pad), weights(g, cols, TYPES[pdt])
        residual = matrix(g, rows, cols, t, pad) if k % 2 else None
        total = empty(rows, cols, t, pad) if k % 4 == 1 else None
        out, rstd = empty(rows, cols, t, pad), torch.full((rows,), float("nan"), device=DEV)
        bfo.rmsnorm_forward(x, w, out, residual=residual, total=total, rstd=rstd)
        check_rms_forward(x, residual, w, 1e-5, total, out, rstd)
        assert untouched(out) and (total is None or untouched(total))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["i8", "e4m3"])
@pytest.mark.parametrize("per_row", [False, True])
@pytest.mark.parametrize("of_out", [False, True])
def test_forward_codes(bfo, dt, kind, per_row, of_out):
    for k, (rows, cols) in enumerate(SHAPES):
        print(rows, cols, flush=True)
        g, t, pad = generator(200 + k), TYPES[dt], k % 4
        x, w = matrix(g, rows, cols, t), weights(g, cols, t)
        residual = matrix(g, rows, cols, t) if k % 2 else None
        codes, scales = codes_for(bfo, rows, cols, kind, per_row, pad)
        out = empty(rows, cols, t) if k % 3 else None
        bfo.rmsnorm_forward(x, w, out, residual=residual, codes=codes, scales=scales,
                            codes_of=bfo.CODES_OF_OUT if of_out else bfo.CODES_OF_NORMALISED)
        check_rms_forward(x, residual, w, 1e-5, None, out, None, codes, scales, of_out)
        assert untouched(codes)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_total_may_be_an_input_and_columns_of_one_buffer(bfo, dt):
    g, t = generator(5), TYPES[dt]
    x, r, w = matrix(g, 37, 1100, t), matrix(g, 37, 1100, t), weights(g, 1100, t)
    for place in ("x", "residual", "columns"):
        a, b = x.clone(), r.clone()
        wide = torch.full((37, 3000), 7.0, dtype=t, device=DEV)
        total = {"x": a, "residual": b, "columns": wide[:, 100:1200]}[place]
        out = wide[:, 1800:2900]
        bfo.rmsnorm_forward(a, w, out, residual=b, total=total)
        check_rms_forward(x, r, w, 1e-5, total, out)
        assert (wide[:, 1200:1800] == 7).all() and (wide[:, 2900:] == 7).all() and (wide[:, :100] == 7).all()
    # no rows, and a weight on an odd element of a buffer
    e = torch.empty(0, 1100, dtype=t, device=DEV)
    bfo.rmsnorm_forward(e, w, torch.empty_like(e))
    flat = torch.zeros(1101, dtype=t, device=DEV)
    flat[1:] = w
    out = torch.empty(37, 1100, dtype=t, device=DEV)
    bfo.rmsnorm_forward(x, flat[1:], out)
    check_rms_forward(x, None, w, 1e-5, None, out)


@pytest.mark.parametrize("kind", ["i8", "e4m3"])
def test_rows_of_zeros_nan_infinity_and_extremes(bfo, kind):
    """Each stays its row's own; codes of a row with a NaN read back as NaN."""
    g = generator(6)
    x, w = matrix(g, 9, 400, torch.float32).clone(), weights(g, 400, torch.float32)
    x[1] = 0
    x[2, 17] = float("nan")
    x[3, 399] = float("inf")
    x[4] *= 1e-30
    x[5] *= 1e15
    x[6, 5] = -float("inf")
    out, rstd = empty(9, 400, torch.float32), empty(1, 9, torch.float32)[0]
    codes, scales = codes_for(bfo, 9, 400, kind)
    bfo.rmsnorm_forward(x, w, out, rstd=rstd, codes=codes, scales=scales)
    keep = [0, 1, 4, 5, 7, 8]
    check_rms_forward(x[keep], None, w, 1e-5, None, out[keep], rstd[keep], codes[keep], scales[keep])
    assert (out[1] == 0).all() and (values(codes, scales)[1] == 0).all()
    assert out[2].isnan().all() and rstd[2].isnan() and values(codes, scales)[2].isnan().all()
    for row, col in ((3, 399), (6, 5)):
        assert rstd[row] == 0 and out[row, col].isnan()
        v = values(codes, scales)[row]
        group = slice(col // 128 * 128, min(400, col // 128 * 128 + 128))
        assert v[group].isnan().all()
        rest = torch.ones(400, dtype=torch.bool, device=DEV)
        rest[group] = False
        assert (v[rest] == 0).all()
        rest[:] = True
        rest[col] = False
        assert (out[row][rest] == 0).all()


def run_backward(bfo, d, x, w, rstd, pad=0, again=True, **kw):
    rows, cols = d.shape
    dx, out = empty(rows, cols, d.dtype, pad), empty(rows, cols, d.dtype, pad) if again else None
    dw = torch.full((cols,), float("nan"), dtype=w.dtype, device=DEV)
    ws = torch.full_like(bfo.new_rmsnorm_workspace(rows, cols, DEV), 255)    # NaN patterns
    bfo.rmsnorm_backward(d, x, w, rstd, dx, dw, out=out, workspace=ws, **kw)
    assert untouched(dx) and (out is None or untouched(out))
    return dx, dw, out


def rstd_of(x, eps=1e-5):
    return (1 / torch.sqrt(x.double().square().mean(1) + eps)).float()


MORE = [(2048, 64), (2049, 768), (5000, 33), (512, 300), (513, 300), (511, 2049), (700, 9000), (1024, 801), (2048, 801),
        (2049, 801), (2047, 2048), (1024, 2049), (1025, 2049), (512, 4097), (513, 4097), (3000, 1600)]


@pytest.mark.parametrize("dt,pdt", COMBOS)
def test_backward_sizes(bfo, dt, pdt):
    for k, (rows, cols) in enumerate(SHAPES + MORE):
        print(dt, pdt, rows, cols, flush=True)
        g, t, pad = generator(300 + k), TYPES[dt], k % 3
        x, d, w = matrix(g, rows, cols, t, pad), matrix(g, rows, cols, t, pad, size=0.01), weights(g, cols, TYPES[pdt])
        rstd = rstd_of(x)
        dx, dw, out = run_backward(bfo, d, x, w, rstd, pad, again=k % 2)
        check_rms_backward(d, x.double() * rstd.double()[:, None], w, rstd, dx, dw, out)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["i8", "e4m3"])
@pytest.mark.parametrize("per_row", [False, True])
def test_backward_from_codes(bfo, dt, kind, per_row):
    for k, (rows, cols) in enumerate(SHAPES + MORE):
        print(rows, cols, flush=True)
        g, t, pad = generator(400 + k), TYPES[dt], k % 4
        x, d, w = matrix(g, rows, cols, t), matrix(g, rows, cols, t, pad, size=0.01), weights(g, cols, t)
        codes, scales = codes_for(bfo, rows, cols, kind, per_row, pad)
        rstd = torch.empty(rows, device=DEV)
        bfo.rmsnorm_forward(x, w, rstd=rstd, codes=codes, scales=scales)
        dx, dw, out = run_backward(bfo, d, None, w, rstd, pad, again=k % 3, codes=codes, scales=scales)
        check_rms_backward(d, values(codes, scales), w, rstd, dx, dw, out)


@pytest.mark.parametrize("dt,pdt", COMBOS)
@pytest.mark.parametrize("rows,cols", [(77, 96), (600, 1600), (5, 5000), (2100, 1600)])
def test_backward_accumulates(bfo, dt, pdt, rows, cols):
    g, t = generator(31), TYPES[dt]
    x, d, w = matrix(g, rows, cols, t), matrix(g, rows, cols, t, size=0.01), weights(g, cols, TYPES[pdt])
    rstd = rstd_of(x)
    old = [normal(g, rows, cols).to(t), normal(g, cols).to(TYPES[pdt])]
    ws = bfo.new_rmsnorm_workspace(rows, cols, DEV)
    for acc_dx in (False, True):
        for acc_p in (False, True):
            dx, dw = (o.clone() for o in old)
            bfo.rmsnorm_backward(d, x, w, rstd, dx, dw, workspace=ws, accumulate_dx=acc_dx, accumulate_params=acc_p)
            kept = [old[0] if acc_dx else torch.zeros_like(old[0]), old[1] if acc_p else torch.zeros_like(old[1])]
            check_rms_backward(d, x.double() * rstd.double()[:, None], w, rstd, dx, dw, old=kept)


def test_backward_without_rows_writes_zeros_or_keeps(bfo):
    e, w = torch.empty(0, 64, device=DEV), torch.ones(64, device=DEV)
    dw = torch.full((64,), 3.0, device=DEV)
    args = (e, e, w, torch.empty(0, device=DEV), torch.empty_like(e), dw)
    bfo.rmsnorm_backward(*args, accumulate_params=True)
    assert (dw == 3).all()
    bfo.rmsnorm_backward(*args)
    assert (dw == 0).all()


@pytest.mark.parametrize("rows,cols", [(20001, 520), (70003, 16), (9001, 2049)])
def test_more_rows_than_workgroups(bfo, rows, cols):
    g = generator(61)
    x, d, w = (matrix(g, rows, cols, torch.bfloat16) for _ in range(3))
    w = w[0].clone()
    out, rstd = empty(rows, cols, torch.bfloat16), torch.empty(rows, device=DEV)
    codes, scales = codes_for(bfo, rows, cols, "i8")
    bfo.rmsnorm_forward(x, w, out, rstd=rstd, codes=codes, scales=scales)
    check_rms_forward(x, None, w, 1e-5, None, out, rstd, codes, scales)
    dx, dw, again = run_backward(bfo, d, None, w, rstd, codes=codes, scales=scales)
    check_rms_backward(d, values(codes, scales), w, rstd, dx, dw, again)


def test_rows_past_32_bit_offsets(bfo):
    """The last rows of matrices whose element offsets pass 2^32."""
    cols, t = 4096, torch.bfloat16
    rows = (1 << 32) // cols + 100
    g = generator(62)
    x, d, w = matrix(g, 100, cols, t), matrix(g, 100, cols, t, size=0.01), weights(g, cols, t)
    big = torch.zeros(rows, cols, dtype=t, device=DEV)
    big[-100:] = x
    out, rstd = torch.empty_like(big), torch.empty(rows, device=DEV)
    codes, scales = bfo.new_codes(rows, cols, DEV)
    bfo.rmsnorm_forward(big, w, out, rstd=rstd, codes=codes, scales=scales)
    check_rms_forward(x, None, w, 1e-5, None, out[-100:], rstd[-100:], codes[-100:], scales[-100:])
    assert not out[:-100].any() and not codes[:-100].any()
    big.zero_()
    big[-100:] = d
    dw = torch.empty_like(w)
    bfo.rmsnorm_backward(big, None, w, rstd, out, dw, codes=codes, scales=scales,
                         workspace=bfo.new_rmsnorm_workspace(rows, cols, DEV))
    check_rms_backward(d, values(codes[-100:], scales[-100:]), w, rstd[-100:], out[-100:], dw)
    assert not out[:-100].any()
    del big, out, codes, scales
    torch.cuda.empty_cache()


def test_gradient_against_differences(bfo):
    """sum(dout * out) moves by sum(dx * step) and sum(dweight * step): its central difference in 64 bits of the
    definition, whose own error is of order step^2."""
    g = generator(8)
    x, d, w = matrix(g, 5, 700, torch.float32), matrix(g, 5, 700, torch.float32), weights(g, 700, torch.float32)
    rstd = rstd_of(x)
    dx, dw, _ = run_backward(bfo, d, x, w, rstd)

    def loss(X, W):
        return (d.double() * (X / torch.sqrt(X.square().mean(1, keepdim=True) + 1e-5)) * W).sum()
    vx, vw, h = normal(g, 5, 700).double(), normal(g, 700).double(), 1e-4
    X, W = x.double(), w.double()
    for got, diff, scale in (((dx.double() * vx).sum(), (loss(X + h * vx, W) - loss(X - h * vx, W)) / (2 * h),
                              (dx.double() * vx).abs().sum()),
                             ((dw.double() * vw).sum(), (loss(X, W + h * vw) - loss(X, W - h * vw)) / (2 * h),
                              (dw.double() * vw).abs().sum())):
        # binary32's share of the terms, and h^2 times third derivatives of the order of the loss
        assert abs(got - diff) <= 100 * U * scale + 100 * h * h * d.double().abs().sum()


def test_same_bits_on_other_streams_and_again(bfo):
    g = generator(9)
    x, d, w = (matrix(g, 3000, 768, torch.bfloat16) for _ in range(3))
    w, rstd = w[0].clone(), rstd_of(x)
    dx, dw, out = run_backward(bfo, d, x, w, rstd)
    torch.cuda.synchronize()
    for _ in range(3):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            again = run_backward(bfo, d, x, w, rstd)
        s.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(again, (dx, dw, out)))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_large_calls(bfo, dt):
    """Calls that pass through the caches are loaded and stored another way; widths of whole chunks and others."""
    for cols in (4096, 5000, 5003):
        rows = 6000 if dt == "bf16" else 3000
        g, t = generator(cols), TYPES[dt]
        x, r, d = (matrix(g, rows, cols, t) for _ in range(3))
        w = weights(g, cols, t)
        out, total, rstd = torch.empty_like(x), torch.empty_like(x), torch.empty(rows, device=DEV)
        codes, scales = codes_for(bfo, rows, cols, "i8")
        bfo.rmsnorm_forward(x, w, out, residual=r, total=total, rstd=rstd, codes=codes, scales=scales)
        check_rms_forward(x, r, w, 1e-5, total, out, rstd, codes, scales)
        check_rms_backward(d, values(codes, scales), w, rstd, *run_backward(bfo, d, None, w, rstd, codes=codes,
                                                                            scales=scales))
        check_rms_backward(d, total.double() * rstd.double()[:, None], w, rstd, *run_backward(bfo, d, total, w, rstd))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["i8", "e4m3"])
@pytest.mark.parametrize("per_row", [False, True])
@pytest.mark.parametrize("of_out", [False, True])
def test_large_calls_of_every_code(bfo, dt, kind, per_row, of_out):
    """128 MB and more: codes of either type and group, of the output or of the normalised row, and its gradient."""
    rows, cols, t = (6000 if dt == "bf16" else 3000), 4096, TYPES[dt]
    g = generator(71)
    x, r, d = (matrix(g, rows, cols, t) for _ in range(3))
    w = weights(g, cols, t)
    out, total, rstd = torch.empty_like(x), torch.empty_like(x), torch.empty(rows, device=DEV)
    codes, scales = codes_for(bfo, rows, cols, kind, per_row)
    bfo.rmsnorm_forward(x, w, out, residual=r, total=total, rstd=rstd, codes=codes, scales=scales,
                        codes_of=bfo.CODES_OF_OUT if of_out else bfo.CODES_OF_NORMALISED)
    check_rms_forward(x, r, w, 1e-5, total, out, rstd, codes, scales, of_out=of_out)
    if not of_out:
        check_rms_backward(d, values(codes, scales), w, rstd, *run_backward(bfo, d, None, w, rstd, codes=codes,
                                                                            scales=scales))
