"""Layer norm on the GPU against its definition in 64 bits.

Tolerances count roundings of half a step u = 2^-24 of binary32 along the
kernels' operation order, plus one rounding to the output's type
(eps / 2 relative).  A row's sums run over at most 64 terms per lane, 6 steps
of the wavefront and 7 more wavefronts: fewer than DEPTH = 80 additions, so a
sum of terms with absolute values t is off by at most DEPTH * u * sum(t).
"""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
DEPTH = 80
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def bfo():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from bf16_numerics_amd import binding
    torch.cuda.set_device(0)
    return binding


def rounding(t):
    """Half a step of the type, relative; 0 for binary32 results counted in u."""
    return torch.finfo(t).eps / 2 if t != torch.float32 else 0.0


def inputs(rows, cols, dt, pdt, seed, pad=0, offset=0.0):
    """x, dout (rows of a buffer `pad` columns wider), weight, bias."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    def normal(*shape):
        return torch.empty(shape, device=DEV).normal_(generator=g)
    x = torch.full((rows, cols + pad), float("nan"), dtype=dt, device=DEV)
    d = x.clone()
    x[:, :cols] = (normal(rows, cols) * torch.exp(0.5 * normal(cols)) + offset).to(dt)
    d[:, :cols] = (0.01 * normal(rows, cols)).to(dt)
    return x[:, :cols], d[:, :cols], (1 + 0.2 * normal(cols)).to(pdt), (0.1 * normal(cols)).to(pdt)


def check(got, ref, tol, what):
    got = got.double()
    assert got.shape == ref.shape
    bad = ~((got - ref).abs() <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float(((got - ref).abs() / tol).max())} " \
                          f"of the tolerance"


def check_forward(x, w, b, eps, out, mean, rstd):
    X, Wt = x.double(), w.double()
    B = b.double() if b is not None else torch.zeros_like(Wt)
    m = X.mean(1, keepdim=True)
    var = ((X - m) ** 2).mean(1, keepdim=True)
    r = 1 / torch.sqrt(var + eps)
    absmean = X.abs().mean(1, keepdim=True)
    em = (DEPTH + 3) * U * absmean                      # the mean
    # relative error of the variance: 2 em / sigma from the mean's error (it enters squared, with the
    # cross term summing to about 0, so this is generous), DEPTH additions, a few single roundings
    er = 0.5 * ((DEPTH + 8) * U + 2 * em * r) + 3 * U
    ref = (X - m) * r * Wt + B
    tol = Wt.abs() * (r * (em + U * (X - m).abs()) + (X - m).abs() * r * (er + 2 * U)) + 2 * U * ref.abs()
    check(out, ref, tol + rounding(out.dtype) * (ref.abs() + tol) + 1e-38, "out")
    if mean is not None:
        check(mean, m[:, 0], em[:, 0] + 1e-38, "mean")
    if rstd is not None:
        check(rstd, r[:, 0], (r * er)[:, 0], "rstd")


def run_forward(bfo, x, w, b, eps=1e-5, stats=True):
    out = torch.full((x.shape[0], x.shape[1]), float("nan"), dtype=x.dtype, device=DEV)
    mean = torch.full((x.shape[0],), float("nan"), device=DEV) if stats else None
    rstd = mean.clone() if stats else None
    bfo.layernorm_forward(x, w, b, out, mean, rstd, eps)
    return out, mean, rstd


SHAPES = [(1, 1), (3, 1), (1, 768), (7, 2), (5, 15), (33, 16), (17, 31), (64, 32), (40, 127), (16, 128), (19, 129),
          (9, 511), (8, 512), (21, 513), (1003, 801), (12, 1024), (5, 1025), (37, 1600), (6, 2047), (4, 2048),
          (3, 2049), (11, 4096), (2, 4099), (5, 8191), (3, 8192), (2, 8200), (3, 16383), (2, 16384), (4099, 40)]
COMBOS = [("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16"), ("f32", "f32")]


@pytest.mark.parametrize("dt,pdt", COMBOS)
def test_forward_sizes(bfo, dt, pdt):
    for k, (rows, cols) in enumerate(SHAPES):
        print(dt, pdt, rows, cols, flush=True)
        x, _, w, b = inputs(rows, cols, TYPES[dt], TYPES[pdt], 100 + k, pad=k % 3)
        out, mean, rstd = run_forward(bfo, x, w, b)
        check_forward(x, w, b, 1e-5, out, mean, rstd)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_forward_optional_arguments_strides_and_guards(bfo, dt):
    t = TYPES[dt]
    x, _, w, b = inputs(37, 100, t, t, 5, pad=3)
    out, mean, rstd = run_forward(bfo, x, w, None, stats=False)
    check_forward(x, w, None, 1e-5, out, None, None)
    # out as every other column block of the buffer that also holds x: neighbours stay as they were
    wide = torch.full((37, 300), 7.0, dtype=t, device=DEV)
    wide[:, :100] = x
    bfo.layernorm_forward(wide[:, :100], w, b, wide[:, 150:250], eps=1e-5)
    check_forward(x, w, b, 1e-5, wide[:, 150:250], None, None)
    assert torch.equal(wide[:, :100], x)
    assert (wide[:, 100:150] == 7).all() and (wide[:, 250:] == 7).all()
    # rows repeated through stride 0 are refused as input rows that overlap
    with pytest.raises(bfo.BfoError):
        bfo.layernorm_forward(x[:1].expand(4, 100), w, b, torch.empty(4, 100, dtype=t, device=DEV))
    # no rows at all
    e = torch.empty(0, 100, dtype=t, device=DEV)
    bfo.layernorm_forward(e, w, b, torch.empty_like(e))
    # a weight on an odd element of a buffer, as a tensor of the flat parameter buffer may be
    flat = torch.zeros(201, dtype=t, device=DEV)
    flat[1:101] = w
    flat[101:201] = b
    out2 = torch.empty(37, 100, dtype=t, device=DEV)
    bfo.layernorm_forward(x, flat[1:101], flat[101:201], out2)
    check_forward(x, w, b, 1e-5, out2, None, None)


@pytest.mark.parametrize("rows,cols", [(20001, 520), (70003, 16), (9001, 2049)])
def test_more_rows_than_workgroups(bfo, rows, cols):
    x, d, w, b = inputs(rows, cols, torch.bfloat16, torch.bfloat16, 61)
    out, mean, rstd = run_forward(bfo, x, w, b)
    check_forward(x, w, b, 1e-5, out, mean, rstd)
    check_backward(x, d, w, mean, rstd, *run_backward(bfo, x, d, w, mean, rstd))


def test_rows_past_32_bit_offsets(bfo):
    """The last rows of matrices whose element offsets pass 2^32."""
    cols = 4096
    rows = (1 << 32) // cols + 100
    big = torch.zeros(rows, cols, dtype=torch.bfloat16, device=DEV)
    x, d, w, b = inputs(100, cols, torch.bfloat16, torch.bfloat16, 62)
    big[-100:] = x
    out = torch.empty_like(big)
    mean, rstd = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    bfo.layernorm_forward(big, w, b, out, mean, rstd)
    check_forward(x, w, b, 1e-5, out[-100:], mean[-100:], rstd[-100:])
    assert (out[:-100] == b).all() and (mean[:-100] == 0).all()
    dout = torch.zeros_like(big)
    dout[-100:] = d
    dw, db = torch.empty_like(w), torch.empty_like(w)
    bfo.layernorm_backward(dout, big, w, mean, rstd, out, dw, db,
                           workspace=bfo.new_layernorm_workspace(rows, cols, DEV))
    # rows of zero gradient add exact zeros, so the 100 rows are all there is
    check_backward(x, d, w, mean[-100:], rstd[-100:], out[-100:], dw, db)
    assert (out[:-100] == 0).all()
    del big, out, dout
    torch.cuda.empty_cache()


def test_forward_far_offset_and_constant_rows(bfo):
    # The variance comes from differences from the mean, so a large common offset costs only the
    # mean's own rounding.
    x, _, w, b = inputs(50, 1600, torch.float32, torch.float32, 11, offset=300.0)
    check_forward(x, w, b, 1e-5, *run_forward(bfo, x, w, b))
    x = torch.full((3, 1000), 2.5, device=DEV)
    w, b = torch.ones(1000, device=DEV), torch.full((1000,), 0.25, device=DEV)
    out, mean, rstd = run_forward(bfo, x, w, b)
    # 2.5 * 1000 is exact, its product with 1/1000 is off by at most a few u, times rstd = 316
    assert ((mean - 2.5).abs() <= 4 * U * 2.5).all()
    assert ((out - 0.25).abs() <= 4 * U * 2.5 * 317 + 2 * U).all()


def test_forward_nonfinite_rows_stay_their_own(bfo):
    x, _, w, b = inputs(8, 300, torch.float32, torch.float32, 12)
    x = x.clone()
    x[2, 17] = float("inf")
    x[5, 299] = float("nan")
    out, mean, rstd = run_forward(bfo, x, w, b)
    assert out[2].isnan().all() and out[5].isnan().all()
    keep = [0, 1, 3, 4, 6, 7]
    check_forward(x[keep], w, b, 1e-5, out[keep], mean[keep], rstd[keep])


def backward_reference(x, d, w, mean, rstd):
    X, D, Wt = x.double(), d.double(), w.double()
    M, R = mean.double()[:, None], rstd.double()[:, None]
    xhat, h = (X - M) * R, D * Wt
    C = X.shape[1]
    c1, c2 = h.sum(1, keepdim=True) / C, (h * xhat).sum(1, keepdim=True) / C
    dx = R * (h - c1 - xhat * c2)
    a1, a2 = h.abs().mean(1, keepdim=True), (h * xhat).abs().mean(1, keepdim=True)
    tol = R * (4 * U * h.abs() + (DEPTH + 4) * U * a1 + xhat.abs() * (DEPTH + 8) * U * a2 + 5 * U * (xhat * c2).abs()
               + 2 * U * c1.abs()) + 4 * U * dx.abs()
    return dx, tol, (D * xhat).sum(0), (D * xhat).abs().sum(0), D.sum(0), D.abs().sum(0)


def param_depth(rows):
    """Additions in a chain of the parameter sums: rows per group of lanes (at least 512 groups once
    there are that many rows), up to 16 groups of a workgroup, 16 partial rows per lane group, 32 groups.
    (Few rows: 16 rows per group of lanes, 8 groups, 4 exchanges -- fewer.)"""
    return rows // 512 + 1 + 16 + 16 + 32 + 4


def check_backward(x, d, w, mean, rstd, dx, dw, db, old=None):
    rx, tol, rw, aw, rb, ab = backward_reference(x, d, w, mean, rstd)
    n = param_depth(x.shape[0])
    if old is not None:
        rx, rw, rb = rx + old[0].double(), rw + old[1].double(), rb + old[2].double()
        tol = tol + U * rx.abs()
        aw, ab = aw + old[1].double().abs(), ab + old[2].double().abs()
    check(dx, rx, tol + rounding(dx.dtype) * (rx.abs() + tol) + 1e-38, "dx")
    tw, tb = (n + 3) * U * aw, n * U * ab
    check(dw, rw, tw + rounding(dw.dtype) * (rw.abs() + tw) + 1e-38, "dweight")
    if db is not None:
        check(db, rb, tb + rounding(db.dtype) * (rb.abs() + tb) + 1e-38, "dbias")


def run_backward(bfo, x, d, w, mean, rstd, bias=True, **kw):
    rows, cols = x.shape
    dx = torch.full((rows, cols), float("nan"), dtype=x.dtype, device=DEV)
    dw = torch.full((cols,), float("nan"), dtype=w.dtype, device=DEV)
    db = dw.clone() if bias else None
    ws = torch.full_like(bfo.new_layernorm_workspace(rows, cols, DEV), 255)    # NaN patterns
    bfo.layernorm_backward(d, x, w, mean, rstd, dx, dw, db, workspace=ws, **kw)
    return dx, dw, db


def stats_of(x, eps=1e-5):
    X = x.double()
    return X.mean(1).float(), (1 / torch.sqrt(X.var(1, unbiased=False) + eps)).float()


@pytest.mark.parametrize("dt,pdt", COMBOS)
def test_backward_sizes(bfo, dt, pdt):
    for k, (rows, cols) in enumerate(SHAPES + [(2048, 64), (2049, 768), (5000, 33), (512, 300), (513, 300), (511, 2049), (700, 9000),
                                             (1024, 801), (2048, 801), (2049, 801), (2047, 2048), (1024, 2049),
                                             (1025, 2049), (512, 4097), (513, 4097)]):
        print(dt, pdt, rows, cols, flush=True)
        x, d, w, _ = inputs(rows, cols, TYPES[dt], TYPES[pdt], 200 + k, pad=k % 3)
        mean, rstd = stats_of(x)
        check_backward(x, d, w, mean, rstd, *run_backward(bfo, x, d, w, mean, rstd))


@pytest.mark.parametrize("dt,pdt", COMBOS)
@pytest.mark.parametrize("rows,cols", [(77, 96), (600, 1600), (5, 5000), (2100, 1600)])
def test_backward_accumulates(bfo, dt, pdt, rows, cols):
    x, d, w, _ = inputs(rows, cols, TYPES[dt], TYPES[pdt], 31)
    mean, rstd = stats_of(x)
    g = torch.Generator(device=DEV).manual_seed(9)
    old = [torch.empty(s, device=DEV).normal_(generator=g).to(t) for s, t in
           (((rows, cols), TYPES[dt]), ((cols,), TYPES[pdt]), ((cols,), TYPES[pdt]))]
    ws = bfo.new_layernorm_workspace(rows, cols, DEV)
    for acc_dx in (False, True):
        for acc_p in (False, True):
            dx, dw, db = (t.clone() for t in old)
            bfo.layernorm_backward(d, x, w, mean, rstd, dx, dw, db, workspace=ws, accumulate_dx=acc_dx,
                                   accumulate_params=acc_p)
            keep = [torch.zeros_like(t) for t in old]
            if acc_dx:
                keep[0] = old[0]
            if acc_p:
                keep[1:] = old[1:]
            check_backward(x, d, w, mean, rstd, dx, dw, db, keep)


def test_backward_without_bias_rows_or_input_grad_scale(bfo):
    x, d, w, _ = inputs(100, 200, torch.bfloat16, torch.bfloat16, 3)
    mean, rstd = stats_of(x)
    dx, dw, _ = run_backward(bfo, x, d, w, mean, rstd, bias=False)
    check_backward(x, d, w, mean, rstd, dx, dw, None)
    e = torch.empty(0, 200, dtype=torch.bfloat16, device=DEV)
    s = torch.empty(0, device=DEV)
    dx, dw, db = run_backward(bfo, e, e, w, s, s)
    assert (dw == 0).all() and (db == 0).all()
    dw.fill_(3)
    db.fill_(4)
    bfo.layernorm_backward(e, e, w, s, s, torch.empty_like(e), dw, db, accumulate_params=True)
    assert (dw == 3).all() and (db == 4).all()


def test_same_bits_from_call_to_call_and_beside_other_rows(bfo):
    x, d, w, b = inputs(3000, 1600, torch.bfloat16, torch.bfloat16, 8)
    mean, rstd = stats_of(x)
    first = run_backward(bfo, x, d, w, mean, rstd)
    for _ in range(3):
        for a, c in zip(first, run_backward(bfo, x, d, w, mean, rstd)):
            assert torch.equal(a, c)
    whole = run_forward(bfo, x, w, b)[0]
    part = run_forward(bfo, x[100:101], w, b)[0]
    assert torch.equal(whole[100:101], part)


def test_gradient_against_differences(bfo):
    """The directional derivative of sum(dout * out) along random directions of
    x, weight and bias, by central differences of the definition in 64 bits."""
    x, d, w, b = inputs(13, 77, torch.float32, torch.float32, 21)
    out, mean, rstd = run_forward(bfo, x, w, b)
    dx, dw, db = run_backward(bfo, x, d, w, mean, rstd)
    D = d.double()

    def value(X, Wt, B):
        m = X.mean(1, keepdim=True)
        return (((X - m) / torch.sqrt(X.var(1, unbiased=False, keepdim=True) + 1e-5) * Wt + B) * D).sum()

    g = torch.Generator(device=DEV).manual_seed(4)
    for which, grad in enumerate((dx, dw, db)):
        at = [x.double(), w.double(), b.double()]
        v = torch.empty(grad.shape, device=DEV, dtype=torch.float64).normal_(generator=g)
        h = 1e-5
        up, down = list(at), list(at)
        up[which] = at[which] + h * v
        down[which] = at[which] - h * v
        slope = (value(*up) - value(*down)) / (2 * h)
        # third derivatives times h^2 are far below the gradient's own rounding, 100 u of its terms
        terms = (grad.double() * v).abs().sum()
        assert abs(float((grad.double() * v).sum() - slope)) <= float(terms) * 200 * U, which


def test_streams_and_two_calls_at_once(bfo):
    xs = [inputs(2500, 768, torch.bfloat16, torch.bfloat16, 40 + i) for i in range(2)]
    stats = [stats_of(x[0]) for x in xs]
    alone = [run_backward(bfo, x, d, w, *s) for (x, d, w, _), s in zip(xs, stats)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    bufs = [[torch.zeros_like(t) for t in a] for a in alone]
    ws = [bfo.new_layernorm_workspace(2500, 768, DEV) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                x, d, w, _ = xs[i]
                bfo.layernorm_backward(d, x, w, *stats[i], *bufs[i], workspace=ws[i])
    torch.cuda.synchronize()
    for a, b in zip(alone, bufs):
        for p, q in zip(a, b):
            assert torch.equal(p, q)


def test_binding_refusals(bfo):
    x, d, w, b = inputs(8, 64, torch.bfloat16, torch.bfloat16, 2)
    out = torch.empty_like(x)
    with pytest.raises(TypeError, match="out must be"):
        bfo.layernorm_forward(x, w, b, out.float())
    with pytest.raises(ValueError, match="weight has 32"):
        bfo.layernorm_forward(x, w[:32], b, out)
    with pytest.raises(TypeError, match="bias must be"):
        bfo.layernorm_forward(x, w, b.float(), out)
    with pytest.raises(ValueError, match="shape"):
        bfo.layernorm_forward(x, w, b, out[:4])
    with pytest.raises(ValueError, match="mean has"):
        bfo.layernorm_forward(x, w, b, out, torch.empty(3, device=DEV))
    with pytest.raises(ValueError, match="weight is on cpu"):
        bfo.layernorm_forward(x, w.cpu(), b.cpu(), out)
    mean, rstd = stats_of(x)
    many, _, _, _ = inputs(3000, 64, torch.bfloat16, torch.bfloat16, 2)
    s = stats_of(many)
    with pytest.raises(ValueError, match="new_layernorm_workspace"):
        bfo.layernorm_backward(many, many.clone(), w, *s, torch.empty_like(many), w.clone(), b.clone())
    with pytest.raises(ValueError, match="new_layernorm_workspace"):
        bfo.layernorm_backward(many, many.clone(), w, *s, torch.empty_like(many), w.clone(), b.clone(),
                               workspace=bfo.new_layernorm_workspace(600, 64, DEV))
    with pytest.raises(bfo.BfoError):
        bfo.layernorm_backward(d, x, w, mean, rstd, d, w.clone(), b.clone(),
                               workspace=bfo.new_layernorm_workspace(8, 64, DEV))


def test_workspace_of_a_larger_call(bfo):
    """The widest layer's workspace serves a narrower one, whose partial sums are more."""
    ws = bfo.new_layernorm_workspace(2100, 4097, DEV)
    x, d, w, _ = inputs(2100, 4096, torch.bfloat16, torch.bfloat16, 71)
    mean, rstd = stats_of(x)
    own = run_backward(bfo, x, d, w, mean, rstd)
    got = [torch.full_like(t, float("nan")) for t in own]
    bfo.layernorm_backward(d, x, w, mean, rstd, *got, workspace=ws)
    for a, b in zip(own, got):
        assert torch.equal(a, b)


@pytest.mark.parametrize("cols", [1, 37, 1600, 16384])
def test_range_of_the_sums(bfo, cols):
    """Rows at the ends of the range in which binary32 holds their sums: differences from the mean just
    below 2^56, values just below 2^113, and differences of 2^-56 with eps 0."""
    x, _, w, b = inputs(6, cols, torch.float32, torch.float32, 81)
    sign = torch.where(torch.arange(cols, device=DEV) % 2 == 0, 1.0, -1.0)
    top = 1 - 2.0 ** -20
    far = x.clone()
    far[0] = sign * 2.0 ** 56 * top                         # the sum of squares reaches 2^112 cols
    far[1] = x[1] * 2.0 ** 50
    far[2] = 2.0 ** 113 * (1 - 2.0 ** -10)                  # a constant row: a difference of at most 4 u 2^113
    if cols > 1:
        check_forward(far[:2], w, b, 1e-5, *(t[:2] for t in run_forward(bfo, far, w, b)))
        near = x * 2.0 ** -60
        near[0] = sign * 2.0 ** -56
        near[:, 0] = 2.0 ** -56
        near[:, 1] = -2.0 ** -56
        check_forward(near, w, b, 0.0, *run_forward(bfo, near, w, b, 0.0))
    mean = run_forward(bfo, far, w, b)[1]
    assert ((mean[2].double() - far[2, 0].double()).abs() <= (DEPTH + 3) * U * 2.0 ** 113)
