"""Definitions in 64 bits, with counted tolerances, of the operators between a
transformer block's matrix products.  Tolerances count roundings of half a step
u = 2^-24 of binary32 along the operation's order, plus one rounding to the
output's type (eps / 2 relative)."""
import math

import torch

DEV = "cuda:0"
U = 2.0 ** -24
GROUP = 128
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
CODES = {"i8": torch.int8, "e4m3": torch.float8_e4m3fn}
TOP = {torch.int8: 127.0, torch.float8_e4m3fn: 448.0}
SMALLEST = 2.0 ** -126


def rounding(t):
    """Half a step of the type, relative; 0 for binary32 results counted in u."""
    return torch.finfo(t).eps / 2 if t != torch.float32 else 0.0


def check(got, ref, tol, what):
    got = got.double()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    bad = ~((got - ref).abs() <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst " \
                          f"{float(((got - ref).abs() / tol).nan_to_num(posinf=1e9, nan=1e9).max())} of the tolerance"


def check_rounded(got, ref, tol, what):
    """A result that is off by `tol` before it is rounded to its type."""
    check(got, ref, tol + rounding(got.dtype) * (ref.abs() + tol) + 1e-38, what)


def group_of(cols, scales):
    """For each column, which of a row's scales is its own."""
    per_row = scales.shape[1] == 1 and cols > GROUP
    return torch.arange(cols, device=scales.device) // (cols if per_row else GROUP)


def values(codes, scales):
    """What codes stand for, in 64 bits."""
    return codes.double() * scales.double()[:, group_of(codes.shape[1], scales)]


def half_step(a, dtype):
    """Half the distance of the codes around a number of size a, in units of the scale."""
    if dtype == torch.int8:
        return torch.full_like(a, 0.5)
    e = torch.frexp(a * (1 + 1e-6)).exponent.clamp(min=-5)       # a < 2^e: codes 2^(e-4) apart, from 2^-6 down 2^-9
    return torch.ldexp(torch.ones_like(a), e - 5)


def check_codes(codes, scales, ref, off, what):
    """Codes and scales of values that are `ref` up to a relative `off`.  The scale is the largest one's by
    two roundings (1 / top and the product); a code is its value's, by the reciprocal and the product two
    roundings off, to the nearest."""
    rows, cols = ref.shape
    own = group_of(cols, scales)
    amax = torch.zeros(rows, scales.shape[1], dtype=torch.float64, device=ref.device)
    amax.scatter_reduce_(1, own.expand(rows, cols), ref.abs(), "amax")
    want = (amax / TOP[codes.dtype]).clamp(min=SMALLEST)
    check(scales, want, (off + 2 * U) * want, what + " scales")
    a = ref / scales.double()[:, own]
    check(codes, a, half_step(a.abs(), codes.dtype) + a.abs() * (off + 2.01 * U), what + " codes")
    assert codes.double().abs().max() <= TOP[codes.dtype]


def normal(g, *shape):
    return torch.empty(shape, device=DEV).normal_(generator=g)


def matrix(g, rows, cols, dt, pad=0, spread=True, size=1.0):
    """Columns of different size, as columns of a buffer `pad` wider (NaN there)."""
    x = torch.full((rows, cols + pad), float("nan"), dtype=dt, device=DEV)
    v = normal(g, rows, cols) * size
    x[:, :cols] = (v * torch.exp(0.5 * normal(g, cols)) if spread else v).to(dt)
    return x[:, :cols]


def empty(rows, cols, dt, pad=0):
    x = torch.full((rows, cols + pad), 72.0, device=DEV).to(dt)
    return x[:, :cols]


def untouched(x):
    """The columns of the buffer behind x are as `empty` made them."""
    rows, cols = x.shape
    if rows == 0 or x.stride(0) == cols:
        return True
    wide = x.as_strided((rows, x.stride(0)), (x.stride(0), 1))
    return bool((wide[:, cols:].float() == 72).all())


# ---------------------------------------------------------------------------
# RMS norm
# ---------------------------------------------------------------------------

# A sum over a row: at most 16 terms a lane, 6 steps of the wavefront and 15 more wavefronts.
DEPTH = 40


def check_rms_forward(x, residual, w, eps, total=None, out=None, rstd=None, codes=None, scales=None, of_out=False):
    t = x
    if residual is not None:
        t = (x.float() + residual.float()).to(x.dtype)
        if total is not None:
            assert torch.equal(total, t)
    X, W = t.double(), w.double()
    r = 1 / torch.sqrt(X.square().mean(1, keepdim=True) + eps)
    off = 0.5 * (DEPTH + 3) * U + 3 * U
    if rstd is not None:
        check(rstd, r[:, 0], off * r[:, 0], "rstd")
    ref = X * r * W
    if out is not None:
        check_rounded(out, ref, (off + 2 * U) * ref.abs(), "out")
    if codes is not None:
        check_codes(codes, scales, ref if of_out else X * r, off + (2 if of_out else 1) * U, "norm")


def rms_param_depth(rows):
    """Additions in a chain of dweight: rows per group of lanes (at least 256 groups once there are that
    many rows), up to 16 groups of a workgroup, 16 partial rows per lane group, 32 groups."""
    return rows // 256 + 1 + 16 + 16 + 32


def check_rms_backward(dout, xhat, w, rstd, dx, dw, out=None, old=None, off=1):
    """xhat: the normalised values in 64 bits, which the kernel has up to `off` roundings."""
    D, W, R = dout.double(), w.double(), rstd.double()[:, None]
    h = D * W
    mean, size = (h * xhat).mean(1, keepdim=True), (h * xhat).abs().mean(1, keepdim=True)
    ref = R * (h - xhat * mean)
    tol = R * (3 * U * h.abs() + xhat.abs() * (DEPTH + off + 4) * U * size + (off + 3) * U * (xhat * mean).abs())
    tol = tol + 2 * U * ref.abs()
    n = rms_param_depth(dout.shape[0]) + off
    rw, aw = (D * xhat).sum(0), (D * xhat).abs().sum(0)
    if old is not None:
        ref, rw, aw = ref + old[0].double(), rw + old[1].double(), aw + old[1].double().abs()
        tol = tol + U * ref.abs()
    check_rounded(dx, ref, tol, "dx")
    check_rounded(dw, rw, n * U * aw, "dweight")
    if out is not None:
        check_rounded(out, xhat * W, (off + 1) * U * (xhat * W).abs(), "out again")


# ---------------------------------------------------------------------------
# Activation
# ---------------------------------------------------------------------------

K = math.sqrt(2 / math.pi)


def activation(kind, g):
    """(act, its derivative, sigma, z, dz/dg) in 64 bits; kind 0: SiLU, 1: GELU."""
    z, dz = (g, torch.ones_like(g)) if kind == 0 else (2 * K * (g + 0.044715 * g ** 3), 2 * K * (1 + 3 * 0.044715 * g * g))
    s, t = torch.sigmoid(z), torch.sigmoid(-z)
    return g * s, s + g * s * t * dz, s, t, z, dz


def activation_tolerances(kind, g):
    """(of act, of its derivative).  z is 6 roundings off in GELU, its product with log2(e) 3, the
    exponential two, their sum one, its reciprocal two; results below 2^-125 may be flushed to 0."""
    act, _, s, t, z, dz = activation(kind, g)
    rel = t * (9 * z.abs() + 2) * U + 4 * U
    tiny = 2.0 ** -124 * (1 + g.abs())
    slope = s * rel + (act * t * dz).abs() * (rel + 10 * U) + (act * dz).abs() * (s * rel + U)
    return act.abs() * (rel + U) + tiny, slope + 2 * U * (s + (act * t * dz).abs()) + tiny * (1 + dz)


def check_activation_forward(kind, gate, up, out):
    g = gate.double()
    act = activation(kind, g)[0]
    tol = activation_tolerances(kind, g)[0]
    if up is None:
        check_rounded(out, act, tol, "out")
    else:
        u = up.double()
        check_rounded(out, act * u, tol * u.abs() + U * (act * u).abs(), "out")


def check_activation_backward(kind, dout, g, u, dgate, dup, again=None, off=0):
    """g, u: the inputs in 64 bits, which the kernel has up to `off` roundings."""
    D = dout.double()
    act, slope, s, t, z, dz = activation(kind, g)
    ta, ts = activation_tolerances(kind, g)
    # a relative error of g moves act by |g act'| and the derivative by |g act''|, for which 4 (1 + |z|) dz serves
    ta = ta + off * U * (g * slope).abs()
    ts = ts + off * U * g.abs() * 4 * (1 + z.abs()) * dz * s * t * (1 + dz)
    into = D if u is None else D * u
    check_rounded(dgate, into * slope, into.abs() * (ts + (2 + off) * U * slope.abs()), "dgate")
    if u is not None:
        check_rounded(dup, D * act, D.abs() * (ta + U * act.abs()), "dup")
    if again is not None:
        ref = act if u is None else act * u
        size = 1.0 if u is None else u.abs()
        check_rounded(again, ref, ta * size + (1 + off) * U * ref.abs(), "out again")


# ---------------------------------------------------------------------------
# Rotary positions
# ---------------------------------------------------------------------------

def pair_columns(rotated, half):
    i = torch.arange(rotated // 2, device=DEV)
    return (i, i + rotated // 2) if half else (2 * i, 2 * i + 1)


def check_rotary(out, x, positions, frequencies, half, amplitude=1.0, backward=False):
    """Angles are formed in 64 bits on both sides (two roundings of 2^-53 more); the turn's rest as a
    float is half a step off, sine and cosine two steps, and the amplitude's product, two products and
    their sum one rounding each."""
    rotated = 2 * frequencies.numel()
    a, b = pair_columns(rotated, half)
    angle = positions.double()[:, None] * frequencies
    c, s = torch.cos(angle)[:, None] * amplitude, torch.sin(angle)[:, None] * amplitude * (-1 if backward else 1)
    X = x.double()
    u, v = X[:, :, a], X[:, :, b]
    ref = X.clone()
    ref[:, :, a] = u * c - v * s
    ref[:, :, b] = u * s + v * c
    off = ((math.pi + 4 + 3) * U + 2.0 ** -51 * angle.abs()[:, None]) * abs(amplitude)
    tol = torch.zeros_like(X)
    tol[:, :, a] = tol[:, :, b] = (u.abs() + v.abs()) * off
    check(out, ref, tol + rounding(out.dtype) * (ref.abs() + tol) + 1e-38, "rotary")
    if rotated < x.shape[2]:
        assert torch.equal(out[:, :, rotated:], x[:, :, rotated:])
