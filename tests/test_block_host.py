"""Refusals of the operators between a block's matrix products, on the host: bad
sizes, types, strides, alignments and overlaps come back as status codes before
any HIP call, and the binding names what is wrong with a tensor.  Only the
rotary frequencies, which need no GPU, are called with what they accept."""
import ctypes
import math

import pytest
import torch


@pytest.fixture(scope="module")
def bfo():
    from bf16_numerics_amd import binding
    return binding


BASE = 1 << 30


def ptr(k, off=0):
    """A distinct 16-byte aligned address 1 GiB apart per k (never read)."""
    return ctypes.c_void_p(BASE * (k + 1) + off)


def rms_forward(bfo, **kw):
    a = dict(x=ptr(0), xs=256, r=ptr(1), rs=256, w=ptr(2), t=ptr(3), ts=256, out=ptr(4), os=256, rstd=ptr(5), q=ptr(6),
             qs=256, s=ptr(7), ct=0, of=0, group=128, rows=4, cols=256, eps=1e-5, dt=0, pdt=0)
    a.update(kw)
    return bfo.library().rmsnorm_forward(a["x"], a["xs"], a["r"], a["rs"], a["w"], a["t"], a["ts"], a["out"], a["os"],
                                         a["rstd"], a["q"], a["qs"], a["s"], a["ct"], a["of"], a["group"], a["rows"],
                                         a["cols"], a["eps"], a["dt"], a["pdt"], None)


def test_rmsnorm_forward_refusals(bfo):
    f = lambda **kw: rms_forward(bfo, **kw)  # noqa: E731
    assert f(cols=0) == bfo.EINVAL
    assert f(cols=bfo.RMSNORM_MAX_COLS + 1, xs=1 << 20, rs=1 << 20, ts=1 << 20, os=1 << 20, qs=1 << 20) == bfo.ERANGE
    for k in ("x", "w", "s", "q"):
        assert f(**{k: None}) == bfo.EINVAL, k
    assert f(r=None) == bfo.EINVAL                                      # a total of nothing
    assert f(out=None, q=None, s=None) == bfo.EINVAL                    # nothing wanted
    for eps in (-1e-5, float("nan"), float("inf")):
        assert f(eps=eps) == bfo.EINVAL, eps
    assert f(dt=2) == bfo.EINVAL and f(pdt=7) == bfo.EINVAL and f(ct=2) == bfo.EINVAL and f(of=2) == bfo.EINVAL
    assert f(group=64) == bfo.EINVAL and f(group=256) == bfo.EINVAL
    for k in ("xs", "rs", "ts", "os", "qs"):
        assert f(**{k: 255}) == bfo.EINVAL, k                           # rows would overlap
        assert f(**{k: 1 << 62}) == bfo.ERANGE, k
    assert f(rows=1 << 40) == bfo.ERANGE
    for k in ("x", "r", "t", "out", "w"):
        assert f(**{k: ptr(9, 1)}) == bfo.EMISALIGNED, k
    assert f(x=ptr(0, 2), dt=1) == bfo.EMISALIGNED and f(w=ptr(2, 2), pdt=1) == bfo.EMISALIGNED
    assert f(rstd=ptr(5, 2)) == bfo.EMISALIGNED and f(s=ptr(7, 2)) == bfo.EMISALIGNED
    for other in (0, 1, 2, 3, 5, 6, 7):
        assert f(out=ptr(other)) == bfo.EINVAL, other
    for other in (0, 1, 2, 3, 4, 5, 7):
        assert f(q=ptr(other)) == bfo.EINVAL, other
    for other in (0, 1, 2, 3, 4, 6):
        assert f(rstd=ptr(other)) == bfo.EINVAL, other
    assert f(t=ptr(0), ts=300) == bfo.EINVAL                            # in place with another stride
    assert f(t=ptr(1, 2)) == bfo.EINVAL and f(t=ptr(2)) == bfo.EINVAL


def rms_backward(bfo, **kw):
    a = dict(g=ptr(0), gs=256, x=ptr(1), xs=256, q=None, qs=256, s=None, ct=0, group=128, w=ptr(2), rstd=ptr(3),
             dx=ptr(4), ds=256, dw=ptr(5), out=ptr(6), os=256, rows=3000, cols=256, dt=0, pdt=0, acc=0, ws=ptr(7))
    a.update(kw)
    return bfo.library().rmsnorm_backward(a["g"], a["gs"], a["x"], a["xs"], a["q"], a["qs"], a["s"], a["ct"], a["group"],
                                          a["w"], a["rstd"], a["dx"], a["ds"], a["dw"], a["out"], a["os"], a["rows"],
                                          a["cols"], a["dt"], a["pdt"], a["acc"], a["ws"], None)


def test_rmsnorm_backward_refusals(bfo):
    f = lambda **kw: rms_backward(bfo, **kw)  # noqa: E731
    for k in ("g", "x", "w", "rstd", "dx", "dw", "ws"):
        assert f(**{k: None}) == bfo.EINVAL, k
    coded = dict(x=None, q=ptr(8), s=ptr(9))
    assert f(q=ptr(8), s=ptr(9)) == bfo.EINVAL                          # both
    assert f(**{**coded, "s": None}) == bfo.EINVAL and f(s=ptr(9)) == bfo.EINVAL
    assert f(**coded, group=7) == bfo.EINVAL and f(**coded, ct=5) == bfo.EINVAL and f(**coded, qs=255) == bfo.EINVAL
    assert f(**{**coded, "s": ptr(9, 1)}) == bfo.EMISALIGNED
    assert f(cols=0) == bfo.EINVAL and f(acc=4) == bfo.EINVAL and f(dt=3) == bfo.EINVAL
    assert f(cols=20000, gs=20000, xs=20000, ds=20000, os=20000) == bfo.ERANGE
    assert f(gs=10) == bfo.EINVAL and f(ds=10) == bfo.EINVAL and f(os=10) == bfo.EINVAL
    assert f(ws=ptr(7, 8)) == bfo.EMISALIGNED and f(dw=ptr(5, 1)) == bfo.EMISALIGNED
    for other in (0, 1, 2, 3, 5, 6, 7):
        assert f(dx=ptr(other)) == bfo.EINVAL, other
    for other in (0, 1, 2, 3, 4, 5, 7):
        assert f(out=ptr(other)) == bfo.EINVAL, other
    for other in (0, 1, 2, 3, 4, 6, 7):
        assert f(dw=ptr(other)) == bfo.EINVAL, other
    assert f(**coded, dx=ptr(8)) == bfo.EINVAL and f(**coded, dw=ptr(9)) == bfo.EINVAL
    out = ctypes.c_uint64()
    lib = bfo.library()
    assert lib.bfo_rmsnorm_workspace_bytes(4, 64, None) == bfo.EINVAL
    assert lib.bfo_rmsnorm_workspace_bytes(4, 0, ctypes.byref(out)) == bfo.EINVAL
    assert lib.bfo_rmsnorm_workspace_bytes(4, 16385, ctypes.byref(out)) == bfo.ERANGE
    assert lib.bfo_rmsnorm_workspace_bytes(1 << 40, 64, ctypes.byref(out)) == bfo.ERANGE
    assert lib.bfo_rmsnorm_workspace_bytes(0, 64, ctypes.byref(out)) == bfo.OK and out.value == 0
    for rows in (1, 5, 512, 513, 1000, 1 << 20):
        assert lib.bfo_rmsnorm_workspace_bytes(rows, 16384, ctypes.byref(out)) == bfo.OK
        assert out.value <= 4 * 16384 * min(rows, 4096)


def test_workspace_of_the_largest_call_serves_every_smaller_one(bfo):
    rows = sorted({1, 2, 3, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 255, 256, 257, 511, 512, 513, 1023, 1024, 1025,
                   2047, 2048, 2049, 4096, 8191, 8192, 16384, 1 << 20, 1 << 31})
    cols = sorted({1, 128, 129, 512, 513, 801, 1024, 1025, 1600, 2048, 2049, 4095, 4096, 4097, 5000, 8192, 8193, 9000,
                   16384})
    f = bfo.rmsnorm_workspace_bytes
    for i, r in enumerate(rows):
        for j, c in enumerate(cols):
            assert i == 0 or f(rows[i - 1], c) <= f(r, c), (r, c)
            assert j == 0 or f(r, cols[j - 1]) <= f(r, c), (r, c)


def act_forward(bfo, **kw):
    a = dict(g=ptr(0), gs=256, u=ptr(1), us=256, out=ptr(2), os=256, gq=ptr(3), gqs=256, gsc=ptr(4), uq=ptr(5), uqs=256,
             usc=ptr(6), ct=0, rows=4, cols=256, kind=0, dt=0)
    a.update(kw)
    return bfo.library().activation_forward(a["g"], a["gs"], a["u"], a["us"], a["out"], a["os"], a["gq"], a["gqs"],
                                            a["gsc"], a["uq"], a["uqs"], a["usc"], a["ct"], a["rows"], a["cols"],
                                            a["kind"], a["dt"], None)


def test_activation_forward_refusals(bfo):
    f = lambda **kw: act_forward(bfo, **kw)  # noqa: E731
    for k in ("g", "out", "gq", "gsc", "uq", "usc"):
        assert f(**{k: None}) == bfo.EINVAL, k
    assert f(u=None) == bfo.EINVAL                                       # codes of what is not there
    assert f(uq=None, usc=None) == bfo.EINVAL and f(gq=None, gsc=None) == bfo.EINVAL
    assert f(kind=2) == bfo.EINVAL and f(kind=-1) == bfo.EINVAL and f(dt=2) == bfo.EINVAL and f(ct=2) == bfo.EINVAL
    assert f(cols=0) == bfo.EINVAL and f(cols=(1 << 28) + 1) == bfo.ERANGE
    assert f(rows=1 << 31) == bfo.ERANGE and f(rows=1 << 63) == bfo.ERANGE
    for k in ("gs", "us", "os", "gqs", "uqs"):
        assert f(**{k: 255}) == bfo.EINVAL, k
    for k in ("g", "u", "out"):
        assert f(**{k: ptr(9, 1)}) == bfo.EMISALIGNED, k
    assert f(gsc=ptr(9, 2)) == bfo.EMISALIGNED
    assert f(out=ptr(0, 2)) == bfo.EINVAL and f(out=ptr(0), os=300) == bfo.EINVAL
    for other in (3, 4, 5, 6):
        assert f(out=ptr(other)) == bfo.EINVAL, other
    for other in (0, 1, 2, 4, 5, 6):
        assert f(gq=ptr(other)) == bfo.EINVAL, other
    lib = bfo.library()
    pack = lambda x, q, s, rows=4, qs=64, ct=0: lib.activation_pack(x, 64, q, qs, s, ct, rows, 64, 0, None)  # noqa: E731
    assert pack(None, ptr(1), ptr(2)) == bfo.EINVAL and pack(ptr(0), None, ptr(2)) == bfo.EINVAL
    assert pack(ptr(0), None, None) == bfo.EINVAL and pack(ptr(0), ptr(1), None) == bfo.EINVAL
    assert pack(ptr(0), ptr(0), ptr(2)) == bfo.EINVAL and pack(ptr(0), ptr(1), ptr(1)) == bfo.EINVAL
    assert pack(ptr(0), ptr(1), ptr(2), qs=63) == bfo.EINVAL and pack(ptr(0), ptr(1), ptr(2), ct=9) == bfo.EINVAL


def act_backward(bfo, **kw):
    a = dict(d=ptr(0), ds=256, g=ptr(1), gs=256, u=ptr(2), us=256, gq=None, gqs=256, gsc=None, uq=None, uqs=256, usc=None,
             ct=0, dg=ptr(3), dgs=256, du=ptr(4), dus=256, out=ptr(5), os=256, rows=4, cols=256, kind=0, dt=0)
    a.update(kw)
    return bfo.library().activation_backward(a["d"], a["ds"], a["g"], a["gs"], a["u"], a["us"], a["gq"], a["gqs"],
                                             a["gsc"], a["uq"], a["uqs"], a["usc"], a["ct"], a["dg"], a["dgs"],
                                             a["du"], a["dus"], a["out"], a["os"], a["rows"], a["cols"], a["kind"],
                                             a["dt"], None)


def test_activation_backward_refusals(bfo):
    f = lambda **kw: act_backward(bfo, **kw)  # noqa: E731
    for k in ("d", "g", "u", "dg", "du"):
        assert f(**{k: None}) == bfo.EINVAL, k
    coded = dict(g=None, u=None, gq=ptr(6), gsc=ptr(7), uq=ptr(8), usc=ptr(9))
    for k in ("gq", "gsc", "uq", "usc"):
        assert f(**{**coded, k: None}) == bfo.EINVAL, k
    assert f(**{**coded, "g": ptr(1)}) == bfo.EINVAL and f(**{**coded, "u": ptr(2)}) == bfo.EINVAL
    assert f(**coded, du=None) == bfo.EINVAL and f(**coded, ct=4) == bfo.EINVAL
    assert f(**coded, dg=ptr(6)) == bfo.EINVAL and f(**coded, out=ptr(9)) == bfo.EINVAL
    assert f(kind=3) == bfo.EINVAL and f(dt=5) == bfo.EINVAL and f(cols=0) == bfo.EINVAL
    assert f(dg=ptr(4)) == bfo.EINVAL and f(out=ptr(3)) == bfo.EINVAL and f(out=ptr(4, 8)) == bfo.EINVAL
    for k in ("ds", "gs", "us", "dgs", "dus", "os"):
        assert f(**{k: 200}) == bfo.EINVAL, k
    assert f(dg=ptr(0, 2)) == bfo.EINVAL and f(dg=ptr(1), dgs=257) == bfo.EINVAL
    lib = bfo.library()
    unpack = lambda q, s, out, group=128, rows=4, ct=0, os=64: \
        lib.activation_unpack(q, 64, s, ct, group, out, os, rows, 64, 0, None)  # noqa: E731
    assert unpack(None, ptr(1), ptr(2)) == bfo.EINVAL and unpack(ptr(0), None, ptr(2)) == bfo.EINVAL
    assert unpack(ptr(0), ptr(1), None) == bfo.EINVAL and unpack(ptr(0), ptr(1), ptr(2), group=1) == bfo.EINVAL
    assert unpack(ptr(0), ptr(1), ptr(0)) == bfo.EINVAL and unpack(ptr(0), ptr(1), ptr(1)) == bfo.EINVAL
    assert unpack(ptr(0), ptr(1), ptr(2), ct=3) == bfo.EINVAL and unpack(ptr(0), ptr(1), ptr(2), os=60) == bfo.EINVAL


def rotary(bfo, **kw):
    a = dict(x=ptr(0), xt=1024, xh=64, out=ptr(1), ot=1024, oh=64, tokens=10, heads=16, dim=64, rotated=32, layout=0,
             f=ptr(2), p=ptr(3), period=0, amplitude=1.0, backward=0, dt=0)
    a.update(kw)
    return bfo.library().rotary_apply(a["x"], a["xt"], a["xh"], a["out"], a["ot"], a["oh"], a["tokens"], a["heads"],
                                      a["dim"], a["rotated"], a["layout"], a["f"], a["p"], a["period"],
                                      a["amplitude"], a["backward"], a["dt"], None)


def test_rotary_refusals(bfo):
    f = lambda **kw: rotary(bfo, **kw)  # noqa: E731
    for k in ("x", "out", "f"):
        assert f(**{k: None}) == bfo.EINVAL, k
    for rotated in (0, 31, 66):
        assert f(rotated=rotated) == bfo.EINVAL, rotated
    assert f(layout=2) == bfo.EINVAL and f(dt=2) == bfo.EINVAL
    assert f(amplitude=float("nan")) == bfo.EINVAL and f(amplitude=float("inf")) == bfo.EINVAL
    assert f(dim=1025, xh=1025, oh=1025, xt=1 << 20, ot=1 << 20) == bfo.ERANGE
    assert f(heads=65536, xt=1 << 24, ot=1 << 24) == bfo.ERANGE and f(tokens=(1 << 31) + 1) == bfo.ERANGE
    assert f(xt=1 << 62) == bfo.ERANGE and f(oh=1 << 62) == bfo.ERANGE
    for k, v in (("xt", 1023), ("xh", 63), ("ot", 1000), ("oh", 0)):
        assert f(**{k: v}) == bfo.EINVAL, k                              # heads reach into one another
    assert f(xt=64, xh=639) == bfo.EINVAL                                # the same with heads outside
    assert f(x=ptr(0, 1)) == bfo.EMISALIGNED and f(out=ptr(1, 2), dt=1) == bfo.EMISALIGNED
    assert f(f=ptr(2, 4)) == bfo.EMISALIGNED and f(p=ptr(3, 2)) == bfo.EMISALIGNED
    assert f(out=ptr(0, 2)) == bfo.EINVAL and f(out=ptr(0), ot=2048) == bfo.EINVAL
    assert f(out=ptr(0), ot=64, oh=640) == bfo.EINVAL                    # in place in the other order
    assert f(out=ptr(2)) == bfo.EINVAL and f(out=ptr(3)) == bfo.EINVAL


def test_rotary_frequencies(bfo):
    f = bfo.rotary_frequencies
    pair = torch.arange(32, dtype=torch.float64)
    plain = 10000.0 ** (-2 * pair / 64)
    assert torch.allclose(f(64), plain, rtol=1e-14, atol=0)
    assert torch.allclose(f(64, scaling=bfo.ROTARY_LINEAR, factor=4.0), plain / 4, rtol=1e-14, atol=0)
    b = f(64, scaling=bfo.ROTARY_BASE, factor=8.0)
    assert b[0] == 1 and math.isclose(b[-1], plain[-1] / 8, rel_tol=1e-12) and (b[1:-1] > plain[1:-1] / 8).all()
    turns = 2048 * plain / (2 * math.pi)
    for kind in (bfo.ROTARY_BY_TURNS, bfo.ROTARY_BY_PAIR):
        g = f(64, scaling=kind, factor=8.0, length=2048, low=1.0, high=32.0)
        assert torch.allclose(g[turns >= 32], plain[turns >= 32], rtol=1e-14, atol=0)
        assert torch.allclose(g[turns <= 1], plain[turns <= 1] / 8, rtol=1e-14, atol=0)
        between = (turns > 1) & (turns < 32)
        assert between.sum() > 5
        if kind == bfo.ROTARY_BY_TURNS:
            keep = (turns - 1) / 31
        else:                                   # turns fall geometrically with the pair
            keep = torch.log(turns) / math.log(32)
        want = plain * keep + plain / 8 * (1 - keep)
        assert torch.allclose(g[between], want[between], rtol=1e-12, atol=0)
    assert f(2).tolist() == [1.0] and len(f(1024)) == 512
    bad = [dict(rotated=0), dict(rotated=7), dict(rotated=64, base=1.0), dict(rotated=64, base=float("nan")),
           dict(rotated=64, scaling=5), dict(rotated=64, scaling=-1), dict(rotated=64, scaling=1, factor=0.5),
           dict(rotated=64, scaling=1, factor=float("inf")), dict(rotated=2, scaling=2, factor=2.0),
           dict(rotated=64, scaling=3, factor=2.0, length=0, low=1, high=2),
           dict(rotated=64, scaling=3, factor=2.0, length=100, low=2, high=2),
           dict(rotated=64, scaling=4, factor=2.0, length=100, low=0, high=2)]
    for kw in bad:
        with pytest.raises(bfo.BfoError) as e:
            f(**kw)
        assert e.value.status == bfo.EINVAL, kw
    for rotated in (1026, 1 << 33, -4):
        with pytest.raises(bfo.BfoError) as e:
            f(rotated)
        assert e.value.status in (bfo.ERANGE, bfo.EINVAL)


def test_binding_names_what_is_wrong(bfo):
    x = torch.zeros(4, 8, dtype=torch.bfloat16)
    w = torch.zeros(8, dtype=torch.bfloat16)
    h = torch.zeros(4, 2, 8)
    freq = torch.zeros(4, dtype=torch.float64)
    for call in (lambda: bfo.rmsnorm_forward(x, w, x), lambda: bfo.rmsnorm_backward(x, x, w, w, x, w),
                 lambda: bfo.activation_forward(x, None, x), lambda: bfo.activation_backward(x, x, None, x, None),
                 lambda: bfo.activation_pack(x, None, None), lambda: bfo.activation_unpack(x, None, x),
                 lambda: bfo.rotary_apply(h, freq, h)):
        with pytest.raises(ValueError, match="expected a GPU"):
            call()
    with pytest.raises(TypeError, match="x must be torch.bfloat16 or torch.float32"):
        bfo.rmsnorm_forward(x.half(), w, x)
    with pytest.raises(ValueError, match="2-D"):
        bfo.activation_forward(x[None], None, x)
    with pytest.raises(ValueError, match="3-D"):
        bfo.rotary_apply(x, freq, x)
    with pytest.raises(ValueError, match="unit column stride"):
        bfo.rotary_apply(h.transpose(1, 2), freq, h)
    for call in (lambda: bfo.rmsnorm_forward(None, w, x), lambda: bfo.activation_backward(None, None, None, x, None),
                 lambda: bfo.rotary_apply(None, freq, h), lambda: bfo.activation_unpack(x, x, None)):
        with pytest.raises(TypeError, match="must be a torch.Tensor"):
            call()
    with pytest.raises(TypeError, match="dtype must be torch.int8 or torch.float8_e4m3fn"):
        bfo.new_codes(4, 8, "cpu", torch.uint8)
    codes, scales = bfo.new_codes(4, 300, "cpu")
    assert codes.shape == (4, 300) and scales.shape == (4, 3) and bfo.new_codes(4, 300, "cpu", per_row=True)[1].shape == (4, 1)
    dev = -1                      # of the CPU
    assert bfo._codes(codes, scales, "codes", dev, 4, 300)[3:] == (bfo.I8, bfo.GROUP)
    assert bfo._codes(codes, scales[:, :1].contiguous(), "codes", dev, 4, 300, whole_row=True)[4] == 0
    for bad, err, match in (((codes, None), ValueError, "scales of codes"), ((None, scales), TypeError, "codes must be"),
                            ((codes, scales.double()), TypeError, "scales must be torch.float32"),
                            ((codes, scales[:, :2].contiguous()), ValueError, "scales of codes"),
                            ((codes, scales[:, :1].contiguous()), ValueError, "scales of codes"),
                            ((codes.float(), scales), TypeError, "codes must be"),
                            ((codes[:3], scales), ValueError, "shape"), ((codes, scales.flatten()), ValueError, "scales")):
        with pytest.raises(err, match=match):
            bfo._codes(*bad, "codes", dev, 4, 300)
    with pytest.raises(bfo.BfoError):
        bfo.rmsnorm_workspace_bytes(4, 1 << 20)
    for cols in ((1 << 32) + 64, 1 << 32, -(1 << 32) + 64):
        with pytest.raises(bfo.BfoError) as e:
            bfo.rmsnorm_workspace_bytes(4, cols)
        assert e.value.status == bfo.ERANGE


def test_activation_gradients_do_not_go_over_the_codes(bfo):
    """Outputs may be dout, gate and up, the matrices of their own type; over codes, a byte a column, they would be
    written where other columns have still to be read: refused also where pointer and bytes from row to row agree."""
    coded = dict(g=None, u=None, gq=ptr(6), gsc=ptr(7), uq=ptr(8), usc=ptr(9))
    for dt, size in ((0, 2), (1, 4)):
        for codes in ("gq", "uq"):
            for out, stride in (("dg", "dgs"), ("du", "dus"), ("out", "os")):
                over = {**coded, "dt": dt, out: coded[codes]}
                what = (dt, codes, out)
                assert act_backward(bfo, **over, rows=1) == bfo.EINVAL, what
                assert act_backward(bfo, **over, rows=1, cols=1) == bfo.EINVAL, what
                over[codes + "s"], over[stride] = 256 * size, 256
                for rows in (1, 2, 4):
                    assert act_backward(bfo, **over, rows=rows) == bfo.EINVAL, (what, rows)
            # without a gate too
            one = dict(g=None, u=None, du=None, gq=ptr(6), gqs=256 * size, gsc=ptr(7), dt=dt, dg=ptr(6))
            assert act_backward(bfo, **one) == bfo.EINVAL and act_backward(bfo, **{**one, "dg": ptr(3)}, out=ptr(6)) == bfo.EINVAL


def test_rotary_frequencies_of_far_parameters(bfo):
    """Whatever the documentation allows has finite frequencies: turns and factors whose quotients or powers pass
    binary64, and bounds whose logarithms are the same number."""
    f, pair = bfo.rotary_frequencies, torch.arange(32, dtype=torch.float64)
    plain = 10000.0 ** (-2 * pair / 64)
    # from low = 1e-310 on the pairs' bounds are real numbers as always
    bound = lambda turns: 64 * (math.log(2048.0) - math.log(turns) - math.log(2 * math.pi)) / (2 * math.log(10000.0))  # noqa: E731
    got = f(64, scaling=bfo.ROTARY_BY_PAIR, factor=8.0, length=2048.0, low=1e-310, high=32.0)
    keep = ((bound(1e-310) - pair) / (bound(1e-310) - bound(32.0))).clamp(0, 1)
    assert torch.allclose(got, plain * keep + plain / 8 * (1 - keep), rtol=1e-12, atol=0)
    # a factor whose power is past binary64: the first pair as it is, the last divided by it
    got = f(4, scaling=bfo.ROTARY_BASE, factor=1e300)
    assert got[0] == 1 and math.isclose(got[1], 0.01 / 1e300, rel_tol=1e-12)
    # bounds next to one another, at the turns of a pair itself: that pair is between them, the others are not
    for low, at in ((32.0, -1), (2048.0 / (2 * math.pi), 0), (2048.0 / (2 * math.pi) * 10000.0 ** -0.5, 16)):
        got = f(64, scaling=bfo.ROTARY_BY_PAIR, factor=8.0, length=2048.0, low=low, high=math.nextafter(low, math.inf))
        above, below = (got - plain).abs() <= 1e-12 * plain, (got - plain / 8).abs() <= 1e-12 * plain
        assert (above | below | (pair == at)).all()
        assert (got <= plain * (1 + 1e-12)).all() and (got >= plain / 8 * (1 - 1e-12)).all()
