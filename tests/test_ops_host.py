"""Refusals of the training-loop operators, on the host: bad sizes, types,
strides, alignments and overlaps come back as status codes before any HIP
call, and the binding names what is wrong with a tensor.  No entry point is
called with arguments it would accept."""
import ctypes

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


def ln_forward(bfo, **kw):
    a = dict(x=ptr(0), xs=64, w=ptr(1), b=ptr(2), out=ptr(3), os=64, mean=ptr(4), rstd=ptr(5), rows=4, cols=64,
             eps=1e-5, dt=0, pdt=0)
    a.update(kw)
    return bfo.library().layernorm_forward(a["x"], a["xs"], a["w"], a["b"], a["out"], a["os"], a["mean"], a["rstd"],
                                           a["rows"], a["cols"], a["eps"], a["dt"], a["pdt"], None)


def test_layernorm_forward_refusals(bfo):
    f = lambda **kw: ln_forward(bfo, **kw)  # noqa: E731
    assert f(cols=0) == bfo.EINVAL
    assert f(cols=bfo.LAYERNORM_MAX_COLS + 1, xs=1 << 20, os=1 << 20) == bfo.ERANGE
    for k in ("x", "w", "out"):
        assert f(**{k: None}) == bfo.EINVAL, k
    for eps in (-1e-5, float("nan"), float("inf")):
        assert f(eps=eps) == bfo.EINVAL, eps
    assert f(dt=2) == bfo.EINVAL and f(dt=-1) == bfo.EINVAL and f(pdt=7) == bfo.EINVAL
    assert f(xs=63) == bfo.EINVAL and f(os=63) == bfo.EINVAL           # rows would overlap
    assert f(xs=1 << 62) == bfo.ERANGE                                 # past the address space
    assert f(rows=1 << 40) == bfo.ERANGE
    assert f(x=ptr(0, 1)) == bfo.EMISALIGNED and f(out=ptr(3, 1)) == bfo.EMISALIGNED
    assert f(x=ptr(0, 2), dt=1) == bfo.EMISALIGNED
    assert f(w=ptr(1, 2), pdt=1) == bfo.EMISALIGNED and f(b=ptr(2, 1)) == bfo.EMISALIGNED
    assert f(mean=ptr(4, 2)) == bfo.EMISALIGNED and f(rstd=ptr(5, 1)) == bfo.EMISALIGNED
    # overlaps: out with x, out with weight, mean with rstd, mean inside x
    assert f(out=ptr(0)) == bfo.EINVAL
    assert f(out=ptr(0, 2 * 64 * 4 - 2)) == bfo.EINVAL
    assert f(out=ptr(1)) == bfo.EINVAL
    assert f(rstd=ptr(4, 12)) == bfo.EINVAL
    assert f(mean=ptr(0, 64)) == bfo.EINVAL
    # interleaved columns of one buffer that do touch
    assert f(x=ptr(0), xs=100, out=ptr(0, 2 * 63), os=100) == bfo.EINVAL


def ln_backward(bfo, **kw):
    a = dict(g=ptr(0), gs=64, x=ptr(1), xs=64, w=ptr(2), mean=ptr(3), rstd=ptr(4), dx=ptr(5), ds=64, dw=ptr(6),
             db=ptr(7), rows=3000, cols=64, dt=0, pdt=0, acc=0, ws=ptr(8))
    a.update(kw)
    return bfo.library().layernorm_backward(a["g"], a["gs"], a["x"], a["xs"], a["w"], a["mean"], a["rstd"], a["dx"],
                                            a["ds"], a["dw"], a["db"], a["rows"], a["cols"], a["dt"], a["pdt"],
                                            a["acc"], a["ws"], None)


def test_layernorm_backward_refusals(bfo):
    f = lambda **kw: ln_backward(bfo, **kw)  # noqa: E731
    for k in ("g", "x", "w", "mean", "rstd", "dx", "dw", "ws"):
        assert f(**{k: None}) == bfo.EINVAL, k
    assert f(dw=None, rows=0) == bfo.EINVAL
    assert f(cols=0) == bfo.EINVAL and f(acc=4) == bfo.EINVAL and f(dt=3) == bfo.EINVAL
    assert f(cols=20000, gs=20000, xs=20000, ds=20000) == bfo.ERANGE
    assert f(gs=10) == bfo.EINVAL and f(ds=10) == bfo.EINVAL
    assert f(ws=ptr(8, 8)) == bfo.EMISALIGNED and f(dw=ptr(6, 1)) == bfo.EMISALIGNED
    assert f(db=ptr(7, 2), pdt=1) == bfo.EMISALIGNED
    for other in (0, 1, 2, 3, 4, 6, 7, 8):
        assert f(dx=ptr(other)) == bfo.EINVAL, other
    for other in (0, 1, 2, 3, 4, 5, 7, 8):
        assert f(dw=ptr(other)) == bfo.EINVAL, other
    out = ctypes.c_uint64()
    lib = bfo.library()
    assert lib.bfo_layernorm_workspace_bytes(4, 64, None) == bfo.EINVAL
    assert lib.bfo_layernorm_workspace_bytes(4, 0, ctypes.byref(out)) == bfo.EINVAL
    assert lib.bfo_layernorm_workspace_bytes(4, 16385, ctypes.byref(out)) == bfo.ERANGE
    assert lib.bfo_layernorm_workspace_bytes(0, 64, ctypes.byref(out)) == bfo.OK and out.value == 0
    for rows in (1, 5, 512, 513, 1000, 1 << 20):
        assert lib.bfo_layernorm_workspace_bytes(rows, 16384, ctypes.byref(out)) == bfo.OK
        assert out.value <= 8 * 16384 * min(rows, 4096) and (out.value > 0) == (rows > 512)


def lp_forward(bfo, **kw):
    a = dict(x=ptr(0), s=100, rows=4, V=100, dt=0, scale=1.0, t=ptr(1), lp=ptr(2), st=ptr(3), en=ptr(4), top=5,
             ti=ptr(5), tl=ptr(6), ws=ptr(7))
    a.update(kw)
    return bfo.library().token_logprobs_forward(a["x"], a["s"], a["rows"], a["V"], a["dt"], a["scale"], a["t"],
                                                a["lp"], a["st"], a["en"], a["top"], a["ti"], a["tl"], a["ws"], None)


def test_token_logprobs_forward_refusals(bfo):
    f = lambda **kw: lp_forward(bfo, **kw)  # noqa: E731
    assert f(x=None) == bfo.EINVAL and f(V=0) == bfo.EINVAL and f(dt=5) == bfo.EINVAL
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        assert f(scale=scale) == bfo.EINVAL, scale
    assert f(V=bfo.VOCAB_MAX + 1, s=1 << 40) == bfo.ERANGE
    assert f(s=99) == bfo.EINVAL
    assert f(t=None) == bfo.EINVAL and f(lp=None) == bfo.EINVAL          # both or neither
    assert f(ti=None) == bfo.EINVAL and f(tl=None) == bfo.EINVAL
    assert f(top=0) == bfo.EINVAL                                         # arrays given, none asked for
    assert f(top=bfo.TOP_MAX + 1, V=1000, s=1000) == bfo.ERANGE
    assert f(top=101) == bfo.EINVAL                                       # more than there are
    for k in ("t", "lp", "st", "en", "ti", "tl"):
        assert f(**{k: ptr(9, 2)}) == bfo.EMISALIGNED, k
    assert f(x=ptr(0, 1)) == bfo.EMISALIGNED and f(ws=ptr(7, 4)) == bfo.EMISALIGNED
    for k in ("lp", "st", "en", "ti", "tl"):
        assert f(**{k: ptr(0)}) == bfo.EINVAL, k                          # on the logits
        assert f(**{k: ptr(1, 8)}) == bfo.EINVAL, k                       # on the targets
    assert f(lp=ptr(3, 16)) == bfo.EINVAL
    out = ctypes.c_uint64()
    lib = bfo.library()
    assert lib.bfo_logits_workspace_bytes(4, 100, 5, None) == bfo.EINVAL
    assert lib.bfo_logits_workspace_bytes(4, 0, 0, ctypes.byref(out)) == bfo.EINVAL
    assert lib.bfo_logits_workspace_bytes(4, 100, 101, ctypes.byref(out)) == bfo.EINVAL
    assert lib.bfo_logits_workspace_bytes(4, 1000, 129, ctypes.byref(out)) == bfo.ERANGE
    assert lib.bfo_logits_workspace_bytes(4, (1 << 28) + 1, 0, ctypes.byref(out)) == bfo.ERANGE
    assert lib.bfo_logits_workspace_bytes(0, 100, 5, ctypes.byref(out)) == bfo.OK and out.value == 0
    # few rows of many scores need a workspace: none, or one on the outputs, is refused
    assert lib.bfo_logits_workspace_bytes(1, 131072, 128, ctypes.byref(out)) == bfo.OK and out.value > 0
    assert f(rows=1, V=131072, s=131072, ws=None) == bfo.EINVAL
    assert f(rows=1, V=131072, s=131072, ws=ptr(3)) == bfo.EINVAL
    assert kd(bfo, rows=1, V=131072, s=131072, ws=None) == bfo.EINVAL
    for rows in range(0, 300):
        for vocab in (1, 65535, 65536, 65537, 131071, 1 << 20, 1 << 28):
            assert lib.bfo_logits_workspace_bytes(rows, vocab, min(vocab, 128), ctypes.byref(out)) == bfo.OK
            assert out.value <= 256 * (16 + 8 * 128)


def lp_backward(bfo, **kw):
    a = dict(x=ptr(0), s=112, rows=4, V=100, W=112, dt=0, scale=1.0, t=ptr(1), st=ptr(2), en=ptr(3), dlp=ptr(4),
             de=ptr(5), dx=ptr(6), ds=112)
    a.update(kw)
    return bfo.library().token_logprobs_backward(a["x"], a["s"], a["rows"], a["V"], a["W"], a["dt"], a["scale"],
                                                 a["t"], a["st"], a["en"], a["dlp"], a["de"], a["dx"], a["ds"], None)


def test_token_logprobs_backward_refusals(bfo):
    f = lambda **kw: lp_backward(bfo, **kw)  # noqa: E731
    for k in ("x", "t", "st", "en", "dlp", "de", "dx"):
        assert f(**{k: None}) == bfo.EINVAL, k
    assert f(t=None, dlp=None, en=None, de=None) == bfo.EINVAL             # nothing to differentiate
    assert f(W=99) == bfo.EINVAL and f(W=113) == bfo.EINVAL                # narrower than vocab; wider than its rows
    assert f(scale=0.0) == bfo.EINVAL and f(V=0) == bfo.EINVAL and f(dt=9) == bfo.EINVAL
    assert f(dx=ptr(6, 1)) == bfo.EMISALIGNED and f(st=ptr(2, 2)) == bfo.EMISALIGNED
    assert f(dx=ptr(0, 2)) == bfo.EINVAL                                   # shifted onto the logits
    assert f(dx=ptr(0), ds=120) == bfo.EINVAL                              # in place with another stride
    for other in (1, 2, 3, 4, 5):
        assert f(dx=ptr(other)) == bfo.EINVAL, other


def kd(bfo, backward=False, **kw):
    a = dict(x=ptr(0), s=112, rows=4, V=100, W=112, dt=0, scale=1.0, ti=ptr(1), tl=ptr(2), n=8, t=ptr(3), kl=ptr(4),
             lp=ptr(5), st=ptr(6), ws=None, dx=ptr(7), ds=112)
    a.update(kw)
    lib = bfo.library()
    if backward:
        return lib.distill_backward(a["x"], a["s"], a["rows"], a["V"], a["W"], a["dt"], a["scale"], a["ti"], a["tl"],
                                    a["n"], a["t"], a["st"], a["kl"], a["lp"], a["dx"], a["ds"], None)
    return lib.distill_forward(a["x"], a["s"], a["rows"], a["V"], a["dt"], a["scale"], a["ti"], a["tl"], a["n"],
                               a["t"], a["kl"], a["lp"], a["st"], a["ws"], None)


@pytest.mark.parametrize("backward", [False, True])
def test_distill_refusals(bfo, backward):
    f = lambda **kw: kd(bfo, backward, **kw)  # noqa: E731
    for k in ("x", "ti", "tl", "kl", "t", "lp") + (("st", "dx") if backward else ()):
        assert f(**{k: None}) == bfo.EINVAL, k
    assert f(n=0) == bfo.EINVAL and f(n=bfo.TOP_MAX + 1) == bfo.ERANGE
    assert f(scale=-2.0) == bfo.EINVAL and f(V=0) == bfo.EINVAL and f(dt=2) == bfo.EINVAL and f(s=99) == bfo.EINVAL
    for k in ("ti", "tl", "kl", "t", "lp", "st"):
        assert f(**{k: ptr(9, 2)}) == bfo.EMISALIGNED, k
    if backward:
        assert f(dx=ptr(0, 4)) == bfo.EINVAL
        for other in (1, 2, 3, 4, 5, 6):
            assert f(dx=ptr(other)) == bfo.EINVAL, other
    else:
        for k in ("kl", "lp", "st"):
            for other in (0, 1, 2, 3):
                assert f(**{k: ptr(other)}) == bfo.EINVAL, (k, other)


def test_binding_names_what_is_wrong(bfo):
    x = torch.zeros(4, 8, dtype=torch.bfloat16)
    w = torch.zeros(8, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="expected a GPU"):
        bfo.layernorm_forward(x, w, w, x)
    with pytest.raises(TypeError, match="x must be torch.bfloat16 or torch.float32"):
        bfo.layernorm_forward(x.half(), w, w, x)
    with pytest.raises(ValueError, match="2-D"):
        bfo.layernorm_forward(x[None], w, w, x)
    with pytest.raises(ValueError, match="unit column stride"):
        bfo.layernorm_forward(torch.zeros(8, 4, dtype=torch.bfloat16).t(), w, w, x)
    with pytest.raises(ValueError, match="expected a GPU"):
        bfo.token_logprobs_forward(x)
    for call in (lambda: bfo.layernorm_forward(None, w, w, x), lambda: bfo.token_logprobs_forward(None),
                 lambda: bfo.layernorm_backward(x.tolist(), None, w, w, w, x, w),
                 lambda: bfo.distill_backward(None, None, None, None, None, x)):
        with pytest.raises(TypeError, match="must be a torch.Tensor"):
            call()
    with pytest.raises(ValueError, match="expected a GPU"):
        bfo.distill_forward(x, None, None, None)
    with pytest.raises(bfo.BfoError):
        bfo.layernorm_workspace_bytes(4, 1 << 20)
    with pytest.raises(bfo.BfoError):
        bfo.logits_workspace_bytes(4, 100, 300)


def test_workspace_of_the_largest_call_serves_every_smaller_one(bfo):
    """Sizes never fall as rows, columns, vocabulary or top grow, so a buffer of the largest call's size
    holds those of a ragged last batch or a narrower layer."""
    rows = sorted({1, 2, 3, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 511, 512, 513, 1023, 1024, 1025,
                   2047, 2048, 2049, 2100, 4096, 8191, 8192, 16384, 1 << 20, 1 << 31})
    cols = sorted({1, 128, 129, 512, 513, 801, 1024, 1025, 1600, 2048, 2049, 4095, 4096, 4097, 5000, 8192, 8193,
                   9000, 16384})
    vocabs = sorted({1, 128, 50257, 65535, 65536, 65537, 81920, 98304, 100000, 128256, 131071, 131072, 131073, 1 << 20,
                     1 << 28})

    def rising(axes, f):
        """f at every point is at least f one step back along each axis."""
        import itertools
        for at in itertools.product(*(range(len(a)) for a in axes)):
            here = f(*(a[i] for a, i in zip(axes, at)))
            for k in range(len(axes)):
                if at[k]:
                    back = at[:k] + (at[k] - 1,) + at[k + 1:]
                    less = tuple(a[i] for a, i in zip(axes, back))
                    assert f(*less) <= here, (less, tuple(a[i] for a, i in zip(axes, at)))

    rising((rows, cols), bfo.layernorm_workspace_bytes)
    rising((rows, vocabs, (0, 1, 20, 128)), lambda r, v, t: bfo.logits_workspace_bytes(r, v, min(t, v)))


def test_binding_passes_no_size_modulo_two_to_the_32(bfo):
    """Column counts are 32-bit arguments of the C ABI: larger ones are out of range, not their low words."""
    def status(f, *sizes):
        with pytest.raises(bfo.BfoError) as e:
            f(*sizes)
        return e.value.status

    for cols in ((1 << 32) + 64, 1 << 32, -(1 << 32) + 64):
        assert status(bfo.layernorm_workspace_bytes, 4, cols) == bfo.ERANGE
        assert status(bfo.logits_workspace_bytes, 4, cols, 0) == bfo.ERANGE
        assert status(bfo.logits_workspace_bytes, 4, 1000, cols) in (bfo.ERANGE, bfo.EINVAL)
    for rows in ((1 << 64) + 4, -(1 << 64) + 4):
        assert status(bfo.layernorm_workspace_bytes, rows, 64) == bfo.ERANGE
        assert status(bfo.logits_workspace_bytes, rows, 1000, 0) == bfo.ERANGE
