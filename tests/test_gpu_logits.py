"""Token log probabilities and distillation on the GPU against their
definitions in 64 bits.

Tolerances count roundings of half a step u = 2^-24 of binary32.  A row's sum
of exponentials is a chain of at most n = V / 64 + 64 additions and
rescalings (each of at most 4 u), the exponential of a distance d costs
(4 |d| + 4) u relative; with E the mean under p,
  log sum:   rel = (n + 4 E|d| + 8) u  absolute
  log prob:  rel + (3 |d| + 4) u
  entropy:   rel + E(|d| (4 |d| + n + 8)) u + E|d| rel + (2 + H) 2 u.
Gradients are compared with the formula on the very stats they are given and
on z as they take it, rounded to binary32.  With d = z - M, |log p| = |d| + log S:
the roundings of d, of log2(e) (half a u) and of log S * log2(e) and the final
fma's leave log p within 4 |log p| u, the exponential adds 2 u, so that a
probability is off by (6 |log p| + 12) u relative and, where log p itself is a
factor, by 4 |log p| u more.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def bfo():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from bf16_numerics_amd import binding
    torch.cuda.set_device(0)
    return binding


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def scores(rows, vocab, dt, seed, pad=0, spread=2.0):
    """Scores with a raised token per row; padding columns hold NaN, never to be read."""
    g = gen(seed)
    z = torch.full((rows, vocab + pad), NAN, device=DEV)
    z[:, :vocab] = spread * torch.empty(rows, vocab, device=DEV).normal_(generator=g)
    t = torch.randint(0, vocab, (rows,), generator=g, device=DEV)
    z[torch.arange(rows, device=DEV), t] += 8 * torch.rand(rows, generator=g, device=DEV)
    t[torch.rand(rows, generator=g, device=DEV) < 0.2] = -1
    return z.to(TYPES[dt]), t.to(torch.int32)


def single(scale):
    """The scale as the entry points take it: a binary32 value."""
    return float(torch.tensor(scale, dtype=torch.float32))


def reference(logits, V, scale, targets):
    scale = single(scale)
    z = logits[:, :V].double() * scale
    m = z.max(1, keepdim=True).values
    d = z - m
    logs = torch.logsumexp(d, 1, keepdim=True)
    logp = d - logs
    p = logp.exp()
    pd = torch.where(p > 0, p * d.abs(), 0.0).sum(1)
    pdd = torch.where(p > 0, p * d * d, 0.0).sum(1)
    ent = -torch.where(p > 0, p * logp, 0.0).sum(1)
    n = V / 64 + 64
    rel = (n + 4 * pd + 8) * U
    t = targets.long()
    at = logp.gather(1, t.clamp(min=0, max=V - 1)[:, None])[:, 0]
    dt = d.gather(1, t.clamp(min=0, max=V - 1)[:, None])[:, 0].abs()
    live = t >= 0
    return {"m": m[:, 0], "logs": logs[:, 0], "rel": rel, "ent": ent, "logp": logp, "d": d,
            "ent_tol": rel + (4 * pdd + (n + 8) * pd) * U + pd * rel + (2 + ent) * 2 * U,
            "at": torch.where(live, at, 0.0), "at_tol": torch.where(live, rel + (3 * dt + 4) * U, 0.0)}


def near(got, ref, tol, what):
    got = got.double()
    bad = ~((got - ref).abs() <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off; worst by {float((got - ref).abs().max())}"


def top_reference(logits, V, K):
    # equal scores by the lower index: stable, largest first; -0 and 0 are equal
    return torch.sort(logits[:, :V].double() + 0.0, dim=1, descending=True, stable=True).indices[:, :K]


def top_reference_nan_first(logits, V, K):
    z = logits[:, :V].double() + 0.0
    z[z == INF] = 1e300
    return torch.sort(torch.where(z.isnan(), INF, z), dim=1, descending=True, stable=True).indices[:, :K]


def run_forward(bfo, logits, targets, V, scale=1.0, top=0):
    R = logits.shape[0]
    f = lambda *s: torch.full(s, NAN, device=DEV)  # noqa: E731
    out = {"logprob": f(R), "stats": f(R, 2), "entropy": f(R)}
    if top:
        out["top_index"] = torch.full((R, top), -7, dtype=torch.int32, device=DEV)
        out["top_logprob"] = f(R, top)
    ws = torch.full_like(bfo.new_logits_workspace(R, V, top, DEV), 255)
    bfo.token_logprobs_forward(logits, targets, out["logprob"], out["stats"], entropy=out["entropy"],
                               top_index=out.get("top_index"), top_logprob=out.get("top_logprob"), vocab=V,
                               scale=scale, workspace=ws)
    return out


def check_forward(out, logits, targets, V, scale, top):
    ref = reference(logits, V, scale, targets)
    near(out["stats"][:, 0], ref["m"], U * ref["m"].abs(), "max")
    near(out["stats"][:, 1], ref["logs"], ref["rel"], "log sum")
    near(out["logprob"], ref["at"], ref["at_tol"], "logprob")
    near(out["entropy"], ref["ent"], ref["ent_tol"], "entropy")
    if top:
        index = top_reference(logits, V, top)
        assert torch.equal(out["top_index"].long(), index)
        near(out["top_logprob"], ref["logp"].gather(1, index),
             ref["rel"][:, None] + (3 * ref["d"].gather(1, index).abs() + 4) * U, "top logprob")


SIZES = [(1, 1), (3, 2), (5, 7), (9, 64), (2, 127), (4, 128), (33, 513), (7, 1000), (3, 4095), (3, 4096), (2, 4097),
         (17, 8193), (5, 32000), (3, 50257), (2, 65537), (1, 131072), (1, 200003)]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_forward_sizes(bfo, dt):
    for k, (rows, V) in enumerate(SIZES):
        for top in sorted({0, 1, min(V, 5), min(V, 20), min(V, 128)}):
            scale = (1.0, 0.5, 1.7)[(k + top) % 3]
            print(dt, rows, V, top, scale, flush=True)
            logits, targets = scores(rows, V, dt, 300 + k, pad=(0, 5, 64)[k % 3])
            check_forward(run_forward(bfo, logits, targets, V, scale, top), logits, targets, V, scale, top)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_forward_many_rows(bfo, dt):
    logits, targets = scores(3001, 1031, dt, 17, pad=3)
    check_forward(run_forward(bfo, logits, targets, 1031, 1.0, 20), logits, targets, 1031, 1.0, 20)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("V", [300, 5000, 40001, 140000])
def test_top_of_rows_that_do_not_thin_out(bfo, dt, V):
    """Equal scores, few distinct scores, sorted rows, all the best in one
    lane's columns, scores at the type's lowest value."""
    t = TYPES[dt]
    E = 16 // t.itemsize
    rows = [torch.zeros(V), torch.full((V,), -3.0), torch.arange(V) % 3 * 1.0, torch.arange(V) * 0.25,
            -torch.arange(V) * 0.25, torch.where(torch.arange(V) // E % 512 == 5, 4.0, 0.0),
            torch.where(torch.arange(V) // E % 512 == 5, torch.arange(V) % 97 * 0.5, -1.0),
            torch.full((V,), float(torch.finfo(t).min)), torch.full((V,), -INF), torch.full((V,), -INF),
            torch.where(torch.arange(V) % 2 == 0, -0.0, 0.0)]
    rows[9][V // 2] = 1.0
    logits = torch.stack(rows).to(t).to(DEV)
    targets = torch.full((len(rows),), V // 2, dtype=torch.int32, device=DEV)
    for top in (1, 20, 128):
        out = run_forward(bfo, logits, targets, V, 1.0, top)
        index = top_reference(logits, V, top)
        assert torch.equal(out["top_index"].long(), index)
        keep = [i for i in range(len(rows)) if i != 8]
        sub = {k: v[keep] for k, v in out.items()}
        ref = reference(logits[keep], V, 1.0, targets[keep])
        near(sub["stats"][:, 1], ref["logs"], ref["rel"], "log sum")
        got, want = sub["top_logprob"].double(), ref["logp"].gather(1, index[keep])
        tol = ref["rel"][:, None] + (3 * ref["d"].gather(1, index[keep]).abs() + 4) * U
        assert (((got - want).abs() <= tol) | (got == want)).all()
        # a row of -inf only
        assert out["stats"][8].tolist() == [-INF, 0.0] and out["entropy"][8] == 0
        assert out["logprob"][8] == -INF and (out["top_logprob"][8] == -INF).all()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_masked_scores_nan_inf_and_odd_targets(bfo, dt):
    V, t = 5003, TYPES[dt]
    logits, _ = scores(8, V, dt, 5)
    logits = logits.clone()
    logits[0, ::2] = -INF                                   # half the vocabulary masked out
    logits[1, 1:] = float(torch.finfo(t).min)               # all but one at the lowest value
    logits[2, 77] = NAN
    logits[3, 78] = INF
    logits[4, :] = -INF
    targets = torch.tensor([3, 0, 5, 78, 9, -1, V, 2 ** 31 - 1], dtype=torch.int32, device=DEV)
    out = run_forward(bfo, logits, targets, V, 1.0, 10)
    keep = [0, 1, 5]
    check_forward({k: v[keep] for k, v in out.items()}, logits[keep], targets[keep], V, 1.0, 10)
    for r in (2, 3):
        for k in ("stats", "logprob", "entropy", "top_logprob"):
            assert out[k][r].isnan().all(), (r, k)
    assert out["top_index"][2, 0] == 77 and out["top_index"][3, 0] == 78
    assert out["logprob"][5] == 0 and out["logprob"][6].isnan() and out["logprob"][7].isnan()
    assert not out["stats"][6:].isnan().any()
    # gradients: the empty row and rows without factors are 0, bad rows NaN, masked scores 0
    R = 8
    g = torch.full((R,), -0.25, device=DEV)
    h = torch.full((R,), 0.125, device=DEV)
    h[5] = 0
    d = torch.full_like(logits, NAN)
    bfo.token_logprobs_backward(logits, targets, out["stats"], g, d, entropy=out["entropy"], dentropy=h)
    assert (d[0, ::2] == 0).all() and not d[0].isnan().any()
    assert not d[1].isnan().any()
    assert d[2].isnan().all() and d[3].isnan().all() and d[6].isnan().all() and d[7].isnan().all()
    assert (d[4] == 0).all() and (d[5] == 0).all()
    # a masked row's scores do not matter, whatever they hold
    h.zero_()
    targets.fill_(-1)
    bfo.token_logprobs_backward(logits, targets, out["stats"], g, d, entropy=out["entropy"], dentropy=h)
    assert (d == 0).all()


@pytest.mark.parametrize("V,rows", [(300, 3), (9001, 3), (70001, 3), (9001, 600)])
def test_scores_far_from_zero_and_far_apart(bfo, V, rows):
    """Rows around large offsets, and rows some of whose scores, or all that a
    lane sees, lie far below the others."""
    g = gen(V)
    base = 3 * torch.empty(rows, V, device=DEV).normal_(generator=g)
    targets = torch.randint(0, V, (rows,), generator=g, device=DEV).to(torch.int32)
    for scale in (1.0, 0.25, 0.7):
        for offset in (0.0, 700.0, -700.0, 712.0, 3000.0, -3000.0, 1e6, -1e6, 1e30):
            logits = base + offset
            check_forward(run_forward(bfo, logits, targets, V, scale, 20), logits, targets, V, scale, 20)
        for low in (-100.0, -1000.0, -1500.0, -5000.0, -65504.0, -1e30, -3e38):
            logits = base.clone()
            logits[:, V // 3:] = low
            logits[0, :] = low
            logits[1, 1::2] = low
            check_forward(run_forward(bfo, logits, targets, V, scale, 20), logits, targets, V, scale, 20)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("V", [100, 70000])
def test_scores_whose_scaled_value_overflows(bfo, dt, V):
    t = TYPES[dt]
    low, high = float(torch.finfo(t).min), float(torch.finfo(t).max)
    logits = torch.zeros(4, V, dtype=t, device=DEV)
    logits[0] = low                                          # z = -inf throughout: an empty row
    logits[1, 1:] = low                                      # z = 0 and -inf
    logits[2, 5] = high                                      # z = +inf somewhere: NaN
    targets = torch.tensor([1, 0, 5, 7], dtype=torch.int32, device=DEV)
    out = run_forward(bfo, logits, targets, V, 2.0, 3)
    assert out["stats"][0].tolist() == [-INF, 0.0] and out["logprob"][0] == -INF and out["entropy"][0] == 0
    assert out["stats"][1].tolist() == [0.0, 0.0] and out["logprob"][1] == 0 and out["entropy"][1] == 0
    assert out["stats"][2].isnan().all() and out["logprob"][2].isnan()
    assert torch.equal(out["top_index"][:3].cpu(), torch.tensor([[0, 1, 2], [0, 1, 2], [5, 0, 1]], dtype=torch.int32))
    d = torch.full_like(logits, NAN)
    bfo.token_logprobs_backward(logits, targets, out["stats"], torch.ones(4, device=DEV), d, scale=2.0)
    assert (d[0] == 0).all() and (d[1] == 0).all() and d[2].isnan().all()
    # a row's gradients cancel; each is off by up to half a bf16 step, of 2 * scale = 4 altogether
    near(d[3].double().sum(), torch.zeros((), device=DEV).double(), 4 * 2.0 ** -8, "sum of a row")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_few_rows_of_a_long_vocabulary(bfo, dt):
    """Rows that are split over workgroups: NaN, +inf and -inf in one stretch of
    the vocabulary only, equal scores across the stretches, targets and teacher
    tokens anywhere, odd starts; the same bits every time."""
    V, pad = 131071, 1
    logits, targets = scores(7, V, dt, 91, pad=pad)
    logits = logits.clone()
    logits[1, 100_000:] = -INF
    logits[2, ::16384] = 40.0                                # ties in every stretch
    logits[3, 5] = NAN
    logits[4, V - 1] = INF
    logits[5, :V] = -INF
    logits[6, :] = 0.0
    targets = torch.tensor([V - 1, 3, 16384, 5, 6, 7, -1], dtype=torch.int32, device=DEV)
    assert bfo.logits_workspace_bytes(7, V, 128) > 0
    for top in (1, 20, 128):
        out = run_forward(bfo, logits, targets, V, 1.0, top)
        assert torch.equal(out["top_index"].long(), top_reference_nan_first(logits, V, top))
        keep = [0, 2, 6]
        check_forward({k: v[keep] for k, v in out.items()}, logits[keep], targets[keep], V, 1.0, top)
        check_forward({k: v[1:2] for k, v in out.items()}, logits[1:2], targets[1:2], V, 1.0, top)
        for r in (3, 4):
            assert all(out[k][r].isnan().all() for k in ("stats", "logprob", "entropy", "top_logprob"))
        assert out["stats"][5].tolist() == [-INF, 0.0] and out["entropy"][5] == 0 and out["logprob"][5] == -INF
        again = run_forward(bfo, logits, targets, V, 1.0, top)
        for k in out:
            assert torch.equal(torch.nan_to_num(out[k], 9.0), torch.nan_to_num(again[k], 9.0)), k
    with pytest.raises(ValueError, match="new_logits_workspace"):
        bfo.token_logprobs_forward(logits, stats=torch.empty(7, 2, device=DEV), vocab=V)
    index, value = teacher(7, V, 128, 92)
    index[0, :3] = torch.tensor([0, V - 1, 16384], dtype=torch.int32)
    kl, _, lp = run_distill(bfo, logits, index, value, V, 1.0, targets)
    keep = [0, 2, 6]
    ref, _, _, _, want, tol = distill_reference(logits[keep], V, 1.0, index[keep], value[keep], targets[keep])
    near(kl[keep], want, tol, "kl")
    near(lp[keep], ref["at"], ref["at_tol"], "logprob")


def test_forward_outputs_are_optional(bfo):
    logits, targets = scores(6, 3001, "bf16", 8)
    full = run_forward(bfo, logits, targets, 3001, 1.0, 7)
    lp = torch.empty(6, device=DEV)
    bfo.token_logprobs_forward(logits, targets, lp)
    assert torch.equal(lp, full["logprob"])
    st = torch.empty(6, 2, device=DEV)
    bfo.token_logprobs_forward(logits, stats=st)
    assert torch.equal(st, full["stats"])
    ti, tl = torch.empty(6, 7, dtype=torch.int32, device=DEV), torch.empty(6, 7, device=DEV)
    bfo.token_logprobs_forward(logits, top_index=ti, top_logprob=tl,
                               workspace=bfo.new_logits_workspace(6, 3001, 7, DEV))
    assert torch.equal(ti, full["top_index"]) and torch.equal(tl, full["top_logprob"])
    e = logits[:0]
    bfo.token_logprobs_forward(e, targets[:0], lp[:0], st[:0])
    bfo.token_logprobs_backward(e, targets[:0], st[:0], lp[:0], e.clone())


# -------------------------------------------------------------------------
# Gradients
# -------------------------------------------------------------------------

def gradient_reference(logits, V, scale, stats, base, slope, ent, sparse):
    """scale * (p * (base + slope * (log p + ent)) + sparse) and its tolerance,
    from the given stats."""
    z = (logits[:, :V].float() * torch.tensor(scale, device=DEV)).double()
    scale = single(scale)
    s = stats.double()
    logp = z - s[:, :1] - s[:, 1:]
    p = logp.exp()
    lp = torch.where(p > 0, logp, 0.0)
    b, k, h = base.double()[:, None], slope.double()[:, None], ent.double()[:, None]
    dense = p * (b + k * (lp + h))
    ref = scale * (dense + sparse)
    size = p * (b.abs() + k.abs() * (lp.abs() + h.abs()))
    tol = scale * (size * (6 * lp.abs() + 16) * U + 4 * U * (size + sparse.abs())) + 2 * U * ref.abs()
    return ref, tol


def check_gradient(d, V, ref, tol, what=""):
    half = torch.finfo(d.dtype).eps / 2 if d.dtype != torch.float32 else 0.0
    near(d[:, :V], ref, tol + half * (ref.abs() + tol) + 1e-37, what)
    assert (d[:, V:] == 0).all()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("with_entropy,with_targets", [(True, True), (False, True), (True, False)])
def test_logprob_gradient(bfo, dt, with_entropy, with_targets):
    for k, (rows, V) in enumerate(SIZES + [(1500, 257)]):
        pad = (0, 7, 64)[k % 3]
        scale = (1.0, 0.5, 1.7)[k % 3]
        print(dt, rows, V, pad, flush=True)
        logits, targets = scores(rows, V, dt, 400 + k, pad=pad)
        out = run_forward(bfo, logits, targets, V, scale)
        g = gen(k)
        dlp = torch.empty(rows, device=DEV).normal_(generator=g)
        den = torch.empty(rows, device=DEV).normal_(generator=g) if with_entropy else torch.zeros(rows, device=DEV)
        d = torch.full_like(logits, NAN)
        bfo.token_logprobs_backward(logits, targets if with_targets else None, out["stats"],
                                    dlp if with_targets else None, d, entropy=out["entropy"] if with_entropy else None,
                                    dentropy=den if with_entropy else None, vocab=V, scale=scale)
        hard = torch.where(targets >= 0, dlp, 0.0) if with_targets else torch.zeros(rows, device=DEV)
        sparse = torch.zeros(rows, V, dtype=torch.float64, device=DEV)
        sparse.scatter_(1, targets.clamp(min=0).long()[:, None], hard.double()[:, None])
        check_gradient(d, V, *gradient_reference(logits, V, scale, out["stats"], -hard, -den, out["entropy"], sparse))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [1.0, 0.7, 0.3])
def test_gradient_of_scores_far_from_zero(bfo, dt, scale):
    """Rows around large offsets and rows masked by the type's lowest value, in
    part and throughout, whose scaled scores are rounded to binary32 before
    anything is subtracted: p = exp(z - M - log S) of those is off by
    (6 |log p| + 16) u whatever z is."""
    V, t = 1003, TYPES[dt]
    low = float(torch.finfo(t).min)
    rows = []
    for offset in (0.0, 700.0, -700.0, 1e4, -1e6, 1e10, -1e30):
        logits, _ = scores(1, V, "f32", 21)
        rows.append((logits + offset).to(t))
    rows += [torch.full((1, V), low, dtype=t, device=DEV), rows[0].clone()]
    rows[-1][:, ::3] = low
    logits = torch.cat(rows)
    R = logits.shape[0]
    targets = torch.arange(R, dtype=torch.int32, device=DEV) * 7 + 1
    out = run_forward(bfo, logits, targets, V, scale)
    z = (logits.float() * torch.tensor(scale, device=DEV)).double()
    stats = out["stats"].double()
    assert torch.equal(stats[:, 0], z.max(1).values)
    assert abs(float(stats[-2, 1]) - math.log(V)) <= (V / 64 + 72) * U
    lp = z - stats[:, :1] - stats[:, 1:]
    p = lp.exp()
    lp = torch.where(p > 0, lp, 0.0)
    one = torch.zeros(R, V, dtype=torch.float64, device=DEV)
    one.scatter_(1, targets.long()[:, None], 1.0)
    a, b = torch.full((R,), -0.75, device=DEV), torch.full((R,), 0.5, device=DEV)
    h = out["entropy"].double()[:, None]
    size = p * (0.75 + 0.5 * (lp.abs() + h.abs()))
    d = torch.full_like(logits, NAN)
    bfo.token_logprobs_backward(logits, targets, out["stats"], a, d, entropy=out["entropy"], dentropy=b, scale=scale)
    tol = single(scale) * size * (6 * lp.abs() + 24) * U + 4 * U * one
    check_gradient(d, V, single(scale) * (-0.75 * (one - p) - 0.5 * p * (lp + h)), tol, "with entropy")
    index, value = teacher(R, V, 9, 22)
    q, _, live, spread = teacher_reference(index, value, scale)
    d = torch.full_like(logits, NAN)
    bfo.distill_backward(logits, index, value, out["stats"], b, d, scale=scale)
    part = torch.zeros_like(one).scatter_add_(1, index.clamp(min=0).long(), q)
    off = torch.zeros_like(one).scatter_add_(1, index.clamp(min=0).long(), q * (4 * spread + 88) * U)
    half = 0.5 * live[:, None]
    check_gradient(d, V, single(scale) * half * (p - part), half * (p * (6 * lp.abs() + 24) * U + off), "distill")


def test_logprob_gradient_in_place_and_strided(bfo):
    logits, targets = scores(65, 5001, "bf16", 3, pad=39)
    out = run_forward(bfo, logits, targets, 5001)
    g = torch.full((65,), -1 / 65, device=DEV)
    apart = torch.empty_like(logits)
    bfo.token_logprobs_backward(logits, targets, out["stats"], g, apart, vocab=5001)
    place = logits.clone()
    bfo.token_logprobs_backward(place, targets, out["stats"], g, place, vocab=5001)
    assert torch.equal(apart, place)
    wide = torch.full((65, 5040 + 33), 5.0, dtype=torch.bfloat16, device=DEV)
    bfo.token_logprobs_backward(logits, targets, out["stats"], g, wide[:, 33:], vocab=5001)
    assert torch.equal(wide[:, 33:], apart) and (wide[:, :33] == 5).all()


def teacher(rows, V, K, seed):
    """K distinct tokens a row, some rows with fewer, some with none."""
    g = gen(seed)
    index = torch.stack([torch.randperm(V, generator=g, device=DEV)[:K] for _ in range(rows)])
    value = 3 * torch.empty(rows, K, device=DEV).normal_(generator=g)
    keep = torch.randint(0, 2 * K + 1, (rows, 1), generator=g, device=DEV)
    index = torch.where(torch.arange(K, device=DEV)[None] < keep, index, -1)
    return index.to(torch.int32), value


def teacher_reference(index, value, scale):
    scale = single(scale)
    v = torch.where(index >= 0, value.double() * scale, -INF)
    live = (v > -INF).any(1, keepdim=True)
    v = torch.where(live, v, 0.0)
    logq = torch.log_softmax(v, 1)
    q = torch.where(live & (index >= 0), logq.exp(), 0.0)
    spread = torch.where(q > 0, v.max(1, keepdim=True).values - v, 0.0)
    return q, logq, live[:, 0], spread


def distill_reference(logits, V, scale, index, value, targets):
    ref = reference(logits, V, scale, targets)
    q, logq, live, spread = teacher_reference(index, value, scale)
    logp = ref["logp"].gather(1, index.clamp(min=0).long())
    dist = ref["d"].gather(1, index.clamp(min=0).long()).abs()
    terms = torch.where(q > 0, q * (logq - logp), 0.0)
    # log q: up to (4 spread + 80) u; log p as above; q itself (4 spread + 80) u relative; 10 additions
    tol = torch.where(q > 0, q * ((4 * spread + 80) * U * (1 + (logq - logp).abs()) + ref["rel"][:, None]
                                  + (3 * dist + 6) * U) + 10 * U * terms.abs(), 0.0)
    return ref, q, live, spread, terms.sum(1), tol.sum(1)


def run_distill(bfo, logits, index, value, V, scale, targets=None):
    R = logits.shape[0]
    f = lambda *s: torch.full(s, NAN, device=DEV)  # noqa: E731
    kl, stats, lp = f(R), f(R, 2), f(R) if targets is not None else None
    bfo.distill_forward(logits, index, value, kl, stats, targets=targets, logprob=lp, vocab=V, scale=scale,
                        workspace=torch.full_like(bfo.new_logits_workspace(R, V, 0, DEV), 255))
    return kl, stats, lp


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("hard", [False, True])
def test_distill_forward_and_gradient(bfo, dt, hard):
    for k, (rows, V) in enumerate(SIZES + [(700, 513)]):
        for K in sorted({1, min(V, 20), min(V, 65), min(V, 128)}):
            scale = (1.0, 0.5, 1.7)[(k + K) % 3]
            print(dt, hard, rows, V, K, flush=True)
            logits, targets = scores(rows, V, dt, 500 + k, pad=(0, 7, 64)[k % 3])
            index, value = teacher(rows, V, K, 600 + k)
            kl, stats, lp = run_distill(bfo, logits, index, value, V, scale, targets if hard else None)
            ref, q, live, spread, want, tol = distill_reference(logits, V, scale, index, value, targets)
            near(kl, want, tol, "kl")
            near(stats[:, 1], ref["logs"], ref["rel"], "log sum")
            if hard:
                near(lp, ref["at"], ref["at_tol"], "logprob")
            g = gen(k + K)
            dkl = torch.empty(rows, device=DEV).normal_(generator=g)
            dlp = torch.empty(rows, device=DEV).normal_(generator=g)
            d = torch.full_like(logits, NAN)
            bfo.distill_backward(logits, index, value, stats, dkl, d, targets=targets if hard else None,
                                 dlogprob=dlp if hard else None, vocab=V, scale=scale)
            h = torch.where(targets >= 0, dlp, 0.0) if hard else torch.zeros(rows, device=DEV)
            sparse = torch.zeros(rows, V, dtype=torch.float64, device=DEV)
            extra = torch.zeros_like(sparse)
            at = index.clamp(min=0).long()
            sparse.scatter_add_(1, at, -dkl.double()[:, None] * q)
            extra.scatter_add_(1, at, dkl.double().abs()[:, None] * q * (4 * spread + 80) * U)
            sparse.scatter_add_(1, targets.clamp(min=0).long()[:, None], h.double()[:, None])
            base = torch.where(live, dkl, 0.0) - h
            zero = torch.zeros(rows, device=DEV)
            r, t = gradient_reference(logits, V, scale, stats, base, zero, zero, sparse)
            # base is one rounded difference of terms that may cancel
            p = (logits[:, :V].double() * single(scale) - stats.double().sum(1, keepdim=True)).exp()
            t = t + scale * (extra + p * (dkl.abs() + h.abs()).double()[:, None] * 2 * U)
            check_gradient(d, V, r, t, "dlogits")


def test_distill_odd_entries(bfo):
    """A token named several times, entries of -inf, rows without entries,
    a student that gives a teacher's token nothing, bad indexes and NaN."""
    V = 3001
    logits, targets = scores(9, V, "f32", 12)
    logits = logits.clone()
    index, value = teacher(9, V, 16, 13)
    index[:] = torch.arange(16, device=DEV, dtype=torch.int32) * 100 + 7
    index[0] = 55                                            # one token, sixteen times
    index[1, ::2] = 1234
    value[2, 3:] = -INF
    index[3] = -1
    value[4] = -INF
    logits[5, 107] = -INF                                    # named by the teacher
    index[6, 4] = V
    value[7, 2] = NAN
    index[8, 9], value[8, 9] = -1, NAN                       # no entry: its value is not looked at
    kl, stats, _ = run_distill(bfo, logits, index, value, V, 1.0)
    keep = [0, 1, 2, 8]
    _, q, _, _, want, tol = distill_reference(logits[keep], V, 1.0, index[keep], value[keep], targets[keep])
    near(kl[keep], want, tol, "kl")
    assert kl[3] == 0 and kl[4] == 0 and kl[5] == INF and kl[6].isnan() and kl[7].isnan()
    d = torch.full_like(logits, NAN)
    dkl = torch.full((9,), 0.5, device=DEV)
    bfo.distill_backward(logits, index, value, stats, dkl, d)
    assert (d[3] == 0).all() and (d[4] == 0).all() and d[6].isnan().all() and d[7].isnan().all()
    assert not d[5].isnan().any()
    p = (logits.double() - stats.double().sum(1, keepdim=True)).exp()
    q5 = torch.softmax(value[5].double(), 0)
    assert abs(float(d[5, 107]) + 0.5 * float(q5[1])) <= 100 * U
    for i, r in enumerate(keep):
        sparse = torch.zeros(V, dtype=torch.float64, device=DEV)
        sparse.index_add_(0, index[r].clamp(min=0).long(), q[i])
        near(d[r], 0.5 * (p[r] - sparse), 0.5 * (p[r] + sparse) * 400 * U + 1e-37, "dlogits")
    # the same bits every time, also where equal indexes add
    again = torch.full_like(logits, NAN)
    for _ in range(5):
        bfo.distill_backward(logits, index, value, stats, dkl, again)
        assert torch.equal(torch.nan_to_num(d, 9.0), torch.nan_to_num(again, 9.0))


def test_factor_of_a_row_without_entries_counts_as_zero(bfo):
    """Whatever it is, and also where the true token's factor is not zero."""
    V = 2003
    logits, _ = scores(3, V, "f32", 14)
    targets = torch.tensor([5, 5, -1], dtype=torch.int32, device=DEV)
    index = torch.arange(6, dtype=torch.int32, device=DEV).repeat(3, 1)
    index[0] = -1
    value = torch.full((3, 6), -INF, device=DEV)
    _, stats, _ = run_distill(bfo, logits, index, value, V, 1.0)
    factor = torch.full((3,), 0.5, device=DEV)
    plain, d = torch.full_like(logits, NAN), torch.full_like(logits, NAN)
    bfo.token_logprobs_backward(logits, targets, stats, factor, plain)
    for dkl in (0.25, INF, NAN):
        bfo.distill_backward(logits, index, value, stats, torch.full((3,), dkl, device=DEV), d, targets=targets,
                             dlogprob=factor)
        assert torch.equal(d, plain), dkl


def test_teacher_side_feeds_the_student_side(bfo):
    """A teacher's top log probabilities serve as its logits."""
    V, K = 4001, 20
    z, t = scores(50, V, "bf16", 21)
    out = run_forward(bfo, z, t, V, 1.0, K)
    student, _ = scores(50, V, "bf16", 22)
    raw = torch.gather(z.float(), 1, out["top_index"].long())
    a, _, _ = run_distill(bfo, student, out["top_index"], out["top_logprob"], V, 1.0)
    b, _, _ = run_distill(bfo, student, out["top_index"], raw, V, 1.0)
    _, _, _, _, want, tol = distill_reference(student, V, 1.0, out["top_index"], raw, t)
    near(a, want, tol + 50 * U * (1 + want.abs()), "kl from log probabilities")
    near(b, want, tol, "kl from scores")
    # the student being the teacher: only the mass outside the top remains, -log of the mass inside
    same, _, _ = run_distill(bfo, z, out["top_index"], raw, V, 1.0)
    inside = torch.softmax(z.double(), 1).gather(1, out["top_index"].long()).sum(1)
    near(same, -inside.log(), 200 * U * (1 + out["entropy"].double()), "kl to itself")


def test_gradients_against_differences(bfo):
    """Directional derivatives of the losses by central differences of their
    definitions in 64 bits."""
    V, R, K, scale = 211, 6, 9, single(0.7)
    logits, targets = scores(R, V, "f32", 31)
    index, value = teacher(R, V, K, 32)
    g = gen(33)
    a, b, c = (torch.empty(R, device=DEV).normal_(generator=g) for _ in range(3))
    out = run_forward(bfo, logits, targets, V, scale)
    d1, d2 = torch.empty_like(logits), torch.empty_like(logits)
    bfo.token_logprobs_backward(logits, targets, out["stats"], a, d1, entropy=out["entropy"], dentropy=b, scale=scale)
    bfo.distill_backward(logits, index, value, out["stats"], c, d2, targets=targets, dlogprob=a, scale=scale)
    q, logq, _, _ = teacher_reference(index, value, scale)

    def losses(z):
        logp = torch.log_softmax(z * scale, 1)
        at = torch.where(targets >= 0, logp.gather(1, targets.clamp(min=0).long()[:, None])[:, 0], 0.0)
        ent = -(logp.exp() * logp).sum(1)
        kl = torch.where(q > 0, q * (logq - logp.gather(1, index.clamp(min=0).long())), 0.0).sum(1)
        return (a * at + b * ent).sum(), (a * at + c * kl).sum()

    z = logits.double()
    # what a gradient's terms are made of before they cancel: its rounding is tens of u of these
    logp = torch.log_softmax(z * scale, 1)
    p, ent = logp.exp(), out["entropy"].double()[:, None]
    size = [p * (a.abs()[:, None] + b.abs()[:, None] * (logp.abs() + ent)), p * (a.abs() + c.abs())[:, None]]
    for s in size:
        s.scatter_add_(1, targets.clamp(min=0).long()[:, None], a.double().abs()[:, None])
    size[1].scatter_add_(1, index.clamp(min=0).long(), c.double().abs()[:, None] * q)
    for trial in range(3):
        v = torch.empty(R, V, dtype=torch.float64, device=DEV).normal_(generator=g)
        h = 1e-5
        up, down = losses(z + h * v), losses(z - h * v)
        for d, x, y, s in ((d1, up[0], down[0], size[0]), (d2, up[1], down[1], size[1])):
            slope = float((x - y) / (2 * h))
            terms = float((scale * s * v.abs()).sum())
            # h^2 times third derivatives, and the loss's rounding over h, stay below 1e-9
            assert abs(float((d.double() * v).sum()) - slope) <= 200 * U * terms + 1e-9


def test_rows_past_32_bit_offsets(bfo):
    """The last rows of a matrix whose element offsets pass 2^32."""
    V, stride = 50257, 50304
    R = (1 << 32) // stride + 40
    buf = torch.zeros(R * stride, dtype=torch.bfloat16, device=DEV)
    logits = buf.view(R, stride)
    few, t = scores(40, V, "bf16", 77)
    logits[-40:, :V] = few
    targets = torch.full((R,), -1, dtype=torch.int32, device=DEV)
    targets[-40:] = t
    out = run_forward(bfo, logits, targets, V, 1.0, 3)
    check_forward({k: v[-40:] for k, v in out.items()}, few, t, V, 1.0, 3)
    g = torch.ones(R, device=DEV)
    bfo.token_logprobs_backward(logits, targets, out["stats"], g, logits, vocab=V)
    apart = torch.empty_like(few)
    bfo.token_logprobs_backward(few, t, out["stats"][-40:].contiguous(), g[-40:].contiguous(), apart)
    assert torch.equal(logits[-40:, :V], apart) and (logits[:-40] == 0).all() and (logits[-40:, V:] == 0).all()
    del buf, logits
    torch.cuda.empty_cache()


def test_same_bits_beside_other_rows_and_on_streams(bfo):
    V = 9001
    logits, targets = scores(600, V, "bf16", 51)
    whole = run_forward(bfo, logits, targets, V, 1.0, 20)
    for r in (0, 299, 599):
        one = run_forward(bfo, logits[r:r + 1], targets[r:r + 1], V, 1.0, 20)
        check_forward(one, logits[r:r + 1], targets[r:r + 1], V, 1.0, 20)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        outs = []
        for s in streams:
            with torch.cuda.stream(s):
                outs.append(run_forward(bfo, logits, targets, V, 1.0, 20))
        torch.cuda.synchronize()
        for o in outs:
            for k in whole:
                assert torch.equal(o[k], whole[k]), k


def test_binding_refusals(bfo):
    logits, targets = scores(4, 100, "bf16", 1)
    f = torch.empty(4, device=DEV)
    with pytest.raises(ValueError, match="vocab is 101"):
        bfo.token_logprobs_forward(logits, targets, f, vocab=101)
    with pytest.raises(TypeError, match="targets must be torch.int32"):
        bfo.token_logprobs_forward(logits, targets.long(), f)
    with pytest.raises(ValueError, match="stats has"):
        bfo.token_logprobs_forward(logits, targets, f, stats=f)
    with pytest.raises(bfo.BfoError):
        bfo.token_logprobs_forward(logits, targets, None)
    with pytest.raises(bfo.BfoError):
        bfo.token_logprobs_forward(logits, targets, f, scale=0.0)
    with pytest.raises(ValueError, match="row of its own"):
        bfo.token_logprobs_forward(logits, top_index=torch.empty(3, 2, dtype=torch.int32, device=DEV),
                                   top_logprob=torch.empty(4, 2, device=DEV))
    with pytest.raises(ValueError, match="shape"):
        bfo.token_logprobs_backward(logits, targets, torch.empty(4, 2, device=DEV), f, logits[:, :99])
    with pytest.raises(TypeError, match="teacher_index must be a torch.Tensor"):
        bfo.distill_forward(logits, None, f, f)
    with pytest.raises(ValueError, match="workspace must be"):
        bfo.token_logprobs_forward(logits, targets, f, workspace=16)
    index = torch.zeros(4, 0, dtype=torch.int32, device=DEV)
    with pytest.raises(bfo.BfoError):
        bfo.distill_forward(logits, index, torch.empty(4, 0, device=DEV), f)
    assert math.isfinite(bfo.logits_workspace_bytes(1, 1 << 28, 128))


@pytest.mark.parametrize("rows,V", [(5, 100), (600, 9001), (3, 70001)])
@pytest.mark.parametrize("scale", [1e37, 2.3e38, 2.4e38, 3.4028234663852886e38])
def test_largest_scales(bfo, rows, V, scale):
    """Scales up to binary32's largest, whose product with log2(e) is past it:
    rows of zeros, rows of equal scores and scores so small that z is of
    ordinary size.  (x - M) is exact on the subnormals' grid, so the counted
    roundings are the usual ones."""
    g = gen(rows)
    z = 3 * torch.empty(rows, V, device=DEV).normal_(generator=g)
    logits = (z.double() / single(scale)).float()
    logits[0] = 0.0
    logits[1] = 0.25 / single(scale)
    targets = torch.randint(0, V, (rows,), generator=g, device=DEV).to(torch.int32)
    out = run_forward(bfo, logits, targets, V, scale, 20)
    check_forward(out, logits, targets, V, scale, 20)
    factor = torch.full((rows,), 0.125, device=DEV)
    d = torch.full_like(logits, NAN)
    bfo.token_logprobs_backward(logits, targets, out["stats"], factor, d, entropy=out["entropy"], dentropy=factor,
                                scale=scale)
    sparse = torch.zeros(rows, V, dtype=torch.float64, device=DEV)
    sparse.scatter_(1, targets.long()[:, None], 0.125)
    check_gradient(d, V, *gradient_reference(logits, V, scale, out["stats"], -factor, -factor, out["entropy"], sparse))
    index, _ = teacher(rows, V, 20, 41)
    value = torch.gather(logits, 1, index.clamp(min=0).long()).contiguous()
    kl, _, lp = run_distill(bfo, logits, index, value, V, scale, targets)
    ref, _, _, _, want, tol = distill_reference(logits, V, scale, index, value, targets)
    near(kl, want, tol, "kl")
    near(lp, ref["at"], ref["at_tol"], "logprob")


def test_workspace_of_a_larger_call(bfo):
    """A full micro-batch's workspace serves its ragged last batch, which is split over workgroups."""
    V = 70001
    logits, targets = scores(64, V, "bf16", 61)
    ws = bfo.new_logits_workspace(8192, V + 5, 128, DEV)
    st, lp = torch.empty(64, 2, device=DEV), torch.empty(64, device=DEV)
    ti, tl = torch.empty(64, 20, dtype=torch.int32, device=DEV), torch.empty(64, 20, device=DEV)
    bfo.token_logprobs_forward(logits, targets, lp, st, top_index=ti, top_logprob=tl, workspace=ws)
    own = run_forward(bfo, logits, targets, V, 1.0, 20)
    for k, t in (("logprob", lp), ("stats", st), ("top_index", ti), ("top_logprob", tl)):
        assert torch.equal(t, own[k]), k
    index, value = teacher(64, V, 20, 62)
    kl = torch.empty(64, device=DEV)
    bfo.distill_forward(logits, index, value, kl, workspace=ws)
    assert torch.equal(kl, run_distill(bfo, logits, index, value, V, 1.0)[0])
    # calls that use none take none
    many, t = scores(129, V, "bf16", 63)
    lp = torch.empty(129, device=DEV)
    bfo.token_logprobs_forward(many, t, lp)
    assert torch.equal(lp, run_forward(bfo, many, t, V)["logprob"])


def test_rows_of_more_columns_than_32_bits(bfo):
    """A vocabulary or a width past 2^32 is out of range; a short vocabulary at the start of such a row is not."""
    wide = torch.zeros(1, (1 << 32) + 5, dtype=torch.bfloat16, device=DEV)
    st, one = torch.empty(1, 2, device=DEV), torch.ones(1, device=DEV)
    t = torch.zeros(1, dtype=torch.int32, device=DEV)
    index, value = torch.zeros(1, 2, dtype=torch.int32, device=DEV), torch.zeros(1, 2, device=DEV)
    for call in (lambda: bfo.token_logprobs_forward(wide, stats=st),
                 lambda: bfo.token_logprobs_backward(wide, t, st, one, wide, vocab=5),
                 lambda: bfo.distill_forward(wide, index, value, one.clone()),
                 lambda: bfo.distill_backward(wide, index, value, st, one, wide, vocab=5),
                 lambda: bfo.layernorm_forward(wide, wide[0], None, torch.empty_like(wide))):
        with pytest.raises(bfo.BfoError) as e:
            call()
        assert e.value.status == bfo.ERANGE
    bfo.token_logprobs_forward(wide, stats=st, vocab=5)
    near(st[0, 1], torch.tensor(5.0, device=DEV).double().log(), 4 * U, "log sum of five zeros")
    del wide
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("rows,V,pad", [(7, 5003, 2), (600, 2051, 0), (3, 70001, 1)])
def test_order_of_sums_and_where_rows_start(bfo, dt, rows, V, pad):
    """Sums over the vocabulary run in an order given by the sizes and by where
    in a 128-byte line the rows start: the same bits at starts that are equal
    modulo 128 bytes, the same values within the counted roundings at others,
    and the same tokens anywhere."""
    line = 128 // TYPES[dt].itemsize
    logits, targets = scores(rows, V, dt, 81, pad=pad)
    index, value = teacher(rows, V, 20, 82)
    flat = torch.empty(rows * (V + pad) + 4 * line, dtype=TYPES[dt], device=DEV)

    def at(start):
        view = flat[start:start + rows * (V + pad)].view(rows, V + pad)
        view.copy_(logits)
        out = run_forward(bfo, view, targets, V, 1.0, 20)
        out["kl"] = run_distill(bfo, view, index, value, V, 1.0)[0]
        return out

    first = at(0)
    for start in (line, 3 * line):
        again = at(start)
        for k in first:
            assert torch.equal(first[k], again[k]), (start, k)
    _, _, _, _, want, tol = distill_reference(logits, V, 1.0, index, value, targets)
    for start in (1, 2, line // 2, line - 1, line + 3):
        other = at(start)
        check_forward(other, logits, targets, V, 1.0, 20)
        near(other["kl"], want, tol, "kl")


@pytest.mark.parametrize("scale", [0.5, 1.7])
def test_teacher_side_at_a_temperature(bfo, scale):
    """At a temperature, the teacher's log probabilities at scale 1 serve, its scores do, and those at the
    temperature itself do once divided by it; undivided they are another teacher's."""
    V, K, R = 4001, 20, 50
    z, t = scores(R, V, "bf16", 21)
    student, _ = scores(R, V, "bf16", 22)
    plain, scaled = run_forward(bfo, z, t, V, 1.0, K), run_forward(bfo, z, t, V, scale, K)
    index = plain["top_index"]
    assert torch.equal(index, scaled["top_index"])
    raw = torch.gather(z.float(), 1, index.long())
    _, _, _, _, want, tol = distill_reference(student, V, scale, index, raw, t)
    s = single(scale)
    # a log probability is off by at most (V / 64 + 100) u and half a step of its size, below 2^6; kl moves by
    # s q (log q - log p - kl) per unit of a teacher's score, in all by at most s (2 kl + 1)
    off = 4 * max(s, 1 / s) * (V / 64 + 100 + 64) * U * (1 + want.abs())
    for value in (raw, plain["top_logprob"], scaled["top_logprob"] / s):
        near(run_distill(bfo, student, index, value.contiguous(), V, scale)[0], want, tol + off, "kl")
    again = run_distill(bfo, student, index, scaled["top_logprob"], V, scale)[0].double()
    _, _, _, _, other, tol = distill_reference(student, V, scale, index, raw * s, t)
    near(again, other, tol + off * (1 + other.abs()), "kl of the teacher scaled twice")
    assert ((again - want).abs() > 0.01).any()


def special_rows(logits, V):
    """Rows that are hard to pick the best of, over the first nine rows."""
    i = torch.arange(V, device=DEV)
    t = logits.dtype
    logits = logits.clone()
    logits[0, :V] = (i * 2.0 ** -6).to(t)                    # all the best in the last stretch (with ties in bf16)
    logits[1, :V] = (i * -2.0 ** -6).to(t)                   # in the first
    logits[2, :V] = (i % 5).to(t)                            # ties everywhere
    logits[3, :V] = torch.where(i >= V - 3, logits[3, :V].float(), -INF).to(t)   # fewer scores than asked for
    logits[4, : V - V // 3] = float(torch.finfo(t).min)
    logits[5, :V] = torch.where(i // 8 % 512 == 17, i % 89 * 0.25, -1.0).to(t)   # in one lane's columns
    logits[6, :V] += 100.0                                   # a common offset
    logits[7, :V] -= 100.0
    logits[8, V // 2] = NAN
    return logits


# (rows, vocabulary, type): a kept maximum covers two or three chunks of a lane's columns, with 512 lanes, with 256,
# with 256 and nontemporal loads, and in segments; then one chunk with nontemporal loads in binary32.
LONG = [(130, 131072, "bf16"), (200, 131071, "f32"), (520, 60001, "bf16"), (520, 30001, "f32"), (600, 65537, "bf16"),
        (600, 50257, "f32"), (9, 1 << 20, "bf16"), (9, (1 << 20) + 77, "f32"), (3001, 20011, "f32")]


@pytest.mark.parametrize("rows,V,dt", LONG)
def test_top_of_stretches_of_several_chunks(bfo, rows, V, dt):
    for k, top in enumerate((1, 20, 128)):
        scale = (1.0, 0.7, 1.7)[k]
        logits, targets = scores(rows, V, dt, 90 + k, pad=(0, 7, 64)[k])
        logits = special_rows(logits, V)
        targets[3] = V - 2
        out = run_forward(bfo, logits, targets, V, scale, top)
        index = top_reference_nan_first(logits[8:9], V, top)
        assert torch.equal(out["top_index"][8:9].long(), index)
        assert out["stats"][8].isnan().all() and out["top_logprob"][8].isnan().all()
        assert torch.equal(out["top_index"][3:4].long(), top_reference(logits[3:4], V, top))
        assert (out["top_logprob"][3, 3:] == -INF).all()
        # a target whose scaled score is past binary32 counts as -inf: the lowest bf16 or binary32 value times 1.7 is
        at = logits.gather(1, targets.clamp(min=0).long()[:, None])[:, 0].double() * single(scale)
        past = (targets >= 0) & (at < -float(torch.finfo(torch.float32).max))
        assert (out["logprob"][past] == -INF).all()
        targets, out["logprob"] = torch.where(past, -1, targets), torch.where(past, 0.0, out["logprob"])
        keep = torch.tensor([r for r in range(rows) if r not in (3, 8)], device=DEV)
        for part in keep.split(128):
            check_forward({n: t[part] for n, t in out.items()}, logits[part], targets[part], V, scale, top)
        check_forward({n: t[3:4] for n, t in out.items() if not n.startswith("top")}, logits[3:4], targets[3:4], V,
                      scale, 0)


@pytest.mark.parametrize("rows,V,dt", [(700, 50257, "bf16"), (600, 50257, "f32"), (2100, 20011, "bf16")])
def test_distill_of_more_scores_than_caches_hold(bfo, rows, V, dt):
    logits, targets = scores(rows, V, dt, 97, pad=3)
    index, value = teacher(rows, V, 65, 98)
    kl, stats, lp = run_distill(bfo, logits, index, value, V, 0.7, targets)
    for part in torch.arange(rows, device=DEV).split(128):
        ref, _, _, _, want, tol = distill_reference(logits[part], V, 0.7, index[part], value[part], targets[part])
        near(kl[part], want, tol, "kl")
        near(stats[part, 0], ref["m"], U * ref["m"].abs(), "max")
        near(stats[part, 1], ref["logs"], ref["rel"], "log sum")
        near(lp[part], ref["at"], ref["at_tol"], "logprob")


@pytest.mark.parametrize("V", [100, 70001])
@pytest.mark.parametrize("scale", [1e-45, 1e-40, 1e-38, 1e-30])
def test_smallest_scales(bfo, V, scale):
    """Down to subnormal scales, whose product with log2(e) is off by up to 2^-150: 2^-22 of an exponent."""
    logits = torch.full((3, V), 1e30, device=DEV)
    logits[1] = torch.linspace(-3e38, 3e38, V, dtype=torch.float64).float().to(DEV)
    logits[2] = torch.linspace(-1, 1, V, device=DEV)
    targets = torch.tensor([0, 7, -1], dtype=torch.int32, device=DEV)
    check_forward(run_forward(bfo, logits, targets, V, scale, 20), logits, targets, V, scale, 20)
    # a teacher of such scores
    index = torch.arange(30, dtype=torch.int32, device=DEV).repeat(3, 1) * 3
    value = torch.gather(logits, 1, index.long()).neg().contiguous()
    kl, _, lp = run_distill(bfo, logits, index, value, V, scale, targets)
    ref, _, _, _, want, tol = distill_reference(logits, V, scale, index, value, targets)
    near(kl, want, tol, "kl")
    near(lp, ref["at"], ref["at_tol"], "logprob")
