"""The operators between a transformer block's matrix products, as measured cases.

Root-mean-square norm with the residual's addition and 8-bit codes, the
feed-forward's activation with its inputs kept in 8 bits for the backward pass,
and rotary positions, each with its gradient.  `listed` names the cases, `draw`
gives more of the same ranges, `prepare` makes inputs from a seed, `run` does
one pass -- with elementary torch operations in 32 bits (angles in 64), or,
where `own` is set, through the library's entry points -- and `exact` gives the
same outputs in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-5
GROUP = 128                        # columns that share a scale, or a whole row
SMALLEST = 2.0 ** -126             # of a scale
TOP = {"e4m3": 448.0, "i8": 127.0}
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
CODES = {"e4m3": torch.float8_e4m3fn, "i8": torch.int8}
CUBIC, SLOPE = 0.044715, 2.0 * math.sqrt(2.0 / math.pi)


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # One norm of the 7B model's block over 8192 tokens: residual added, the normalised rows kept in 8 bits.
        _rms("rms_fwd_7b", "rms_fwd", 8192, 4096, "bf16", "bf16", "group", True),
        # A single sampled token: the next product reads 8 bits with one scale, nothing is kept.
        _rms("rms_fwd_token", "rms_fwd", 1, 4096, "bf16", "bf16", "row", True),
        # Its gradient from the kept codes, with the norm's output again for the weight's gradient.
        _rms("rms_bwd_7b", "rms_bwd", 8192, 4096, "bf16", "bf16", "group", True),
        # 32-bit rows of an odd width and count, kept as they are: a debugging run of a small model.
        _rms("rms_bwd_odd_f32", "rms_bwd", 1003, 801, "f32", "f32", "none", False),
        # The 7B model's gated feed-forward over 8192 tokens, both inputs kept in 8 bits.
        _act("act_fwd_7b", "act_fwd", 8192, 11008, "bf16", "silu", True, "e4m3"),
        # The same for one sampled token: nothing is kept.
        _act("act_fwd_token", "act_fwd", 1, 11008, "bf16", "silu", True, "none"),
        # Its gradient from what was kept, with the output again for the weight's gradient.
        _act("act_bwd_7b", "act_bwd", 8192, 11008, "bf16", "silu", True, "i8"),
        # The 1.5B model's feed-forward over a ragged micro-batch, forward and backward, without a gate.
        _act("act_step_1p5b", "act_step", 1003, 6400, "bf16", "gelu", False, "i8"),
        # Queries and keys of the 7B model over 8192 tokens of 2048-token sequences.
        _rope("rope_fwd_7b", "rope_fwd", 8192, 64, 128, 128, "bf16", "half", 2048, 1.0),
        # One sampled token far into a context whose positions are scaled.
        _rope("rope_token", "rope_fwd", 1, 64, 128, 128, "bf16", "half", 131072, 8.0),
        # The gradient of queries and keys, pairs side by side.
        _rope("rope_bwd_7b", "rope_bwd", 8192, 64, 128, 128, "bf16", "interleaved", 2048, 1.0),
        # 32 bits, a quarter of an odd head, far positions.
        _rope("rope_odd_f32", "rope_fwd", 1003, 25, 80, 20, "f32", "half", 1000000, 4.0),
    ]


def _rms(name, op, rows, cols, dtype, pdtype, codes, residual):
    """codes: "group" (of the normalised row), "row" (of the output, in its place) or "none"."""
    return {"name": name, "op": op, "rows": rows, "cols": cols, "dtype": dtype, "pdtype": pdtype, "codes": codes,
            "residual": residual}


def _act(name, op, rows, cols, dtype, kind, gated, codes):
    return {"name": name, "op": op, "rows": rows, "cols": cols, "dtype": dtype, "kind": kind, "gated": gated,
            "codes": codes}


def _rope(name, op, tokens, heads, dim, rotated, dtype, layout, reach, factor):
    """reach: positions lie below it; factor: of the context's extension."""
    return {"name": name, "op": op, "tokens": tokens, "heads": heads, "dim": dim, "rotated": rotated, "dtype": dtype,
            "layout": layout, "reach": reach, "factor": factor}


def _spread(rng, lo, hi):
    """An integer spread over [lo, hi] by its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rms_fwd", "rms_bwd", "act_fwd", "act_bwd", "act_step", "rope_fwd", "rope_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    half = 1 if dtype == "bf16" else 2
    if op.startswith("rms"):
        cols = _spread(rng, 16, 16384)
        rows = _spread(rng, 1, min(16384, (8192 * 4096) // half // cols))
        codes = rng.choice(["group", "none", "row"] if op == "rms_fwd" else ["group", "none"])
        case = _rms("", op, rows, cols, dtype, rng.choice([dtype, "f32"]), codes, rng.random() < 0.7)
    elif op.startswith("act"):
        # What the step keeps is rounded to 8 bits: where 32-bit results follow, both sides would have to agree on
        # every tie.
        dtype, half = ("bf16", 1) if op == "act_step" else (dtype, half)
        cols = _spread(rng, 16, 32768)
        most = 8192 * 11008 // half // (2 if op == "act_step" else 1)
        rows = _spread(rng, 1, min(16384, most // cols))
        codes = rng.choice({"act_fwd": ["e4m3", "e4m3", "none"], "act_bwd": ["i8", "e4m3", "none"],
                            "act_step": ["i8", "e4m3"]}[op])
        case = _act("", op, rows, cols, dtype, rng.choice(["silu", "gelu"]), rng.random() < 0.6, codes)
    else:
        dim = rng.choice([32, 64, 80, 96, 100, 128, 192, 256])
        rotated = rng.choice([dim, dim, dim // 2, dim // 4 // 2 * 2])
        heads = rng.randint(1, 80)
        tokens = _spread(rng, 1, min(16384, 8192 * 64 * 128 // half // (heads * dim)))
        case = _rope("", op, tokens, heads, dim, rotated, dtype, rng.choice(["half", "interleaved"]),
                     _spread(rng, 128, 1000000), rng.choice([1.0, 1.0, 4.0, 8.0]))
    del case["name"]
    return case


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 1000003 + 29)
    return {"rms": _prepare_rms, "act": _prepare_act, "rop": _prepare_rope}[case["op"][:3]](case, g)


def _normal(g, *shape):
    return torch.empty(shape, dtype=torch.float32, device=DEV).normal_(0.0, 1.0, generator=g)


def _empty_codes(rows, cols, kind, per_row=False):
    groups = 1 if per_row else (cols + GROUP - 1) // GROUP
    return (torch.empty(rows, cols, dtype=CODES[kind], device=DEV),
            torch.empty(rows, groups, dtype=torch.float32, device=DEV))


def _kept(v, kind):
    """Codes and scales of the groups of v, as a forward pass left them."""
    rows, cols = v.shape
    wide = torch.nn.functional.pad(v, (0, -cols % GROUP)).view(rows, -1, GROUP)
    scales = (wide.abs().amax(2) * (1.0 / TOP[kind])).clamp(min=SMALLEST)
    wide = (wide * (1.0 / scales)[:, :, None]).view(rows, -1)[:, :cols]
    return (wide.round() if kind == "i8" else wide).to(CODES[kind]).contiguous(), scales


def _prepare_rms(case, g):
    R, C, dt, pdt = case["rows"], case["cols"], DTYPES[case["dtype"]], DTYPES[case["pdtype"]]
    # A residual stream: channels of different size, a few of them large, and what the layer adds to it.
    size = torch.exp(0.5 * _normal(g, C))
    size[:: max(1, C // 4)] *= 8.0
    x = (_normal(g, R, C) * size).to(dt)
    s = {"case": case, "x": x, "weight": (1.0 + 0.2 * _normal(g, C)).to(pdt)}
    if case["op"] == "rms_fwd":
        s["rstd"] = torch.empty(R, device=DEV)
        if case["residual"]:
            s.update(residual=(0.3 * _normal(g, R, C) * size).to(dt), total=torch.empty_like(x))
        if case["codes"] != "row":
            s["out"] = torch.empty_like(x)
        if case["codes"] != "none":
            s["codes"], s["scales"] = _empty_codes(R, C, "e4m3", case["codes"] == "row")
        return s
    f = x.float()
    s["rstd"] = ((f * f).sum(1, dtype=torch.float64) / C + EPS).rsqrt().float()
    if case["codes"] == "group":
        s["codes"], s["scales"] = _kept(f * s["rstd"][:, None], "i8")
        del s["x"]
    s.update(dout=(1e-3 * _normal(g, R, C)).to(dt), dx=torch.empty_like(x),
             dweight=torch.empty(C, dtype=pdt, device=DEV))
    if case["residual"]:  # in a block: its output is wanted again
        s["out"] = torch.empty_like(x)
    return s


def _prepare_act(case, g):
    R, C, dt = case["rows"], case["cols"], DTYPES[case["dtype"]]
    # Projections of normalised rows: channels of different size, a few of them large.
    size = torch.exp(0.4 * _normal(g, C))
    size[:: max(1, C // 5)] *= 6.0
    s = {"case": case}
    names = ["gate", "up"] if case["gated"] else ["gate"]
    s.update((n, (_normal(g, R, C) * size).to(dt)) for n in names)
    if case["op"] != "act_bwd":
        s["out"] = torch.empty(R, C, dtype=dt, device=DEV)
        if case["codes"] != "none":
            for n in names:
                s[n + "_codes"], s[n + "_scales"] = _empty_codes(R, C, case["codes"])
    elif case["codes"] != "none":
        for n in names:
            s[n + "_codes"], s[n + "_scales"] = _kept(s.pop(n).float(), case["codes"])
    if case["op"] != "act_fwd":
        s["dout"] = (1e-3 * _normal(g, R, C)).to(dt)
        s.update(("d" + n, torch.empty(R, C, dtype=dt, device=DEV)) for n in names)
        s["again"] = torch.empty(R, C, dtype=dt, device=DEV)
    return s


def _prepare_rope(case, g):
    T, H, D, r = case["tokens"], case["heads"], case["dim"], case["rotated"]
    x = _normal(g, T, H, D).to(DTYPES[case["dtype"]])
    first = torch.randint(0, max(1, case["reach"] - T), (1,), generator=g, device=DEV)
    positions = ((first + torch.arange(T, device=DEV)) % case["reach"]).to(torch.int32)
    pair = torch.arange(r // 2, dtype=torch.float64, device=DEV)
    return {"case": case, "x": x, "out": torch.empty_like(x), "positions": positions,
            "frequencies": 10000.0 ** (-2.0 * pair / r) / case["factor"]}


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(state):
    return (_OWN if own else _PLAIN)[state["case"]["op"]](state)


def _plain_codes(v, kind, per_row=False):
    """(codes, scales) of the groups of v, or of its rows."""
    rows, cols = v.shape
    group = cols if per_row else GROUP
    wide = torch.nn.functional.pad(v, (0, -cols % group)).view(rows, -1, group)
    scales = (wide.abs().amax(2) * (1.0 / TOP[kind])).clamp(min=SMALLEST)
    wide = (wide * (1.0 / scales)[:, :, None]).view(rows, -1)[:, :cols]
    return (wide.round() if kind == "i8" else wide).to(CODES[kind]), scales


def _plain_values(codes, scales):
    rows, cols = codes.shape
    return codes.float() * scales.repeat_interleave(GROUP, 1)[:, :cols]


def _plain_rms_fwd(s):
    c = s["case"]
    t = s["x"].float()
    out = {}
    if c["residual"]:
        out["total"] = (t + s["residual"].float()).to(s["x"].dtype)
        t = out["total"].float()
    rstd = 1.0 / torch.sqrt((t * t).sum(1) / c["cols"] + EPS)
    xhat = t * rstd[:, None]
    y = xhat * s["weight"].float()
    out["rstd"] = rstd
    if c["codes"] != "row":
        out["out"] = y.to(s["x"].dtype)
    if c["codes"] != "none":
        out["codes"], out["scales"] = _plain_codes(*((y, "e4m3", True) if c["codes"] == "row" else (xhat, "e4m3")))
    return out


def _plain_rms_bwd(s):
    C, w = s["case"]["cols"], s["weight"].float()
    dout, rstd = s["dout"].float(), s["rstd"][:, None]
    xhat = _plain_values(s["codes"], s["scales"]) if "codes" in s else s["x"].float() * rstd
    h = dout * w
    dx = (h - xhat * ((h * xhat).sum(1, keepdim=True) / C)) * rstd
    out = {"dx": dx.to(s["dx"].dtype), "dweight": (dout * xhat).sum(0).to(s["weight"].dtype)}
    if "out" in s:
        out["out"] = (xhat * w).to(s["out"].dtype)
    return out


def _plain_sigmoid(kind, g):
    """(sigma(z), dz/dg) of an activation g * sigma(z)."""
    z = g if kind == "silu" else SLOPE * (g + CUBIC * g * g * g)
    return 1.0 / (1.0 + torch.exp(-z)), 1.0 if kind == "silu" else SLOPE * (1.0 + 3.0 * CUBIC * g * g)


def _plain_act_fwd(s):
    c = s["case"]
    g = s["gate"].float()
    y = g * _plain_sigmoid(c["kind"], g)[0]
    if c["gated"]:
        y = y * s["up"].float()
    out = {"out": y.to(s["gate"].dtype)}
    if c["codes"] != "none":
        out["gate_codes"], out["gate_scales"] = _plain_codes(g, c["codes"])
        if c["gated"]:
            out["up_codes"], out["up_scales"] = _plain_codes(s["up"].float(), c["codes"])
    return out


def _plain_act_gradient(s, g, up):
    dout, dt = s["dout"].float(), s["dout"].dtype
    sigma, slope = _plain_sigmoid(s["case"]["kind"], g)
    act = g * sigma
    into = dout if up is None else dout * up
    out = {"dgate": (into * (sigma + act * (1.0 - sigma) * slope)).to(dt),
           "again": (act if up is None else act * up).to(dt)}
    if up is not None:
        out["dup"] = (dout * act).to(dt)
    return out


def _plain_act_bwd(s):
    gated = s["case"]["gated"]
    if s["case"]["codes"] == "none":
        return _plain_act_gradient(s, s["gate"].float(), s["up"].float() if gated else None)
    up = _plain_values(s["up_codes"], s["up_scales"]) if gated else None
    return _plain_act_gradient(s, _plain_values(s["gate_codes"], s["gate_scales"]), up)


def _plain_act_step(s):
    f = _plain_act_fwd(s)
    up = _plain_values(f["up_codes"], f["up_scales"]) if s["case"]["gated"] else None
    out = _plain_act_gradient(s, _plain_values(f["gate_codes"], f["gate_scales"]), up)
    out["out"] = f["out"]
    return out


def _plain_rope(s):
    c, r = s["case"], s["case"]["rotated"]
    angle = s["positions"].double()[:, None] * s["frequencies"]
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    if c["op"] == "rope_bwd":
        sin = -sin
    x = s["x"].float()
    out = x.clone()
    first, second = (slice(0, r // 2), slice(r // 2, r)) if c["layout"] == "half" else (slice(0, r, 2), slice(1, r, 2))
    a, b = x[:, :, first], x[:, :, second]
    out[:, :, first] = a * cos - b * sin
    out[:, :, second] = a * sin + b * cos
    return {"out": out.to(s["x"].dtype)}


def _library():
    from bf16_numerics_amd import binding
    return binding


def _own_rms_fwd(s):
    bfo = _library()
    bfo.rmsnorm_forward(s["x"], s["weight"], s.get("out"), residual=s.get("residual"), total=s.get("total"),
                        rstd=s["rstd"], codes=s.get("codes"), scales=s.get("scales"),
                        codes_of=bfo.CODES_OF_OUT if s["case"]["codes"] == "row" else bfo.CODES_OF_NORMALISED,
                        eps=EPS)
    return {k: s[k] for k in ("total", "rstd", "out", "codes", "scales") if k in s}


def _own_rms_bwd(s):
    bfo, c = _library(), s["case"]
    if "workspace" not in s:  # the scratch memory a training loop allocates once and keeps
        s["workspace"] = bfo.new_rmsnorm_workspace(c["rows"], c["cols"], s["dout"].device)
    bfo.rmsnorm_backward(s["dout"], s.get("x"), s["weight"], s["rstd"], s["dx"], s["dweight"], codes=s.get("codes"),
                         scales=s.get("scales"), out=s.get("out"), workspace=s["workspace"])
    return {k: s[k] for k in ("dx", "dweight", "out") if k in s}


def _own_kept(s):
    return {k: s.get(k) for k in ("gate_codes", "gate_scales", "up_codes", "up_scales")}


def _own_act_fwd(s):
    bfo = _library()
    bfo.activation_forward(s["gate"], s.get("up"), s["out"], kind=_own_kind(bfo, s), **_own_kept(s))
    return {k: s[k] for k in ("out", "gate_codes", "gate_scales", "up_codes", "up_scales") if k in s}


def _own_kind(bfo, s):
    return bfo.SILU if s["case"]["kind"] == "silu" else bfo.GELU


def _own_act_bwd(s):
    bfo = _library()
    bfo.activation_backward(s["dout"], s.get("gate"), s.get("up"), s["dgate"], s.get("dup"), kind=_own_kind(bfo, s),
                            out=s["again"], **_own_kept(s))
    return {k: s[k] for k in ("dgate", "dup", "again") if k in s}


def _own_act_step(s):
    bfo = _library()
    kind, kept = _own_kind(bfo, s), _own_kept(s)
    bfo.activation_forward(s["gate"], s.get("up"), s["out"], kind=kind, **kept)
    bfo.activation_backward(s["dout"], None, None, s["dgate"], s.get("dup"), kind=kind, out=s["again"], **kept)
    return {k: s[k] for k in ("out", "dgate", "dup", "again") if k in s}


def _own_rope(s):
    bfo, c = _library(), s["case"]
    bfo.rotary_apply(s["x"], s["frequencies"], s["out"], positions=s["positions"],
                     layout=bfo.ROTARY_HALF if c["layout"] == "half" else bfo.ROTARY_INTERLEAVED,
                     backward=c["op"] == "rope_bwd")
    return {"out": s["out"]}


_PLAIN = {"rms_fwd": _plain_rms_fwd, "rms_bwd": _plain_rms_bwd, "act_fwd": _plain_act_fwd, "act_bwd": _plain_act_bwd,
          "act_step": _plain_act_step, "rope_fwd": _plain_rope, "rope_bwd": _plain_rope}
_OWN = {"rms_fwd": _own_rms_fwd, "rms_bwd": _own_rms_bwd, "act_fwd": _own_act_fwd, "act_bwd": _own_act_bwd,
        "act_step": _own_act_step, "rope_fwd": _own_rope, "rope_bwd": _own_rope}


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    b = 2 if case["dtype"] == "bf16" else 4
    if case["op"].startswith("rope"):
        T, H, D, r = case["tokens"], case["heads"], case["dim"], case["rotated"]
        return {"bytes": 2 * b * T * H * D + 4 * T + 4 * r, "flops": 3 * T * H * r}
    R, C = case["rows"], case["cols"]
    coded = 1 + 4 / GROUP  # bytes of a value in 8 bits and its share of a scale
    if case["op"].startswith("rms"):
        pb = 2 if case["pdtype"] == "bf16" else 4
        kept = coded if case["codes"] == "group" else 1
        if case["op"] == "rms_fwd":
            each = b * (1 + 2 * case["residual"] + (case["codes"] != "row")) + kept * (case["codes"] != "none")
            return {"bytes": int(each * R * C) + pb * C + 4 * R, "flops": 6 * R * C}
        each = (kept if case["codes"] == "group" else b) + b * (2 + case["residual"])
        return {"bytes": int(each * R * C) + 2 * pb * C + 4 * R, "flops": 10 * R * C}
    n = 2 if case["gated"] else 1
    kept = coded if case["codes"] != "none" else 0
    forward = n * (b + kept) + b
    backward = n * ((kept or b) + b) + 2 * b
    if case["op"] == "act_fwd":
        return {"bytes": int(forward * R * C), "flops": 8 * R * C}
    if case["op"] == "act_bwd":
        return {"bytes": int(backward * R * C), "flops": 16 * R * C}
    # What the step keeps is read again, but is no output of it.
    return {"bytes": int((n * b + b + n * b + 2 * b) * R * C), "flops": 24 * R * C}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"rms": _exact_rms, "act": _exact_act, "rop": _exact_rope}[case["op"][:3]](case, s)


def _exact_scales(v, kind, cols_each):
    """The scale of every group of v and, per column, the group's."""
    parts = [p.abs().amax(1) for p in v.split(cols_each, 1)]
    scales = (torch.stack(parts, 1) / TOP[kind]).clamp(min=SMALLEST)
    return scales, scales[:, torch.arange(v.shape[1], device=DEV) // cols_each]


def _exact_codes(v, kind, cols_each=GROUP):
    """The values that the codes stand for in units of their scales, and the scales."""
    scales, each = _exact_scales(v, kind, cols_each)
    a = v / each
    if kind == "i8":
        return torch.round(a), scales
    # Three bits behind the leading one; below 2^-6 steps of 2^-9.
    step = torch.ldexp(torch.ones_like(a), torch.frexp(a).exponent.clamp(min=-5) - 4)
    return torch.round(a / step) * step, scales


def _exact_values(codes, scales):
    return codes.double() * scales.double()[:, torch.arange(codes.shape[1], device=DEV) // GROUP]


def _exact_rms(case, s):
    C, w = case["cols"], s["weight"].double()
    if case["op"] == "rms_fwd":
        t, out = s["x"].double(), {}
        if case["residual"]:
            out["total"] = t + s["residual"].double()
            t = out["total"].to(s["x"].dtype).double()  # the norm is that of the stored row
        out["rstd"] = (t.square().mean(1) + EPS).pow(-0.5)
        xhat = t * out["rstd"][:, None]
        if case["codes"] != "row":
            out["out"] = xhat * w
        if case["codes"] == "row":
            out["codes"], out["scales"] = _exact_codes(xhat * w, "e4m3", C)
        elif case["codes"] == "group":
            out["codes"], out["scales"] = _exact_codes(xhat, "e4m3")
        return out
    rstd, dout = s["rstd"].double()[:, None], s["dout"].double()
    xhat = _exact_values(s["codes"], s["scales"]) if "codes" in s else rstd * s["x"].double()
    # dx is rstd times what is left of w * dout after its projection on xhat.
    h = w * dout
    out = {"dx": rstd * (h - xhat * (xhat * h).mean(1, keepdim=True)), "dweight": (dout * xhat).sum(0)}
    if "out" in s:
        out["out"] = w * xhat
    return out


def _exact_act(case, s):
    def act(g):
        """The activation and its derivative, through tanh."""
        if case["kind"] == "silu":
            half = torch.tanh(0.5 * g)
            return 0.5 * g * (1 + half), 0.5 * (1 + half) + 0.25 * g * (1 - half * half)
        k = math.sqrt(2.0 / math.pi)
        t = torch.tanh(k * (g + CUBIC * g.pow(3)))
        return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * k * (1 + 3 * CUBIC * g.square())

    out = {}
    names = ["gate", "up"] if case["gated"] else ["gate"]
    if case["op"] != "act_bwd":
        value = act(s["gate"].double())[0]
        out["out"] = value * s["up"].double() if case["gated"] else value
    kept = {}
    if case["codes"] == "none":
        kept = {n: s[n].double() for n in names}
    elif case["op"] == "act_bwd":
        kept = {n: _exact_values(s[n + "_codes"], s[n + "_scales"]) for n in names}
    else:
        for n in names:
            codes, scales = _exact_codes(s[n].double(), case["codes"])
            if case["op"] == "act_fwd":
                out[n + "_codes"], out[n + "_scales"] = codes, scales
            kept[n] = _exact_values(codes, scales)
    if case["op"] == "act_fwd":
        return out
    value, slope = act(kept["gate"])
    dout, up = s["dout"].double(), kept.get("up", 1.0)
    out["dgate"], out["again"] = dout * up * slope, value * up
    if case["gated"]:
        out["dup"] = dout * value
    return out


def _exact_rope(case, s):
    T, H, r = case["tokens"], case["heads"], case["rotated"]
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEV),
                       s["positions"].double()[:, None] * s["frequencies"])[:, None]
    turn = turn.conj() if case["op"] == "rope_bwd" else turn
    x = s["x"].double()
    out = x.clone()
    if case["layout"] == "half":
        pairs = x[:, :, :r].reshape(T, H, 2, r // 2).transpose(2, 3)
    else:
        pairs = x[:, :, :r].reshape(T, H, r // 2, 2)
    turned = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
    out[:, :, :r] = (turned.transpose(2, 3) if case["layout"] == "half" else turned).reshape(T, H, r)
    return {"out": out}
