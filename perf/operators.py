"""The training-loop operators around the optimizer step, as measured cases.

Three operators with their gradients: layer norm (its weight and bias
gradients are what the grad norm and the update read), the log probabilities
of given tokens with entropy and top alternatives, and distillation from a
teacher's top logits.  `listed` names the cases, `draw` gives more of the same
ranges, `prepare` makes inputs from a seed, `run` does one pass -- with
elementary torch operations in 32 bits, or, where `own` is set, through the
library's entry points -- and `exact` gives the same outputs in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-5
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # One layer norm of the 124M model over a micro-batch of 8 sequences of 1024 tokens.
        _ln("ln_fwd_124m", "ln_fwd", 8192, 768, "bf16", "bf16"),
        # A single token through one layer norm of the 1.5B model: sampling, where latency counts.
        _ln("ln_fwd_token", "ln_fwd", 1, 1600, "bf16", "bf16"),
        # The 1.5B model's layer norm backward over 16 sequences: the bulk of a training run's calls.
        _ln("ln_bwd_1p5b", "ln_bwd", 16384, 1600, "bf16", "bf16"),
        # 32-bit activations of an odd width and row count: a debugging run of a small model.
        _ln("ln_bwd_odd_f32", "ln_bwd", 1003, 801, "f32", "f32"),
        # Evaluation of a micro-batch: every next token's log probability, the entropy, and the 20
        # most likely tokens; 50,257 tokens of a head padded to 50,304 columns, prompts masked.
        _lp("lp_fwd_eval", "lp_fwd", 8192, 50257, 50304, "bf16", 1.0, 0.1, 20),
        # One sampled token at a temperature, with five alternatives, as a server reports it.
        _lp("lp_fwd_token", "lp_fwd", 1, 32000, 32000, "bf16", 0.8, 0.0, 5),
        # The training loss's gradient for a micro-batch (cross entropy with an entropy bonus).
        _lp("lp_bwd_train", "lp_bwd", 8192, 50257, 50304, "bf16", 1.0, 0.1, 0),
        # The same in 32 bits at odd sizes whose rows start off every boundary.
        _lp("lp_bwd_odd_f32", "lp_bwd", 257, 50257, 50257, "f32", 1.0, 0.1, 0),
        # A student's loss against a teacher's 64 best tokens, and the true tokens beside it.
        _kd("kd_fwd_train", "kd_fwd", 4096, 32000, 32000, "bf16", 0.5, 0.1, 64, True),
        # A short sequence against few teacher tokens: a small fine-tuning step.
        _kd("kd_fwd_short", "kd_fwd", 63, 50257, 50304, "bf16", 1.0, 0.1, 20, False),
        # The student's gradient for a full micro-batch, both losses in one pass.
        _kd("kd_bwd_train", "kd_bwd", 8192, 50257, 50304, "bf16", 0.5, 0.1, 64, True),
        # 32-bit logits of an odd vocabulary, a ragged micro-batch, the teacher alone.
        _kd("kd_bwd_odd_f32", "kd_bwd", 301, 32001, 32001, "f32", 1.0, 0.2, 50, False),
    ]


def _ln(name, op, rows, cols, dtype, pdtype):
    return {"name": name, "op": op, "rows": rows, "cols": cols, "dtype": dtype, "pdtype": pdtype}


def _lp(name, op, rows, vocab, width, dtype, scale, masked, top):
    return {"name": name, "op": op, "rows": rows, "vocab": vocab, "width": width, "dtype": dtype,
            "scale": scale, "masked": masked, "top": top}


def _kd(name, op, rows, vocab, width, dtype, scale, masked, count, hard):
    return {"name": name, "op": op, "rows": rows, "vocab": vocab, "width": width, "dtype": dtype,
            "scale": scale, "masked": masked, "count": count, "hard": hard}


def _spread(rng, lo, hi):
    """An integer spread over [lo, hi] by its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["ln_fwd", "ln_bwd", "lp_fwd", "lp_bwd", "kd_fwd", "kd_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op.startswith("ln"):
        cols = _spread(rng, 16, 8192)
        rows = _spread(rng, 1, min(16384, (1 << 25) // cols))
        case = _ln("", op, rows, cols, dtype, rng.choice([dtype, "f32"]))
    else:
        vocab = _spread(rng, 128, 131072)
        width = rng.choice([vocab, (vocab + 63) // 64 * 64, vocab + rng.randint(1, 40)])
        most = 8192 * 50304 // (1 if dtype == "bf16" else 2)
        rows = _spread(rng, 1, min(8192, most // width))
        scale = rng.choice([1.0, 0.5, 0.8])
        masked = rng.choice([0.0, 0.1, 0.5])
        if op.startswith("lp"):
            top = rng.choice([0, 1, 5, 20, 64]) if op == "lp_fwd" else 0
            case = _lp("", op, rows, vocab, width, dtype, scale, masked, top)
        else:
            case = _kd("", op, rows, vocab, width, dtype, scale, masked, rng.choice([1, 8, 20, 50, 64, 128]),
                       rng.random() < 0.5)
    del case["name"]
    return case


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 1000003 + 17)
    return _prepare_ln(case, g) if case["op"].startswith("ln") else _prepare_logits(case, g)


def _normal(g, *shape):
    return torch.empty(shape, dtype=torch.float32, device=DEV).normal_(0.0, 1.0, generator=g)


def _prepare_ln(case, g):
    R, C, dt, pdt = case["rows"], case["cols"], DTYPES[case["dtype"]], DTYPES[case["pdtype"]]
    # A residual stream: channels of different size around an offset of their own, a few of them large.
    size = torch.exp(0.5 * _normal(g, C))
    size[:: max(1, C // 4)] *= 8.0
    x = (_normal(g, R, C) * size + 0.5 * _normal(g, C)).to(dt)
    s = {"case": case, "x": x, "weight": (1.0 + 0.1 * _normal(g, C)).to(pdt), "bias": (0.1 * _normal(g, C)).to(pdt)}
    if case["op"] == "ln_fwd":
        s.update(out=torch.empty_like(x), mean=torch.empty(R, device=DEV), rstd=torch.empty(R, device=DEV))
    else:
        x64 = x.double()
        mean = x64.mean(1)
        s.update(mean=mean.float(), rstd=(x64.var(1, unbiased=False) + EPS).rsqrt().float(),
                 dout=(1e-3 * _normal(g, R, C)).to(dt), dx=torch.empty_like(x),
                 dweight=torch.empty(C, dtype=pdt, device=DEV), dbias=torch.empty(C, dtype=pdt, device=DEV))
    return s


def _prepare_logits(case, g):
    R, V, W, dt = case["rows"], case["vocab"], case["width"], DTYPES[case["dtype"]]
    # Scores of a trained model: a broad bulk, and the true token raised by some amount in most rows.
    z = 2.0 * _normal(g, R, W)
    targets = torch.randint(0, V, (R,), generator=g, device=DEV)
    z[torch.arange(R, device=DEV), targets] += 12.0 * torch.rand(R, generator=g, device=DEV)
    live = torch.rand(R, generator=g, device=DEV) >= case["masked"]
    live[0] = True
    live_count = max(1, R - int(R * case["masked"]))
    s = {"case": case, "targets": torch.where(live, targets, -1).to(torch.int32)}
    if case["op"].startswith("kd"):
        K = case["count"]
        teacher = z[:, :V] + 0.7 * _normal(g, R, V)
        value, index = torch.topk(teacher, K, dim=1)
        del teacher
        # Some rows carry fewer teacher tokens than K; masked rows carry none.
        kept = torch.randint(max(1, K // 2), 2 * K + 1, (R, 1), generator=g, device=DEV)
        used = (torch.arange(K, device=DEV)[None, :] < kept) & live[:, None]
        s.update(teacher_index=torch.where(used, index, -1).to(torch.int32), teacher_logits=value.contiguous())
    logits = z.to(dt)
    s["logits"] = logits
    f = dict(dtype=torch.float32, device=DEV)
    if case["op"] == "lp_fwd":
        s.update(logprob=torch.empty(R, **f), stats=torch.empty(R, 2, **f), entropy=torch.empty(R, **f))
        if case["top"]:
            s.update(top_index=torch.empty(R, case["top"], dtype=torch.int32, device=DEV),
                     top_logprob=torch.empty(R, case["top"], **f))
    elif case["op"] == "kd_fwd":
        s.update(kl=torch.empty(R, **f), stats=torch.empty(R, 2, **f))
        if case["hard"]:
            s.update(logprob=torch.empty(R, **f))
    else:
        # What the forward pass left behind: the row's largest score, the log of the sum, the entropy.
        z = logits[:, :V].float() * case["scale"]
        m = z.amax(1, keepdim=True)
        z -= m
        e = torch.exp(z)
        total = e.sum(1, dtype=torch.float64)
        logsum = torch.log(total)
        s["stats"] = torch.stack([m[:, 0], logsum.float()], 1).contiguous()
        s["dlogits"] = torch.empty_like(logits)
        if case["op"] == "lp_bwd":
            s["entropy"] = (logsum - (e * z).sum(1, dtype=torch.float64) / total).float()
            s["dlogprob"] = torch.where(live, -1.0 / live_count, 0.0).float()
            s["dentropy"] = torch.where(live, -0.01 / live_count, 0.0).float()
        else:
            s["dkl"] = torch.where(live, 1.0 / live_count, 0.0).float()
            if case["hard"]:
                s["dlogprob"] = torch.where(live, -0.5 / live_count, 0.0).float()
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(state):
    return (_OWN if own else _PLAIN)[state["case"]["op"]](state)


def _plain_ln_fwd(s):
    C = s["case"]["cols"]
    x = s["x"].float()
    mean = x.sum(1) / C
    d = x - mean[:, None]
    rstd = 1.0 / torch.sqrt((d * d).sum(1) / C + EPS)
    out = d * rstd[:, None] * s["weight"].float() + s["bias"].float()
    return {"out": out.to(s["x"].dtype), "mean": mean, "rstd": rstd}


def _plain_ln_bwd(s):
    C = s["case"]["cols"]
    dout = s["dout"].float()
    xhat = (s["x"].float() - s["mean"][:, None]) * s["rstd"][:, None]
    h = dout * s["weight"].float()
    c1 = h.sum(1, keepdim=True) / C
    c2 = (h * xhat).sum(1, keepdim=True) / C
    dx = (h - c1 - xhat * c2) * s["rstd"][:, None]
    return {"dx": dx.to(s["x"].dtype), "dweight": (dout * xhat).sum(0).to(s["weight"].dtype),
            "dbias": dout.sum(0).to(s["bias"].dtype)}


def _plain_scores(s):
    """(scores minus the row's largest, that largest, the log of the sum of exponentials)."""
    z = s["logits"][:, :s["case"]["vocab"]].float() * s["case"]["scale"]
    m = z.amax(1, keepdim=True)
    z = z - m
    return z, m, torch.exp(z).sum(1, keepdim=True).log()


def _plain_at(z, logsum, targets):
    """The targets' log probabilities; 0 for masked rows."""
    at = torch.gather(z, 1, targets.clamp(min=0).long()[:, None]) - logsum
    return torch.where(targets >= 0, at[:, 0], 0.0)


def _plain_lp_fwd(s):
    z, m, logsum = _plain_scores(s)
    p = torch.exp(z - logsum)
    out = {"logprob": _plain_at(z, logsum, s["targets"]), "stats": torch.cat([m, logsum], 1),
           "entropy": logsum[:, 0] - (p * z).sum(1)}
    K, V = s["case"]["top"], s["case"]["vocab"]
    if K:
        # Unique whole-number keys: the score's order first, then the lower index.
        bits = (s["logits"][:, :V].float() + 0.0).view(torch.int32)
        key = (bits ^ ((bits >> 31) & 0x7FFFFFFF)).to(torch.int64) * (1 << 32)
        key += (V - 1) - torch.arange(V, device=DEV)
        best = torch.topk(key, K, dim=1).values
        index = (V - 1) - (best & 0xFFFFFFFF)
        out["top_index"] = index.to(torch.int32)
        out["top_logprob"] = torch.gather(z, 1, index) - logsum
    return out


def _plain_probabilities(s):
    z = s["logits"][:, :s["case"]["vocab"]].float() * s["case"]["scale"]
    logp = z - s["stats"][:, :1] - s["stats"][:, 1:]
    return torch.exp(logp), logp


def _plain_spread(s, d):
    """Gradients of the scores as gradients of the logits; padding columns get 0."""
    V, W = s["case"]["vocab"], s["case"]["width"]
    out = torch.zeros_like(s["logits"]) if W > V else torch.empty_like(s["logits"])
    out[:, :V] = (d * s["case"]["scale"]).to(out.dtype)
    return out


def _plain_hard(s, d, p):
    """Adds the gradient of the targets' log probabilities."""
    t = s["targets"]
    w = torch.where(t >= 0, s["dlogprob"], 0.0)[:, None]
    d = d - w * p
    return d.scatter_add_(1, t.clamp(min=0).long()[:, None], w)


def _plain_lp_bwd(s):
    p, logp = _plain_probabilities(s)
    d = -s["dentropy"][:, None] * p * (logp + s["entropy"][:, None])
    return {"dlogits": _plain_spread(s, _plain_hard(s, d, p))}


def _plain_teacher(s):
    """(the teacher's probabilities, their logarithms, 1 for rows with any entry)."""
    used = s["teacher_index"] >= 0
    t = torch.where(used, s["teacher_logits"] * s["case"]["scale"], -math.inf)
    any_used = used.any(1, keepdim=True)
    t = t - torch.where(any_used, t.amax(1, keepdim=True), 0.0)
    e = torch.exp(t)
    total = torch.where(any_used, e.sum(1, keepdim=True), 1.0)
    return e / total, t - total.log(), any_used.float()


def _plain_kd_fwd(s):
    z, m, logsum = _plain_scores(s)
    q, logq, _ = _plain_teacher(s)
    logp = torch.gather(z, 1, s["teacher_index"].clamp(min=0).long()) - logsum
    out = {"kl": torch.where(q > 0, q * (logq - logp), 0.0).sum(1), "stats": torch.cat([m, logsum], 1)}
    if s["case"]["hard"]:
        out["logprob"] = _plain_at(z, logsum, s["targets"])
    return out


def _plain_kd_bwd(s):
    p, _ = _plain_probabilities(s)
    q, _, live = _plain_teacher(s)
    d = p * (live * s["dkl"][:, None])
    d.scatter_add_(1, s["teacher_index"].clamp(min=0).long(), -q * s["dkl"][:, None])
    return {"dlogits": _plain_spread(s, _plain_hard(s, d, p) if s["case"]["hard"] else d)}


def _library():
    from bf16_numerics_amd import binding
    return binding


def _workspace(s, make):
    """The scratch memory a training loop allocates once and keeps."""
    if "workspace" not in s:
        s["workspace"] = make()
    return s["workspace"]


def _own_ln_fwd(s):
    _library().layernorm_forward(s["x"], s["weight"], s["bias"], s["out"], s["mean"], s["rstd"], eps=EPS)
    return {"out": s["out"], "mean": s["mean"], "rstd": s["rstd"]}


def _own_ln_bwd(s):
    bfo = _library()
    ws = _workspace(s, lambda: bfo.new_layernorm_workspace(s["case"]["rows"], s["case"]["cols"], s["x"].device))
    bfo.layernorm_backward(s["dout"], s["x"], s["weight"], s["mean"], s["rstd"], s["dx"], s["dweight"], s["dbias"],
                           workspace=ws)
    return {"dx": s["dx"], "dweight": s["dweight"], "dbias": s["dbias"]}


def _own_lp_fwd(s):
    bfo, c = _library(), s["case"]
    ws = _workspace(s, lambda: bfo.new_logits_workspace(c["rows"], c["vocab"], c["top"], s["logits"].device))
    bfo.token_logprobs_forward(s["logits"], s["targets"], s["logprob"], s["stats"], entropy=s["entropy"],
                               top_index=s.get("top_index"), top_logprob=s.get("top_logprob"), vocab=c["vocab"],
                               scale=c["scale"], workspace=ws)
    return {k: s[k] for k in ("logprob", "stats", "entropy", "top_index", "top_logprob") if k in s}


def _own_lp_bwd(s):
    _library().token_logprobs_backward(s["logits"], s["targets"], s["stats"], s["dlogprob"], s["dlogits"],
                                       entropy=s["entropy"], dentropy=s["dentropy"], vocab=s["case"]["vocab"],
                                       scale=s["case"]["scale"])
    return {"dlogits": s["dlogits"]}


def _own_kd_fwd(s):
    bfo, c = _library(), s["case"]
    ws = _workspace(s, lambda: bfo.new_logits_workspace(c["rows"], c["vocab"], 0, s["logits"].device))
    bfo.distill_forward(s["logits"], s["teacher_index"], s["teacher_logits"], s["kl"], s["stats"],
                        targets=s["targets"] if c["hard"] else None, logprob=s.get("logprob"), vocab=c["vocab"],
                        scale=c["scale"], workspace=ws)
    return {k: s[k] for k in ("kl", "stats", "logprob") if k in s}


def _own_kd_bwd(s):
    hard = s["case"]["hard"]
    _library().distill_backward(s["logits"], s["teacher_index"], s["teacher_logits"], s["stats"], s["dkl"],
                                s["dlogits"], targets=s["targets"] if hard else None, dlogprob=s.get("dlogprob"),
                                vocab=s["case"]["vocab"], scale=s["case"]["scale"])
    return {"dlogits": s["dlogits"]}


_PLAIN = {"ln_fwd": _plain_ln_fwd, "ln_bwd": _plain_ln_bwd, "lp_fwd": _plain_lp_fwd, "lp_bwd": _plain_lp_bwd,
          "kd_fwd": _plain_kd_fwd, "kd_bwd": _plain_kd_bwd}
_OWN = {"ln_fwd": _own_ln_fwd, "ln_bwd": _own_ln_bwd, "lp_fwd": _own_lp_fwd, "lp_bwd": _own_lp_bwd,
        "kd_fwd": _own_kd_fwd, "kd_bwd": _own_kd_bwd}


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    R, b = case["rows"], 2 if case["dtype"] == "bf16" else 4
    if case["op"].startswith("ln"):
        C, pb = case["cols"], 2 if case["pdtype"] == "bf16" else 4
        if case["op"] == "ln_fwd":
            return {"bytes": 2 * b * R * C + 2 * pb * C + 8 * R, "flops": 8 * R * C}
        return {"bytes": 3 * b * R * C + 3 * pb * C + 8 * R, "flops": 16 * R * C}
    V, W = case["vocab"], case["width"]
    if case["op"] == "lp_fwd":
        return {"bytes": b * R * V + R * (4 + 16 + 8 * case["top"]), "flops": 6 * R * V}
    if case["op"] == "kd_fwd":
        return {"bytes": b * R * V + R * (12 + 8 * case["count"] + (8 if case["hard"] else 0)), "flops": 4 * R * V}
    if case["op"] == "lp_bwd":
        return {"bytes": b * R * (V + W) + R * 24, "flops": 8 * R * V}
    return {"bytes": b * R * (V + W) + R * (12 + 8 * case["count"] + (8 if case["hard"] else 0)), "flops": 6 * R * V}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("ln"):
        return _exact_ln(case, s)
    parts = [_exact_logits(case, s, slice(r, min(r + 512, case["rows"]))) for r in range(0, case["rows"], 512)]
    return {k: torch.cat([p.pop(k) for p in parts]) for k in list(parts[0])}


def _exact_ln(case, s):
    x, w, C = s["x"].double(), s["weight"].double(), case["cols"]
    if case["op"] == "ln_fwd":
        var, mean = torch.var_mean(x, dim=1, correction=0)
        rstd = (var + EPS).pow(-0.5)
        return {"out": torch.addcmul(s["bias"].double(), (x - mean[:, None]) * rstd[:, None], w), "mean": mean,
                "rstd": rstd}
    # The derivative with mean and rstd as the forward pass stored them: dx is
    # rstd times what is left of w * dout after its projections on 1 and xhat.
    dout, rstd = s["dout"].double(), s["rstd"].double()[:, None]
    xhat = rstd * (x - s["mean"].double()[:, None])
    h = w * dout
    dx = rstd * (h - h.mean(1, keepdim=True) - xhat * (xhat * h).mean(1, keepdim=True))
    return {"dx": dx, "dweight": (xhat * dout).sum(0), "dbias": dout.sum(0)}


def _exact_logits(case, s, rows):
    V, W, scale, op = case["vocab"], case["width"], case["scale"], case["op"]
    raw = s["logits"][rows, :V].double()
    z = raw * scale
    lse = torch.logsumexp(z, 1, keepdim=True)
    logp = z - lse
    t = s["targets"][rows].long()
    at = (t >= 0).nonzero()[:, 0]
    if op in ("lp_fwd", "kd_fwd"):
        m = z.max(1, keepdim=True).values
        out = {"stats": torch.cat([m, lse - m], 1)}
        logprob = torch.zeros(len(t), dtype=torch.float64, device=DEV)
        logprob[at] = logp[at, t[at]]
    if op == "lp_fwd":
        out["logprob"] = logprob
        out["entropy"] = -(logp.exp() * logp).sum(1)
        if case["top"]:
            index = torch.sort(raw, dim=1, descending=True, stable=True).indices[:, :case["top"]]
            out["top_index"] = index.to(torch.int32)
            out["top_logprob"] = logp.gather(1, index)
        return out
    if op == "lp_bwd":
        # The gradient by the row's stored sum and entropy, which are inputs here.
        logp = z - s["stats"][rows].double().sum(1, keepdim=True)
        p = logp.exp()
        d = -(s["dentropy"][rows].double()[:, None]) * p * (logp + s["entropy"][rows].double()[:, None])
        g = s["dlogprob"][rows].double()
        d[at] -= g[at, None] * p[at]
        d[at, t[at]] += g[at]
    else:
        index, value = s["teacher_index"][rows].long(), s["teacher_logits"][rows].double() * scale
        value = value.masked_fill(index < 0, -math.inf)
        full = (index >= 0).any(1)
        q = torch.zeros_like(value)
        q[full] = torch.softmax(value[full], 1)
        if op == "kd_fwd":
            logq = torch.zeros_like(value)
            logq[full] = torch.log_softmax(value[full], 1)
            term = q * (logq - logp.gather(1, index.clamp(min=0)))
            out["kl"] = term.masked_fill(q == 0, 0.0).sum(1)
            if case["hard"]:
                out["logprob"] = logprob
            return out
        p = (z - s["stats"][rows].double().sum(1, keepdim=True)).exp()
        g = s["dkl"][rows].double()[:, None]
        d = p * g * full[:, None]
        d.scatter_add_(1, index.clamp(min=0), -g * q)
        if case["hard"]:
            h = s["dlogprob"][rows].double()
            d[at] -= h[at, None] * p[at]
            d[at, t[at]] += h[at]
    wide = torch.zeros(len(t), W, dtype=torch.float64, device=DEV)
    wide[:, :V] = scale * d
    return {"dlogits": wide}
