"""The operators as a training step runs them: final layer norm, logits, loss
and its gradient, layer norm's gradient into the flat grads buffer, the grad
norm and the update -- on the d=32 model's table -- and the same recorded into
a HIP graph."""
import numpy as np
import pytest
import torch

import oracle as o
from bf16_numerics_amd import workloads as W
from gpu_harness import assert_norm_parity, assert_state_parity, host_copy, oracle_step, step_seed
from test_gpu_layernorm import check_backward, check_forward as check_ln_forward
from test_gpu_logits import check_forward as check_lp_forward, check_gradient, gradient_reference, teacher, \
    teacher_reference

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
ROWS, COLS, VOCAB = 96, 32, 61      # 61 of the 64 rows of the embedding are tokens


@pytest.fixture(scope="module")
def bfo():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from bf16_numerics_amd import binding
    torch.cuda.set_device(0)
    return binding


class Step:
    """The end of a training step on the d=32 model: everything is allocated
    once, so that the step can be recorded."""

    def __init__(self, bfo, distill):
        self.bfo, self.distill, self.w = bfo, distill, W.tiny()
        w, e = self.w, dict(zip([n for n, _ in W.tiny().tensors], W.tiny().entries()))
        self.table = bfo.Table(w.entries())
        self.P, self.M, self.m, self.v = W.init_state(torch, w, 0, w.n, DEV)
        self.G = torch.zeros(w.n, dtype=torch.bfloat16, device=DEV)
        def piece(buf, name):
            off, numel, _ = e[name]
            return buf[off:off + numel]
        self.wte, self.lnw, self.lnb = piece(self.P, "wte").view(64, 32), piece(self.P, "lnfw"), piece(self.P, "lnfb")
        self.lnw.add_(1.0)
        self.M.copy_(self.P.float())
        self.gwte, self.glnw, self.glnb = piece(self.G, "wte").view(64, 32), piece(self.G, "lnfw"), \
            piece(self.G, "lnfb")
        bf = dict(dtype=torch.bfloat16, device=DEV)
        self.x, self.y, self.dx, self.dy = (torch.zeros(ROWS, COLS, **bf) for _ in range(4))
        self.mean, self.rstd, self.logprob, self.entropy, self.kl = (torch.zeros(ROWS, device=DEV) for _ in range(5))
        self.stats = torch.zeros(ROWS, 2, device=DEV)
        self.logits, self.dlogits = torch.zeros(ROWS, 64, **bf), torch.zeros(ROWS, 64, **bf)
        self.targets = torch.zeros(ROWS, dtype=torch.int32, device=DEV)
        self.index, self.value = torch.zeros(ROWS, 8, dtype=torch.int32, device=DEV), torch.zeros(ROWS, 8, device=DEV)
        self.dlogprob = torch.full((ROWS,), -1.0 / ROWS, device=DEV)
        self.dentropy = torch.full((ROWS,), -0.01 / ROWS, device=DEV)
        self.dkl = torch.full((ROWS,), 0.5 / ROWS, device=DEV)
        self.res = bfo.new_norm_result(DEV)
        self.ws = bfo.new_norm_workspace(self.table)
        self.lnws = bfo.new_layernorm_workspace(ROWS, COLS, DEV)
        self.lpws = bfo.new_logits_workspace(ROWS, VOCAB, 0, DEV)

    def new_batch(self, seed):
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.x.copy_(torch.empty(ROWS, COLS, device=DEV).normal_(generator=g))
        self.targets.copy_(torch.randint(-1, VOCAB, (ROWS,), generator=g, device=DEV).to(torch.int32))
        i, v = teacher(ROWS, VOCAB, 8, seed)
        self.index.copy_(i)
        self.value.copy_(v)

    def gradients(self):
        b = self.bfo
        b.layernorm_forward(self.x, self.lnw, self.lnb, self.y, self.mean, self.rstd)
        self.logits.copy_(20 * (self.y.float() @ self.wte.float().t()))
        if self.distill:
            b.distill_forward(self.logits, self.index, self.value, self.kl, self.stats, targets=self.targets,
                              logprob=self.logprob, vocab=VOCAB, workspace=self.lpws)
            b.distill_backward(self.logits, self.index, self.value, self.stats, self.dkl, self.dlogits,
                               targets=self.targets, dlogprob=self.dlogprob, vocab=VOCAB)
        else:
            b.token_logprobs_forward(self.logits, self.targets, self.logprob, self.stats, entropy=self.entropy,
                                     vocab=VOCAB, workspace=self.lpws)
            b.token_logprobs_backward(self.logits, self.targets, self.stats, self.dlogprob, self.dlogits,
                                      entropy=self.entropy, dentropy=self.dentropy, vocab=VOCAB)
        self.dy.copy_(20 * (self.dlogits.float() @ self.wte.float()))
        self.gwte.copy_(20 * (self.dlogits.float().t() @ self.y.float()))
        b.layernorm_backward(self.dy, self.x, self.lnw, self.mean, self.rstd, self.dx, self.glnw, self.glnb,
                             workspace=self.lnws)
        b.grad_global_norm(self.table, self.G, self.res, self.w.hparams.max_norm, workspace=self.ws)

    def update(self, t):
        self.bfo.adamw_sr_step(self.table, self.P, self.G, self.M, self.m, self.v, self.w.hparams, t, step_seed(t),
                               scale=self.res)


@pytest.mark.parametrize("distill", [False, True])
def test_steps_match_the_definitions_and_the_oracle(bfo, distill):
    s = Step(bfo, distill)
    tbl = o.table(s.w.entries())
    for t in range(1, 4):
        s.new_batch(t)
        s.gradients()
        check_ln_forward(s.x, s.lnw, s.lnb, 1e-5, s.y, s.mean, s.rstd)
        zero = torch.zeros(ROWS, device=DEV)
        hard = torch.where(s.targets >= 0, s.dlogprob, 0.0)
        sparse = torch.zeros(ROWS, VOCAB, dtype=torch.float64, device=DEV)
        sparse.scatter_(1, s.targets.clamp(min=0).long()[:, None], hard.double()[:, None])
        if distill:
            q, _, live, _ = teacher_reference(s.index, s.value, 1.0)
            sparse.scatter_add_(1, s.index.clamp(min=0).long(), -s.dkl.double()[:, None] * q)
            ref, tol = gradient_reference(s.logits, VOCAB, 1.0, s.stats, torch.where(live, s.dkl, 0.0) - hard, zero,
                                          zero, sparse)
            # the teacher's probabilities are off by up to 120 u, the two factors of p may cancel
            tol = tol + 120 * 2.0 ** -24 * (s.dkl + hard.abs()).double()[:, None]
        else:
            check_lp_forward({"logprob": s.logprob, "stats": s.stats, "entropy": s.entropy}, s.logits, s.targets,
                             VOCAB, 1.0, 0)
            ref, tol = gradient_reference(s.logits, VOCAB, 1.0, s.stats, -hard, -s.dentropy, s.entropy, sparse)
        check_gradient(s.dlogits, VOCAB, ref, tol)
        check_backward(s.x, s.dy, s.lnw, s.mean, s.rstd, s.dx, s.glnw, s.glnb)
        # the flat buffer the optimizer reads holds those gradients
        st = {"P": s.P, "M": s.M, "m": s.m, "v": s.v, "G": s.G}
        host = host_copy(st)
        assert_norm_parity(bfo.read_norm_result(s.res), o.grad_norm(host["G"], s.w.hparams.max_norm))
        scale = bfo.read_norm_result(s.res)[2]
        s.update(t)
        oracle_step(tbl, 0, host, s.w.hparams, scale, t, step_seed(t))
        assert_state_parity(host_copy(st), host, f"step {t}")
        assert not np.array_equal(host["M"], np.zeros_like(host["M"]))


@pytest.mark.parametrize("distill", [False, True])
def test_recorded_step_replays_like_the_eager_one(bfo, distill):
    eager, rec = Step(bfo, distill), Step(bfo, distill)
    side = torch.cuda.Stream()
    rec.new_batch(0)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        rec.gradients()                       # libraries set themselves up outside the recording
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        rec.gradients()
    for t in range(1, 6):
        for s in (eager, rec):
            s.new_batch(t)
        eager.gradients()
        eager.update(t)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for k in ("y", "mean", "rstd", "logprob", "stats", "entropy", "kl", "dlogits", "dx", "G"):
            assert torch.equal(getattr(eager, k), getattr(rec, k)), (t, k)
        rec.update(t)
        for k in ("P", "M", "m", "v"):
            assert torch.equal(getattr(eager, k), getattr(rec, k)), (t, k)


def test_two_graphs_with_their_own_workspaces_at_once(bfo):
    """Layer norm's backward recorded twice, replayed on two streams at once."""
    g = torch.Generator(device=DEV).manual_seed(1)
    R, C = 3000, 768
    sets = []
    for _ in range(2):
        x = torch.empty(R, C, device=DEV).normal_(generator=g).bfloat16()
        d = torch.empty(R, C, device=DEV).normal_(generator=g).bfloat16()
        w = torch.ones(C, dtype=torch.bfloat16, device=DEV)
        mean, rstd = x.float().mean(1), (x.float().var(1, unbiased=False) + 1e-5).rsqrt()
        sets.append(dict(dout=d, x=x, weight=w, mean=mean, rstd=rstd, dx=torch.zeros_like(x),
                         dweight=torch.zeros_like(w), dbias=torch.zeros_like(w),
                         workspace=bfo.new_layernorm_workspace(R, C, DEV)))
    want = []
    for s in sets:
        bfo.layernorm_backward(**s)
        torch.cuda.synchronize()
        want.append([s[k].clone() for k in ("dx", "dweight", "dbias")])
    streams, graphs = [torch.cuda.Stream() for _ in sets], []
    for s, st in zip(sets, streams):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            bfo.layernorm_backward(**s)
        graphs.append(graph)
    for _ in range(10):
        for s in sets:
            for k in ("dx", "dweight", "dbias"):
                s[k].zero_()
        torch.cuda.synchronize()
        for graph, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                graph.replay()
        torch.cuda.synchronize()
        for s, ref in zip(sets, want):
            for k, r in zip(("dx", "dweight", "dbias"), ref):
                assert torch.equal(s[k], r), k
