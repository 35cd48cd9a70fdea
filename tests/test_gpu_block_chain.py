"""The operators between a block's matrix products as a training step runs them:
a small block of the 7B model's kind (norm, queries and keys turned, norm, gated
feed-forward) forward, keeping 8-bit checkpoints only, and backward from those into
the flat grads buffer, the grad norm and the update -- eagerly, every operator held
to its definition on the arrays it had, and recorded into a HIP graph."""
import numpy as np
import pytest
import torch

import oracle as o
from bf16_numerics_amd import workloads as W
from block_reference import DEV, check_activation_backward, check_activation_forward, check_rms_backward, \
    check_rms_forward, check_rotary, values
from gpu_harness import assert_norm_parity, assert_state_parity, host_copy, oracle_step, step_seed

pytestmark = pytest.mark.gpu
T, D, F, HEADS = 96, 160, 416, 5
DIM = D // HEADS


@pytest.fixture(scope="module")
def bfo():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from bf16_numerics_amd import binding
    torch.cuda.set_device(0)
    return binding


class Block:
    """Everything is allocated once, so that the step can be recorded.  The attention's place is taken by a
    product of the turned queries and keys, element by element, with the values."""

    def __init__(self, bfo, codes):
        self.bfo = bfo
        self.w = w = W.Workload("block", W.llama_tensors(64, D, F, 1), param_std=0.05)
        place = {n: (off, numel, shape) for (n, shape), (off, numel, _) in zip(w.tensors, w.entries())}
        self.table = bfo.Table(w.entries())
        self.P, self.M, self.m, self.v = W.init_state(torch, w, 0, w.n, DEV)
        self.G = torch.zeros(w.n, dtype=torch.bfloat16, device=DEV)

        def views(buf):
            return {n.split(".")[-1]: buf[off:off + numel].view(shape) for n, (off, numel, shape) in place.items()}
        self.p, self.g = views(self.P), views(self.G)
        for n in ("attn_norm", "ffn_norm"):
            self.p[n].add_(1.0)
        self.M.copy_(self.P.float())
        self.frequencies = bfo.rotary_frequencies(DIM, device=DEV)

        def mat(cols):
            return torch.zeros(T, cols, dtype=torch.bfloat16, device=DEV)
        self.x, self.dy = mat(D), mat(D)
        for n in ("h1", "a", "total", "h2", "d", "dx", "dh1", "dh2", "h1_again", "h2_again"):
            setattr(self, n, mat(D))
        self.qkv, self.turned, self.dqkv, self.dturned = (torch.zeros(T, 3 * HEADS, DIM, dtype=torch.bfloat16, device=DEV)
                                                          for _ in range(4))
        self.fused, self.dfused = mat(2 * F), mat(2 * F)
        self.f, self.df, self.f_again = mat(F), mat(F), mat(F)
        self.rstd1, self.rstd2 = torch.zeros(T, device=DEV), torch.zeros(T, device=DEV)
        new = lambda cols: bfo.new_codes(T, cols, DEV, codes)  # noqa: E731
        self.kept1, self.kept2, self.kept_gate, self.kept_up = new(D), new(D), new(F), new(F)
        self.res = bfo.new_norm_result(DEV)
        self.ws, self.rws = bfo.new_norm_workspace(self.table), bfo.new_rmsnorm_workspace(T, D, DEV)

    def new_batch(self, seed):
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.x.copy_(torch.empty(T, D, device=DEV).normal_(generator=g))
        self.dy.copy_(torch.empty(T, D, device=DEV).normal_(generator=g) * 0.01)

    @staticmethod
    def product(out, a, b):
        """The library's matrix products, in binary32."""
        out.copy_((a.float() @ b.float()).view(out.shape))

    def forward(self):
        b, p, H = self.bfo, self.p, HEADS
        b.rmsnorm_forward(self.x, p["attn_norm"], self.h1, rstd=self.rstd1, codes=self.kept1[0], scales=self.kept1[1])
        for k, n in enumerate(("wq", "wk", "wv")):
            self.product(self.qkv[:, k * H:(k + 1) * H], self.h1, p[n].t())
        b.rotary_apply(self.qkv[:, :2 * H], self.frequencies, self.turned[:, :2 * H], period=32)
        self.turned[:, 2 * H:].copy_(self.qkv[:, 2 * H:])
        mixed = self.turned[:, :H].float() * self.turned[:, H:2 * H].float() * self.turned[:, 2 * H:].float()
        self.product(self.a, mixed.reshape(T, D), p["wo"].t())
        b.rmsnorm_forward(self.a, p["ffn_norm"], self.h2, residual=self.x, total=self.total, rstd=self.rstd2,
                          codes=self.kept2[0], scales=self.kept2[1])
        self.product(self.fused[:, :F], self.h2, p["w1"].t())
        self.product(self.fused[:, F:], self.h2, p["w3"].t())
        b.activation_forward(self.fused[:, :F], self.fused[:, F:], self.f, gate_codes=self.kept_gate[0],
                             gate_scales=self.kept_gate[1], up_codes=self.kept_up[0], up_scales=self.kept_up[1])
        self.product(self.d, self.f, p["w2"].t())

    def backward(self):
        b, p, g, H = self.bfo, self.p, self.g, HEADS
        self.product(self.df, self.dy, p["w2"])
        b.activation_backward(self.df, None, None, self.dfused[:, :F], self.dfused[:, F:], gate_codes=self.kept_gate[0],
                              gate_scales=self.kept_gate[1], up_codes=self.kept_up[0], up_scales=self.kept_up[1],
                              out=self.f_again)
        self.product(g["w2"], self.dy.t(), self.f_again)
        self.product(self.dh2, torch.cat([self.dfused[:, :F], self.dfused[:, F:]], 1), torch.cat([p["w1"], p["w3"]]))
        self.dx.copy_(self.dy)                                  # the residual stream's gradient
        b.rmsnorm_backward(self.dh2, None, p["ffn_norm"], self.rstd2, self.dx, g["ffn_norm"], codes=self.kept2[0],
                           scales=self.kept2[1], out=self.h2_again, workspace=self.rws, accumulate_dx=True)
        self.product(g["w1"], self.dfused[:, :F].t(), self.h2_again)
        self.product(g["w3"], self.dfused[:, F:].t(), self.h2_again)
        dmixed = (self.dx.float() @ p["wo"].float()).view(T, H, DIM)
        q, k, v = (self.turned[:, i * H:(i + 1) * H].float() for i in range(3))
        self.product(g["wo"], self.dx.t(), (q * k * v).reshape(T, D))
        for i, d in enumerate((dmixed * k * v, dmixed * q * v, dmixed * q * k)):
            self.dturned[:, i * H:(i + 1) * H].copy_(d)
        b.rotary_apply(self.dturned[:, :2 * H], self.frequencies, self.dqkv[:, :2 * H], period=32, backward=True)
        self.dqkv[:, 2 * H:].copy_(self.dturned[:, 2 * H:])
        flat = self.dqkv.view(T, 3, D)
        self.dh1.copy_(sum(flat[:, i].float() @ p[n].float() for i, n in enumerate(("wq", "wk", "wv"))))
        b.rmsnorm_backward(self.dh1, None, p["attn_norm"], self.rstd1, self.dx, g["attn_norm"], codes=self.kept1[0],
                           scales=self.kept1[1], out=self.h1_again, workspace=self.rws, accumulate_dx=True)
        for i, n in enumerate(("wq", "wk", "wv")):
            self.product(g[n], flat[:, i].t(), self.h1_again)
        b.grad_global_norm(self.table, self.G, self.res, self.w.hparams.max_norm, workspace=self.ws)

    def update(self, t):
        self.bfo.adamw_sr_step(self.table, self.P, self.G, self.M, self.m, self.v, self.w.hparams, t, step_seed(t),
                               scale=self.res)


@pytest.mark.parametrize("codes", [torch.int8, torch.float8_e4m3fn])
def test_steps_match_the_definitions_and_the_oracle(bfo, codes):
    s = Block(bfo, codes)
    tbl = o.table(s.w.entries())
    index = torch.arange(T, device=DEV) % 32
    for t in range(1, 4):
        s.new_batch(t)
        s.forward()
        p, g = s.p, s.g
        check_rms_forward(s.x, None, p["attn_norm"], 1e-5, None, s.h1, s.rstd1, *s.kept1)
        check_rotary(s.turned[:, :2 * HEADS], s.qkv[:, :2 * HEADS], index, s.frequencies, True)
        check_rms_forward(s.a, s.x, p["ffn_norm"], 1e-5, s.total, s.h2, s.rstd2, *s.kept2)
        check_activation_forward(0, s.fused[:, :F], s.fused[:, F:], s.f)
        s.backward()
        gate, up = values(*s.kept_gate), values(*s.kept_up)
        check_activation_backward(0, s.df, gate, up, s.dfused[:, :F], s.dfused[:, F:], s.f_again, 1)
        check_rotary(s.dqkv[:, :2 * HEADS], s.dturned[:, :2 * HEADS], index, s.frequencies, True, backward=True)
        # dx holds both norms' gradients by now: the second norm's again, from the residual stream's
        dx, dw = s.dy.clone(), torch.empty_like(g["ffn_norm"])
        args = dict(codes=s.kept2[0], scales=s.kept2[1], workspace=s.rws, accumulate_dx=True)
        bfo.rmsnorm_backward(s.dh2, None, p["ffn_norm"], s.rstd2, dx, dw, **args)
        zero = torch.zeros_like(dw)
        check_rms_backward(s.dh2, values(*s.kept2), p["ffn_norm"], s.rstd2, dx, g["ffn_norm"], s.h2_again, (s.dy, zero))
        check_rms_backward(s.dh1, values(*s.kept1), p["attn_norm"], s.rstd1, s.dx, g["attn_norm"], s.h1_again, (dx, zero))
        st = {"P": s.P, "M": s.M, "m": s.m, "v": s.v, "G": s.G}
        host = host_copy(st)
        assert_norm_parity(bfo.read_norm_result(s.res), o.grad_norm(host["G"], s.w.hparams.max_norm))
        scale = bfo.read_norm_result(s.res)[2]
        s.update(t)
        oracle_step(tbl, 0, host, s.w.hparams, scale, t, step_seed(t))
        assert_state_parity(host_copy(st), host, f"step {t}")
        assert np.abs(host["m"]).max() > 0


def test_recorded_step_replays_like_the_eager_one(bfo):
    eager, rec = Block(bfo, torch.int8), Block(bfo, torch.int8)
    side = torch.cuda.Stream()
    rec.new_batch(0)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):                 # libraries set themselves up outside the recording
        rec.forward()
        rec.backward()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        rec.forward()
        rec.backward()
    for t in range(1, 6):
        for s in (eager, rec):
            s.new_batch(t)
        eager.forward()
        eager.backward()
        eager.update(t)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for k in ("h1", "turned", "total", "h2", "f", "d", "dfused", "f_again", "h2_again", "dqkv", "h1_again", "dx", "G"):
            assert torch.equal(getattr(eager, k), getattr(rec, k)), (t, k)
        rec.update(t)
        for k in ("P", "M", "m", "v"):
            assert torch.equal(getattr(eager, k), getattr(rec, k)), (t, k)


def test_gradients_of_the_block_against_autograd(bfo):
    """The block in 64 bits from the same weights: with what is kept in 8-bit integers, the grads that the optimizer
    reads are off by the roundings to bf16 of a chain of ten arrays and by half a code's step of four: their norm's
    error is below the sum of 14 relative roundings of 2^-8 (bf16) and 4 of 2^-7 (of a group's largest value, and the
    typical value is a third of it)."""
    s = Block(bfo, torch.int8)
    s.new_batch(7)
    s.forward()
    s.backward()
    p = {n: s.p[n].double().requires_grad_() for n in ("attn_norm", "wq", "wk", "wv", "wo", "ffn_norm", "w1", "w2", "w3")}
    x = s.x.double().requires_grad_()

    def norm(v, w):
        return v / torch.sqrt(v.square().mean(1, keepdim=True) + 1e-5) * w
    angle = (torch.arange(T, device=DEV) % 32).double()[:, None] * s.frequencies
    c, sn = torch.cos(angle)[:, None], torch.sin(angle)[:, None]

    def turn(v):
        a, b = v[..., :DIM // 2], v[..., DIM // 2:]
        return torch.cat([a * c - b * sn, a * sn + b * c], 2)
    h = norm(x, p["attn_norm"])
    q, k, v = ((h @ p[n].t()).view(T, HEADS, DIM) for n in ("wq", "wk", "wv"))
    y = x + (turn(q) * turn(k) * v).reshape(T, D) @ p["wo"].t()
    h = norm(y, p["ffn_norm"])
    y = y + (torch.nn.functional.silu(h @ p["w1"].t()) * (h @ p["w3"].t())) @ p["w2"].t()
    (y * s.dy.double()).sum().backward()
    bound = 14 * 2.0 ** -8 + 4 * 2.0 ** -7
    for n, t in list(p.items()) + [("x", x)]:
        got = s.dx if n == "x" else s.g[n]
        off = (got.double() - t.grad).norm() / t.grad.norm()
        assert off < bound, (n, float(off))


def test_two_graphs_with_their_own_workspaces_at_once(bfo):
    """The norm's backward recorded twice, replayed on two streams at once."""
    g = torch.Generator(device=DEV).manual_seed(1)
    R, C = 3000, 768
    sets = []
    for _ in range(2):
        x = torch.empty(R, C, device=DEV).normal_(generator=g).bfloat16()
        d = torch.empty(R, C, device=DEV).normal_(generator=g).bfloat16()
        w = torch.ones(C, dtype=torch.bfloat16, device=DEV)
        rstd = (x.float().square().mean(1) + 1e-5).rsqrt()
        sets.append(dict(dout=d, x=x, weight=w, rstd=rstd, dx=torch.zeros_like(x), dweight=torch.zeros_like(w),
                         out=torch.zeros_like(x), workspace=bfo.new_rmsnorm_workspace(R, C, DEV)))
    want = []
    for s in sets:
        bfo.rmsnorm_backward(**s)
        torch.cuda.synchronize()
        want.append([s[k].clone() for k in ("dx", "dweight", "out")])
    streams, graphs = [torch.cuda.Stream() for _ in sets], []
    for s, st in zip(sets, streams):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            bfo.rmsnorm_backward(**s)
        graphs.append(graph)
    for _ in range(10):
        for s in sets:
            for k in ("dx", "dweight", "out"):
                s[k].zero_()
        torch.cuda.synchronize()
        for graph, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                graph.replay()
        torch.cuda.synchronize()
        for s, ref in zip(sets, want):
            for k, r in zip(("dx", "dweight", "out"), ref):
                assert torch.equal(s[k], r), k
