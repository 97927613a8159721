"""A training loop made of the operators around the step: lookup, attention logits, clipped step, QK-Clip.

A two-layer model small enough to follow in fp64 on the side: embedding lookup
-> query and key projections -> attention scores (torch) -> loss. Its backward
pass fills the table's gradient through the sorted-token kernel, straight into
the buffer the optimizer reads; the step clips by the global norm; QK-Clip then
rescales the projections by the largest logits of the forward pass. Every
gradient is checked against fp64 autograd of the same formulas, the norm and
the clipped logits against their definitions, and the whole loop, captured in
a CUDA graph where that is possible, against its eager run.
"""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import adamw_hybrid_optimizer_muon_b200 as ma

pytestmark = pytest.mark.gpu

V, D, H, DH, B, T = 500, 64, 4, 32, 3, 40
U = 2.0 ** -24


class Loop:
    def __init__(self, max_norm, tau):
        g = torch.Generator(device="cuda")
        g.manual_seed(1)
        new = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
        self.table = torch.nn.Parameter(new(V, D))
        self.wq = torch.nn.Parameter(new(H * DH, D) * 0.5)
        self.wk = torch.nn.Parameter(new(H * DH, D) * 0.5)
        self.gain = torch.nn.Parameter(torch.ones(D, device="cuda"))
        self.params = [self.table, self.wq, self.wk, self.gain]
        self.grads = [torch.zeros_like(p) for p in self.params]
        self.opt = ma.MuonAdamW([(self.table, ma.ROLE_EMBED, 1), (self.wq, ma.ROLE_HIDDEN, 0),
                                 (self.wk, ma.ROLE_HIDDEN, 0), (self.gain, ma.ROLE_HIDDEN, 1)],
                                [("muon", ma.muon_hparams(heads=H)), ("adamw", ma.adamw_hparams(lr=0.01))])
        self.max_norm, self.tau = max_norm, tau

    def forward(self, ids):
        x = ma.embedding(ids, self.table, scale=2.0, grad=self.grads[0]) * self.gain
        q, k = (x @ w.T for w in (self.wq, self.wk))
        q, k = q.view(B, T, H, DH), k.view(B, T, H, DH)
        return x, q, k

    @staticmethod
    def loss(q, k):
        s = torch.einsum("bihd,bjhd->bhij", q, k) * DH ** -0.5
        mask = torch.ones((T, T), dtype=torch.bool, device=q.device).tril()
        return torch.logsumexp(s.masked_fill(~mask, -math.inf), dim=-1).mean()

    def step(self, ids, graph=False):
        for g in self.grads:
            g.zero_()
        for p, g in zip(self.params[1:], self.grads[1:]):
            p.grad = g
        x, q, k = self.forward(ids)
        self.loss(q, k).backward()
        self.top = ma.qk_max_logit(q.detach().bfloat16(), k.detach().bfloat16())
        self.opt.step(self.grads, graph=graph, max_norm=self.max_norm)
        ma.qk_clip(self.wq.data, self.wk.data, self.top, tau=self.tau)
        return q, k


def batch(seed):
    return torch.from_numpy(np.random.default_rng(seed).integers(0, V, (B, T))).cuda()


def test_gradients_norm_and_clip_of_one_step():
    a = Loop(max_norm=1e-3, tau=1.0)
    ids = batch(0)
    before = [p.detach().clone() for p in a.params]
    # fp64 on the side
    t64, q64, k64, g64 = (p.detach().double().requires_grad_() for p in a.params)
    x = t64[ids] * 2 * g64
    q = (x @ q64.T).view(B, T, H, DH)
    k = (x @ k64.T).view(B, T, H, DH)
    a.loss(q, k).backward()
    ref = [p.grad for p in (t64, q64, k64, g64)]
    a.step(ids)
    assert a.table.grad is None  # its gradient went straight into the optimizer's buffer
    for got, want in zip(a.grads, ref):
        # fp32 forward and backward (torch's products in fp32): 1e-4 of the gradient's size is a generous bound
        assert float((got.double() - want).norm()) <= 1e-4 * float(want.norm())
    norm = math.sqrt(sum(float(g.double().square().sum()) for g in a.grads))
    assert float(a.opt.grad_norm) == pytest.approx(norm, rel=33 * U)
    # the step saw the gradients times max_norm / norm: the first exp_avg is (1 - beta1) of that
    m = a.opt.state[0][0].double()
    want = a.grads[0].double() * (1e-3 / norm) * (1 - float(np.float32(0.9)))
    assert ((m - want).abs() <= want.abs() * 40 * U + 1e-30).all()
    assert not torch.equal(before[1], a.wq)
    # the largest logits, of q and k rounded to bf16: within their rounding of the fp64 ones
    s = torch.einsum("bihd,bjhd->bhij", q, k) * DH ** -0.5
    mags = torch.einsum("bihd,bjhd->bhij", q.abs(), k.abs()) * DH ** -0.5
    mask = torch.ones((T, T), dtype=torch.bool, device="cuda").tril()
    top = s.masked_fill(~mask, -math.inf).amax(dim=(0, 2, 3))
    bound = 3 * 2.0 ** -8 * mags.amax(dim=(0, 2, 3)) + 1e-4 * top.abs()
    assert ((a.top.double() - top).abs() <= bound).all()


def test_clipped_logits_stay_at_tau_over_steps():
    a = Loop(max_norm=1.0, tau=2.0)
    tops = []
    for i in range(6):
        a.step(batch(i % 2))
        tops.append(float(a.top.max()))
    assert ma.ma_device_status() == ma.MA_OK
    assert tops[0] > 4.0 and all(math.isfinite(t) for t in tops)
    assert max(tops[2:]) < tops[0]  # what a head exceeds tau by is taken out of its weights after each step


@pytest.mark.parametrize("accumulated", [1, 3])
def test_graph_steps_and_micro_batches_agree_with_eager(accumulated):
    runs = [Loop(max_norm=0.5, tau=2.0) for _ in range(2)]
    for i in range(4):
        for r, graph in zip(runs, (False, True)):
            for g in r.grads:
                g.zero_()
            for p, g in zip(r.params[1:], r.grads[1:]):
                p.grad = g
            top = None
            for m in range(accumulated):
                x, q, k = r.forward(batch(10 * i + m))
                r.loss(q, k).backward()
                top = ma.qk_max_logit(q.detach().bfloat16(), k.detach().bfloat16(), out=top, accumulate=top is not None)
            r.opt.step(r.grads, graph=graph, max_norm=0.5, grad_scale=1.0 / accumulated)
            ma.qk_clip(r.wq.data, r.wk.data, top, tau=2.0)
        # torch's products may choose another kernel from call to call; the operators repeat bit for bit
        for p, q in zip(runs[0].params, runs[1].params):
            assert float((p - q).detach().double().norm()) <= 1e-5 * float(p.detach().double().norm())
    assert runs[1].opt.graph_captures == 1
    assert ma.ma_device_status() == ma.MA_OK


def test_captured_loop_replays():
    # forward, backward, clipped step and QK-Clip in one graph, beside an eager optimizer of the same table
    a, b = Loop(max_norm=0.5, tau=2.0), Loop(max_norm=0.5, tau=2.0)
    ids = batch(0).clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(2):
            a.step(ids)
            b.step(ids)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    hp_step = a.opt.step_count
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):  # captures the next step, with the step count it has then
        a.step(ids)
    assert a.opt.step_count == hp_step + 1
    ids.copy_(batch(7))
    graph.replay()
    with torch.cuda.stream(s):
        s.wait_stream(torch.cuda.current_stream())
        b.step(batch(7))
    torch.cuda.synchronize()
    for p, q in zip(a.params, b.params):
        assert float((p - q).detach().double().norm()) <= 1e-5 * float(q.detach().double().norm())
    assert ma.ma_device_status() == ma.MA_OK
