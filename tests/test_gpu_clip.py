"""Global gradient norm and clipping on the GPU, against the formulas in fp64.

Tolerances, from the arithmetic: a thread sums at most 64 squares in fp32 (64
roundings of 2^-24 of a sum of positive terms), everything after that is in
fp64, so the sum is within 64 * 2^-24 and its root within 32 * 2^-24; norm and
coef are then rounded to fp32 (2^-24 each). A clipped gradient adds the product's
rounding and, for bf16, half a step of the type.
"""
import datetime
import math
import socket

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import adamw_hybrid_optimizer_muon_b200 as ma

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TOL_NORM = 33 * U
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
LISTS = {
    "one value": [(1, "fp32", 0)],
    "empty list": [],
    "only empty": [(0, "fp32", 0), (0, "bf16", 0)],
    "small mixed": [(1, "bf16", 0), (7, "fp32", 1), (0, "bf16", 0), (513, "bf16", 3), (1280, "fp32", 0)],
    "offsets": [(5000 + k, "bf16", k) for k in range(9)] + [(3000 + k, "fp32", k) for k in range(5)],
    "chunk edges": [(16384, "bf16", 0), (16385, "bf16", 0), (16383, "bf16", 0), (8192, "fp32", 0), (8193, "fp32", 3),
                    (16384, "bf16", 7), (16377, "bf16", 7), (2 * 16384 + 1, "bf16", 1)],
    "97 tensors": [(100 + 7 * k, "bf16" if k % 2 else "fp32", k % 4) for k in range(97)],
    "640 tensors": [(1 + k % 70, "bf16" if k % 3 else "fp32", k % 4) for k in range(640)],
    "641 tensors": [(1 + k % 70, "bf16" if k % 3 else "fp32", k % 4) for k in range(641)],
    "256 small chunks": [(128 * 4 * 100, "fp32", 0), (128 * 8 * 156, "bf16", 0)],
    "257 small chunks": [(128 * 4 * 100 + 1, "fp32", 0), (128 * 8 * 156, "bf16", 0)],
    "1024 small chunks": [(512, "fp32", 0)] * 99 + [(128 * 8 * 925, "bf16", 0)],
    "1025 small chunks": [(512, "fp32", 0)] * 99 + [(128 * 8 * 925 + 1, "bf16", 0)],
    "1281 tensors": [(1 + k % 50, "bf16" if k % 3 else "fp32", k % 4) for k in range(1281)],
    "3000 tensors, some long": [(40000 if k % 500 == 0 else 1 + k % 9, "bf16", 0) for k in range(3000)],
    "long": [(9_000_001, "bf16", 1), (4_000_003, "fp32", 0)],
}


def make(spec, seed, std=1e-2):
    """Views into buffers with guard elements around them; returns (buffers, views)."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    bufs, views = [], []
    for n, dt, off in spec:
        b = torch.randn(n + off + 9, generator=g, device="cuda").mul_(std).to(DT[dt])
        bufs.append(b)
        views.append(b[off:off + n])
    return bufs, views


def norm64(views):
    return math.sqrt(sum(float(v.double().square().sum()) for v in views))


def check_clipped(before, after, coef):
    """after = before * coef, within the norm's error, the coefficient's and the product's rounding, and the type's."""
    for b, a in zip(before, after):
        want = b.double() * coef
        half = torch.finfo(a.dtype).eps / 2
        tiny = torch.finfo(a.dtype).tiny * torch.finfo(a.dtype).eps  # a subnormal's step
        assert ((a.double() - want).abs() <= want.abs() * (TOL_NORM + 2 * U + half) + tiny).all()


@pytest.mark.parametrize("name", list(LISTS))
def test_norm_and_clip_match_fp64(name):
    bufs, views = make(LISTS[name], 11)
    kept = [b.clone() for b in bufs]
    ref = norm64(views)
    clip = ma.GradClip(views)
    norm = float(clip.norm(max_norm=0.5 * ref, scale=3.0))
    assert abs(norm - 3 * ref) <= TOL_NORM * 3 * ref
    assert all(torch.equal(a, b) for a, b in zip(bufs, kept))  # measuring leaves the gradients alone
    coef = float(clip.buffer[1])
    want = 0.5 if ref > 0 else 3.0
    assert abs(coef - want) <= TOL_NORM * want
    assert float(clip.buffer.view(torch.float64)[1]) == pytest.approx(ref * ref, rel=64 * U, abs=0)
    # above the norm: only the scale
    clip.norm(max_norm=4 * ref + 1, scale=3.0)
    assert float(clip.buffer[1]) == 3.0
    # in place
    assert float(clip.clip(0.5 * ref, scale=3.0)) == norm  # the same bits either way
    check_clipped([b[off:off + n] for b, (n, _, off) in zip(kept, LISTS[name])], views, want)
    for b, k, (n, _, off) in zip(bufs, kept, LISTS[name]):  # nothing beside the gradients is touched
        assert torch.equal(b[:off], k[:off]) and torch.equal(b[off + n:], k[off + n:])
    if ref > 0:
        assert norm64(views) == pytest.approx(0.5 * ref, rel=2.0 ** -8 + 100 * U)
    assert ma.ma_device_status() == ma.MA_OK


def test_clipping_that_changes_nothing_writes_nothing():
    _, views = make(LISTS["small mixed"], 3)
    kept = [v.clone() for v in views]
    clip = ma.GradClip(views)
    clip.clip(math.inf)
    assert all(torch.equal(a, b) for a, b in zip(views, kept)) and float(clip.buffer[1]) == 1.0


@pytest.mark.parametrize("value", [1e30, 3e38, 1e-30, 1e-38, 1e-41, 0.0])
@pytest.mark.parametrize("dt", ["fp32", "bf16"])
def test_squares_beyond_fp32(value, dt):
    # the squares overflow or vanish in fp32; the norm does not
    v = torch.full((20001,), value, device="cuda").to(DT[dt])
    v[::2] *= -1
    clip = ma.GradClip([v])
    ref = norm64([v])
    norm = float(clip.norm(max_norm=1.0))
    root = math.sqrt(float(clip.buffer.view(torch.float64)[1]))
    assert root == pytest.approx(ref, rel=TOL_NORM, abs=0)
    if ref < 3e38:
        assert abs(norm - ref) <= TOL_NORM * ref + 2.0 ** -149
    else:
        assert math.isinf(norm)  # beyond fp32: the norm is, the coefficient is not
    if ref > 1:
        assert float(clip.buffer[1]) == pytest.approx(1 / ref, rel=TOL_NORM, abs=2.0 ** -149)


def test_one_large_value_among_small_ones():
    v = torch.full((100_000,), 1e-25, device="cuda")
    v[54321] = 2e25
    clip = ma.GradClip([v])
    assert float(clip.norm()) == pytest.approx(norm64([v]), rel=TOL_NORM)


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("dt", ["fp32", "bf16"])
def test_a_norm_that_is_not_finite_drops_the_gradients(bad, dt):
    _, views = make([(5000, dt, 1), (33, dt, 0)], 5)
    views[0][1234] = bad
    clip = ma.GradClip(views)
    norm = float(clip.norm(max_norm=1.0))
    assert not math.isfinite(norm) and float(clip.buffer[1]) == 0.0
    P, M, V = ([torch.randn(v.numel(), device="cuda") * 0.1 for v in views] for _ in range(3))
    V = [v.square() for v in V]
    P2, M2, V2 = ([x.clone() for x in xs] for xs in (P, M, V))
    hp = ma.adamw_hparams(lr=0.01, step=3)
    ma.adamw_step_fused(P, views, M, V, hp, clip=clip.buffer)
    ma.adamw_step_fused(P2, [torch.zeros_like(v) for v in views], M2, V2, hp)
    for a, b in zip(P + M + V, P2 + M2 + V2):
        assert torch.equal(a, b)
    clip.clip(1.0)
    assert all(not v.any() for v in views)


def test_max_norm_zero_zeroes():
    _, views = make(LISTS["small mixed"], 6)
    ma.GradClip(views).clip(0.0)
    assert all(not v.any() for v in views)


@pytest.mark.parametrize("dt", ["fp32", "bf16"])
@pytest.mark.parametrize("off", [0, 1])
def test_clipped_adamw_is_adamw_on_the_product(dt, off):
    # coef * g in fp32 is what the kernel forms: the same bits as fp32 gradients that hold the product
    bufs, views = make([(8192 * 2 + 5, dt, off), (3, dt, off), (0, dt, 0)], 7)
    clip = ma.GradClip(views)
    clip.norm(max_norm=0.37)
    G2 = [v.float() * clip.buffer[1] for v in views]
    P, M, V = ([torch.randn(v.numel(), device="cuda") * 0.1 for v in views] for _ in range(3))
    V = [v.square() for v in V]
    P2, M2, V2 = ([x.clone() for x in xs] for xs in (P, M, V))
    hp = ma.adamw_hparams(lr=0.01, step=2)
    ma.adamw_step_fused(P, views, M, V, hp, clip=clip.buffer)
    ma.adamw_step_fused(P2, G2, M2, V2, hp)
    for a, b in zip(P + M + V, P2 + M2 + V2):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dt", ["fp32", "bf16"])
@pytest.mark.parametrize("shape,heads,precision", [((256, 512), 1, 0), ((520, 200), 1, 0), ((256, 128), 4, 0),
                                                   ((200, 136), 1, 1), ((136, 200), 1, 1)])
def test_clipped_muon_is_muon_on_the_product(dt, shape, heads, precision):
    r = torch.Generator(device="cuda")
    r.manual_seed(8)
    new = lambda std: [torch.randn(shape, generator=r, device="cuda") * std for _ in range(3)]  # noqa: E731
    G = [g.to(DT[dt]) for g in new(1e-2)]
    W, M = new(0.02), new(1e-3)
    W2, M2 = [w.clone() for w in W], [m.clone() for m in M]
    clip = ma.GradClip(G)
    clip.norm(max_norm=0.11)
    hp = ma.muon_hparams(heads=heads, precision=precision)
    ws = torch.empty(ma.muon_workspace_bytes(3, *shape, hp), dtype=torch.uint8, device="cuda")
    ma.muon_step_batched(W, G, M, hp, ws, clip=clip.buffer)
    ma.muon_step_batched(W2, [g.float() * clip.buffer[1] for g in G], M2, hp, ws)
    assert ma.ma_device_status() == ma.MA_OK
    for a, b in zip(W + M, W2 + M2):
        assert torch.equal(a, b)


TABLE = [((1000, 64), ma.ROLE_EMBED, 1), ((256, 512), ma.ROLE_HIDDEN, 0), ((512, 256), ma.ROLE_HIDDEN, 0),
         ((256, 512), ma.ROLE_HIDDEN, 0), ((96,), ma.ROLE_HIDDEN, 1), ((), ma.ROLE_HIDDEN, 1)]


def _table(seed, dt):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return ([torch.randn(s, generator=g, device="cuda") * 0.02 for s, _, _ in TABLE],
            [(torch.randn(s, generator=g, device="cuda") * 1e-2).to(DT[dt]) for s, _, _ in TABLE])


def _opt(params):
    return ma.MuonAdamW([(p, role, g) for p, (_, role, g) in zip(params, TABLE)],
                        [("muon", ma.muon_hparams()), ("adamw", ma.adamw_hparams(lr=0.01))])


@pytest.mark.parametrize("dt", ["fp32", "bf16"])
@pytest.mark.parametrize("overlap", [False, True])
def test_whole_step_paths_agree(dt, overlap):
    # eager, graph and from-host steps with changing max_norm and scale against steps on gradients that
    # hold the product: the same bits; and one capture serves every max_norm
    ma.ma_set_momentum_overlap(overlap)
    try:
        runs = [_table(1, dt) for _ in range(4)]
        opts = [_opt(p) for p, _ in runs]
        prods = [torch.empty_like(g, dtype=torch.float32) for g in runs[0][1]]
        host = [g.cpu().pin_memory() for g in runs[0][1]]
        for k, kw in enumerate([dict(max_norm=0.5), dict(max_norm=0.05, grad_scale=2.0), dict(max_norm=1e9),
                                dict(grad_scale=0.5), dict(), dict(max_norm=0.7)]):
            _, fresh = _table(20 + k, dt)
            for _, G in runs:
                for a, b in zip(G, fresh):
                    a.copy_(b)
            for h, b in zip(host, fresh):
                h.copy_(b)
            opts[0].step(runs[0][1], **kw)
            opts[1].step(runs[1][1], graph=True, **kw)
            for g in runs[2][1]:
                g.zero_()
            opts[2].step_from_host(host, runs[2][1], **kw)
            if kw:
                ref = norm64(fresh) * kw.get("grad_scale", 1.0)
                assert float(opts[0].grad_norm) == pytest.approx(ref, rel=TOL_NORM)
                for p, g in zip(prods, fresh):
                    p.copy_(g.float() * opts[0]._clip[1])
                opts[3].step(prods)
            else:  # the same gradients: the unclipped momentum passes of the two dtypes round differently
                opts[3].step(runs[3][1])
            opts[2].host_copies_done.synchronize()
            torch.cuda.synchronize()
            assert ma.ma_device_status() == ma.MA_OK
            for which in (1, 2, 3):
                for i, (a, b) in enumerate(zip(runs[0][0], runs[which][0])):
                    assert torch.equal(a, b), (k, which, i)
                for i, (sa, sb) in enumerate(zip(opts[0].state, opts[which].state)):
                    assert torch.equal(sa[0], sb[0]) and (sa[1] is None or torch.equal(sa[1], sb[1])), (k, which, i)
            for a, b in zip(runs[0][1], fresh):
                assert torch.equal(a, b)  # the gradients stay as they are
        # captured: clipped; then without clipping; then clipped again
        assert opts[1].graph_captures == 3
    finally:
        ma.ma_set_momentum_overlap(False)


def test_other_stream_and_captured_replay():
    _, views = make(LISTS["offsets"], 9)
    clip = ma.GradClip(views)
    P, M, V = ([torch.zeros(v.numel(), device="cuda") for v in views] for _ in range(3))
    hp = ma.adamw_hparams(step=1)
    bf = [k for k, v in enumerate(views) if v.dtype == torch.bfloat16]
    pick = lambda xs: [xs[k] for k in bf]  # noqa: E731
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        clip.norm(max_norm=0.1)
    s.synchronize()
    assert float(clip.buffer[0]) == pytest.approx(norm64(views), rel=TOL_NORM)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        clip.norm(max_norm=0.1)
        ma.adamw_step_fused(pick(P), pick(views), pick(M), pick(V), hp, clip=clip.buffer)
    for k in range(3):
        for v in views:
            v.normal_(std=0.01 * (k + 1))
        for x in P + M + V:
            x.zero_()
        graph.replay()
        ref = norm64(views)
        assert float(clip.buffer[0]) == pytest.approx(ref, rel=TOL_NORM)
        for v, m in zip(pick(views), pick(M)):
            want = v.double() * (0.1 / ref) * (1 - np.float32(0.9).astype(np.float64))
            assert ((m.double() - want).abs() <= want.abs() * (TOL_NORM + 4 * U)).all()


def test_results_repeat_bit_for_bit():
    _, views = make(LISTS["long"], 10)
    clip, other = ma.GradClip(views), ma.GradClip(views)
    clip.norm()
    for _ in range(3):
        other.norm()
        assert torch.equal(clip.buffer[:4], other.buffer[:4])


@pytest.mark.parametrize("dt", ["fp32", "bf16"])
def test_sharded_step_on_one_rank(dt):
    import torch.distributed as dist
    from adamw_hybrid_optimizer_muon_b200.dist import DistMuonAdamW
    s = socket.socket()
    s.bind(("127.0.0.1", 0))
    port = s.getsockname()[1]
    s.close()
    torch.cuda.set_device(0)
    dist.init_process_group("nccl", init_method=f"tcp://127.0.0.1:{port}", rank=0, world_size=1,
                            timeout=datetime.timedelta(seconds=120))
    try:
        (pa, G), (pb, _) = _table(2, dt), _table(2, dt)
        ref = _opt(pa)
        opt = DistMuonAdamW([(p, role, g) for p, (_, role, g) in zip(pb, TABLE)],
                            [("muon", ma.muon_hparams()), ("adamw", ma.adamw_hparams(lr=0.01))],
                            grad_dtype=DT[dt], seg_cap=1 << 16)
        hf = torch.zeros(opt.flat_grad.shape, dtype=DT[dt], pin_memory=True)
        for k, kw in enumerate([dict(max_norm=0.3), dict(max_norm=0.2, grad_scale=0.5), {}, dict(max_norm=0.1)]):
            before = [p.clone() for p in pa]
            ref.step(G, **kw)
            if k == 1:
                for h, g in zip(opt.host_views(hf), G):
                    h.copy_(g)
                opt.step_from_host(hf, **kw)
            else:
                for v, g in zip(opt.grads, G):
                    v.copy_(g)
                opt.step(**kw)
            torch.cuda.synchronize()
            assert ma.ma_device_status() == ma.MA_OK
            if kw:
                assert float(opt.grad_norm) == pytest.approx(float(ref.grad_norm), rel=2 * TOL_NORM)
            # Chunks of other tensors' pieces add in another order, so coef may differ by 2 TOL_NORM. One AdamW
            # update moves by at most that times its own size (it is a ratio that does not grow with g); a Muon
            # update stays within its bf16 operands' tolerance.
            for (shape, role, grp), a, b, p0 in zip(TABLE, pa, pb, before):
                moved = float((a - p0).double().norm())
                tol = 2e-2 if grp == 0 else 1e-4
                assert float((a - b).double().norm()) <= tol * moved + 1e-7 * float(a.double().norm()), (k, shape)
        opt.close()
    finally:
        dist.destroy_process_group()
