"""QK-Clip on the GPU, against the formulas in fp64.

Tolerances, from the arithmetic. A logit is a sum of dim exact bf16 products
in fp32; whatever the order and rounding of the adds (a tensor core may cut
instead of rounding: a whole step, 2^-23), it is off by at most
(dim + 8) 2^-23 of the sum of the products' magnitudes, and so is a maximum of
logits by the largest of those; the scale adds 2^-24. A clipped weight has the
roundings of a quotient, a root (or powf, 4 steps) and a quotient, and of the
product.
"""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import adamw_hybrid_optimizer_muon_b200 as ma

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def reference(q, k, spans, scale, causal, absolute):
    """(maximum, error bound) per head, in fp64. q: tokens x H x D, k: tokens x KV x D; spans: (begin, end) of sequences."""
    H, KV, D = q.shape[1], k.shape[1], q.shape[2]
    top = torch.full((H,), -math.inf, dtype=torch.float64, device="cuda")
    mag = torch.zeros(H, dtype=torch.float64, device="cuda")
    for lo, hi in spans:
        if hi <= lo:
            continue
        for h in range(H):
            a, b = q[lo:hi, h].double(), k[lo:hi, h // (H // KV)].double()
            for r0 in range(0, hi - lo, 2048):
                x = a[r0:r0 + 2048] @ b.T * scale
                if absolute:
                    x = x.abs()
                if causal:
                    see = torch.arange(r0, r0 + x.shape[0], device="cuda")[:, None] >= torch.arange(hi - lo, device="cuda")
                    x = torch.where(see, x, -math.inf)
                top[h] = torch.maximum(top[h], x.max())
            mag[h] = torch.maximum(mag[h], (a.abs() @ b.abs().T * scale).max())
    return top, (D + 8) * 2 * U * mag + U * top.abs().nan_to_num(posinf=0.0, neginf=0.0)


def check(got, ref):
    top, err = ref
    assert got.dtype == torch.float32 and got.shape == top.shape
    fin = torch.isfinite(top)
    assert torch.equal(torch.isfinite(got), fin)
    assert torch.equal(got[~fin].double().nan_to_num(nan=7.0), top[~fin].nan_to_num(nan=7.0))
    bad = (got.double() - top).abs()[fin] > err[fin]
    assert not bad.any(), (got, top)


def randn(shape, seed, std=1.0):
    return (torch.randn(shape, generator=gen(seed), device="cuda") * std).bfloat16()


SHAPES = [  # sequences, tokens, query heads, key heads, dim
    (1, 1, 1, 1, 8), (1, 2, 3, 1, 64), (3, 1, 4, 4, 128), (2, 127, 2, 2, 64), (1, 128, 2, 1, 128), (1, 129, 2, 2, 72),
    (2, 255, 4, 2, 128), (1, 256, 1, 1, 256), (1, 257, 3, 3, 192), (2, 300, 6, 2, 96), (1, 385, 2, 2, 200),
    (5, 512, 2, 1, 128), (1, 513, 1, 1, 16), (1, 1000, 5, 5, 128), (1, 1025, 8, 2, 256), (2, 2049, 2, 2, 128),
    (40, 33, 3, 1, 64), (1, 1100, 2, 2, 160), (300, 5, 2, 2, 8),
]


@pytest.mark.parametrize("S,T,H,KV,D", SHAPES)
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("absolute", [True, False])
def test_max_logit_matches_fp64(S, T, H, KV, D, causal, absolute):
    q, k = randn((S, T, H, D), S + T, 2.0), randn((S, T, KV, D), D + 1)
    got = ma.qk_max_logit(q, k, scale=0.3, causal=causal, absolute=absolute)
    spans = [(i * T, (i + 1) * T) for i in range(S)]
    check(got, reference(q.view(-1, H, D), k.view(-1, KV, D), spans, float(np.float32(0.3)), causal, absolute))
    assert torch.equal(got, ma.qk_max_logit(q, k, scale=0.3, causal=causal, absolute=absolute))
    assert ma.ma_device_status() == ma.MA_OK


@pytest.mark.parametrize("T", [2, 128, 129, 256, 300, 511, 700])
@pytest.mark.parametrize("D", [64, 256])
def test_each_border_pair_counts_and_no_masked_one(T, D):
    # one visible pair has the largest logit, and larger ones lie right behind the mask
    pairs = {(0, 0), (T - 1, 0), (T - 1, T - 1), (T // 2, T // 2), (T // 2, 0), (T - 1, T // 2)}
    pairs |= {(i, j) for i in (127, 128, 255, 256, 257) for j in (0, 127, 128, 255, 256) if j <= i < T}
    for i, j in pairs:
        q = torch.zeros((1, T, 1, D), dtype=torch.bfloat16, device="cuda")
        k = torch.zeros_like(q)
        q[0, i, 0, 0], k[0, j, 0, 0] = 3, 5
        if j + 1 < T:
            q[0, :j + 1, 0, 1], k[0, j + 1:, 0, 1] = 100, 7  # every pair behind the diagonal of column j + 1
        assert float(ma.qk_max_logit(q, k, scale=1.0)) == 15.0, (i, j)
        q.neg_()
        assert float(ma.qk_max_logit(q, k, scale=1.0, absolute=True)) == 15.0, (i, j)


@pytest.mark.parametrize("lengths", [[1], [5], [128, 0, 256], [0, 0, 7], [300, 1, 0, 129, 77], [0], [1000, 24],
                                     [1] * 700, [17] * 90, list(range(40))])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("D", [72, 256])
def test_packed_sequences(lengths, causal, D):
    H, KV, gap = 4, 2, 3
    n = sum(lengths)
    q, k = randn((n + 2 * gap, H, D), n, 2.0), randn((n + 2 * gap, KV, D), n + 1)
    q[:gap], k[:gap], q[n + gap:], k[n + gap:] = math.nan, math.inf, math.nan, math.nan  # of no sequence
    ends = np.cumsum([gap] + lengths)
    off = torch.tensor(ends, dtype=torch.int32, device="cuda")
    got = ma.qk_max_logit(q, k, causal=causal, offsets=off, max_len=max(1, max(lengths)))
    check(got, reference(q, k, list(zip(ends[:-1], ends[1:])), float(np.float32(D ** -0.5)), causal, False))
    assert torch.equal(got, ma.qk_max_logit(q, k, causal=causal, offsets=off))  # max_len: all tokens
    assert ma.ma_device_status() == ma.MA_OK


def test_offsets_that_do_not_fit_are_cut_and_recorded():
    n, H, D = 200, 2, 64
    q, k = randn((n, H, D), 1), randn((n, H, D), 2)
    call = lambda off, **kw: ma.qk_max_logit(  # noqa: E731
        q, k, offsets=torch.tensor(off, dtype=torch.int32, device="cuda"), **kw)
    sc = float(np.float32(D ** -0.5))
    for off, kw, spans in [([0, 100, 300], {}, [(0, 100), (100, 200)]), ([-50, 100], {}, [(0, 100)]),
                           ([0, 150, 50, 60], {}, [(0, 150), (50, 60)]), ([0, 200], dict(max_len=90), [(0, 90)]),
                           ([500, 600], {}, [])]:
        got = call(off, **kw)
        assert ma.ma_device_status() == ma.MA_ERR_BOUNDS, off
        check(got, reference(q, k, spans, sc, True, False))
    call([0, 200])
    assert ma.ma_device_status() == ma.MA_OK


def test_nan_and_infinity():
    q, k = randn((1, 300, 3, 64), 3), randn((1, 300, 3, 64), 4)
    q[0, 200, 1, 5] = math.nan
    k[0, 17, 2, 9] = math.inf
    got = ma.qk_max_logit(q, k, absolute=True)
    assert math.isfinite(float(got[0])) and math.isnan(float(got[1])) and math.isinf(float(got[2]))
    got = ma.qk_max_logit(q, k, out=got, accumulate=True)  # a NaN stays
    assert math.isfinite(float(got[0])) and math.isnan(float(got[1]))
    w = torch.ones((192, 8), device="cuda")
    ma.qk_clip(w, w.clone(), got, tau=1e-3)
    assert bool((w[64:] == 1).all()) and bool((w[:64] < 1).all())  # heads that are not finite stay


def test_negative_maxima_and_zero():
    q = torch.full((1, 130, 2, 64), -1.0, dtype=torch.bfloat16, device="cuda")
    k = torch.ones((1, 130, 2, 64), dtype=torch.bfloat16, device="cuda")
    k[0, :, 1] = 0
    got = ma.qk_max_logit(q, k, scale=1.0)
    assert got.tolist() == [-64.0, 0.0]
    out = torch.tensor([-70.0, -1.0], device="cuda")
    assert ma.qk_max_logit(q, k, scale=1.0, out=out, accumulate=True).tolist() == [-64.0, 0.0]
    out = torch.tensor([-3.0, 2.0], device="cuda")
    assert ma.qk_max_logit(q, k, scale=1.0, out=out, accumulate=True).tolist() == [-3.0, 2.0]


def test_no_tokens():
    e = torch.zeros((0, 5, 2, 64), dtype=torch.bfloat16, device="cuda")
    assert ma.qk_max_logit(e, e).tolist() == [-math.inf] * 2
    e = torch.zeros((3, 0, 2, 64), dtype=torch.bfloat16, device="cuda")
    assert ma.qk_max_logit(e, e).tolist() == [-math.inf] * 2
    out = torch.tensor([1.0, 2.0], device="cuda")
    assert ma.qk_max_logit(e, e, out=out, accumulate=True).tolist() == [1.0, 2.0]


@pytest.mark.parametrize("KV", [2, 6])
def test_views_of_a_fused_projection(KV):
    S, T, H, D = 2, 333, 6, 64
    x = randn((S, T, (H + 2 * KV) * D), 5)
    q = x[..., :H * D].view(S, T, H, D)
    k = x[..., H * D:(H + KV) * D].view(S, T, KV, D)
    got = ma.qk_max_logit(q, k)
    spans = [(0, T), (T, 2 * T)]
    ref = reference(q.reshape(-1, H, D), k.reshape(-1, KV, D), spans, float(np.float32(D ** -0.5)), True, False)
    check(got, ref)
    # heads before tokens
    qh, kh = q.transpose(1, 2).contiguous(), k.transpose(1, 2).contiguous()
    assert torch.equal(got, ma.qk_max_logit(qh.transpose(1, 2), kh.transpose(1, 2)))


def test_strides_of_extents_of_one_are_not_looked_at():
    q, k = randn((1, 200, 1, 64), 30), randn((1, 200, 1, 64), 31)
    odd = lambda x: x.as_strided(x.shape, (3, 64, 5, 1))  # noqa: E731  one sequence, one head
    assert torch.equal(ma.qk_max_logit(q, k), ma.qk_max_logit(odd(q), odd(k)))


def test_micro_batches_add_up():
    q, k = randn((6, 200, 2, 128), 6), randn((6, 200, 2, 128), 7)
    whole = ma.qk_max_logit(q, k)
    out = ma.qk_max_logit(q[:2], k[:2])
    ma.qk_max_logit(q[2:5], k[2:5], out=out, accumulate=True)
    ma.qk_max_logit(q[5:], k[5:], out=out, accumulate=True)
    assert torch.equal(out, whole)


def test_long_sequence():
    q, k = randn((1, 8200, 2, 128), 8, 3.0), randn((1, 8200, 1, 128), 9)
    check(ma.qk_max_logit(q, k), reference(q[0], k[0], [(0, 8200)], float(np.float32(128 ** -0.5)), True, False))


def test_streams_and_captured_replay():
    q, k = randn((2, 400, 4, 64), 10), randn((2, 400, 4, 64), 11)
    wq, wk = (torch.randn((256, 128), generator=gen(12), device="cuda") for _ in range(2))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = ma.qk_max_logit(q, k, stream=s)
    s.synchronize()
    assert torch.equal(got, ma.qk_max_logit(q, k))
    a, b = wq.clone(), wk.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ma.qk_max_logit(q, k, out=got)
        ma.qk_clip(a, b, got, tau=2.0)
    for i in range(3):
        q.copy_(randn(q.shape, 20 + i))
        a.copy_(wq), b.copy_(wk), got.fill_(99.0)
        graph.replay()
        torch.cuda.synchronize()
        a2, b2 = wq.clone(), wk.clone()
        top = ma.qk_max_logit(q, k)
        ma.qk_clip(a2, b2, top, tau=2.0)
        assert torch.equal(got, top) and torch.equal(a, a2) and torch.equal(b, b2)
        assert not torch.equal(a, wq)
    assert ma.ma_device_status() == ma.MA_OK


@pytest.mark.parametrize("H,KV,dq,dk,C", [(1, 1, 1, 1, 1), (4, 4, 64, 64, 256), (6, 2, 32, 32, 100), (3, 1, 5, 7, 33),
                                          (8, 8, 128, 128, 1024), (2000, 40, 1, 2, 9), (2, 2, 0, 4, 8)])
@pytest.mark.parametrize("alpha", [0.5, 0.0, 1.0, 0.3])
@pytest.mark.parametrize("shift", [0, 1])
def test_clip_scales_the_weights(H, KV, dq, dk, C, alpha, shift):
    g = gen(13)
    flat = lambda rows: torch.randn(rows * C + shift, generator=g, device="cuda")[shift:].view(rows, C)  # noqa: E731
    wq, wk = flat(H * dq), flat(KV * dk)
    top = torch.rand(H, generator=g, device="cuda") * 150
    if H > 3:
        top[0], top[1], top[2], top[3] = math.inf, math.nan, -500.0, 100.0
    a, b = wq.clone(), wk.clone()
    ma.qk_clip(a, b, top, tau=100.0, alpha=alpha, kv_heads=KV)
    t = top.double()
    gam = torch.where((t > 100) & torch.isfinite(t), 100 / t, torch.ones_like(t))
    low = gam.view(KV, -1).amin(dim=1)
    fk = low ** (1 - alpha)
    fq = gam / fk.repeat_interleave(H // KV)
    tol = (8 if alpha in (0.0, 0.5, 1.0) else 24) * U
    for w, x, f in ((wq, a, fq), (wk, b, fk)):
        want = w.double().view(f.numel(), -1) * f[:, None]
        assert ((x.double().view(f.numel(), -1) - want).abs() <= tol * want.abs() + 1e-44).all()
        still = (f == 1)
        assert torch.equal(x.reshape(f.numel(), -1)[still], w.reshape(f.numel(), -1)[still])
    # every head's logits scale by its own factor
    assert ((fq * fk.repeat_interleave(H // KV) - gam).abs() <= 1e-12).all()


@pytest.mark.parametrize("H,KV", [(2, 2), (4, 2)])
def test_a_factor_below_the_smallest_number(H, KV):
    # tau / S underflows: the factor is the smallest normal number, never 0 or 0 / 0
    wq, wk = torch.full((H * 2, 8), 1e20, device="cuda"), torch.full((KV * 2, 8), 1e20, device="cuda")
    top = torch.full((H,), 1e20, device="cuda")
    top[1] = 0.5e-30
    ma.qk_clip(wq, wk, top, tau=1e-30, alpha=0.5, kv_heads=KV)
    tiny = torch.finfo(torch.float32).tiny  # 2^-126
    fq, fk = (wq.view(H, -1)[:, 0].double() / 1e20).cpu(), (wk.view(KV, -1)[:, 0].double() / 1e20).cpu()
    gam = torch.full((H,), tiny, dtype=torch.float64)
    gam[1] = 1.0
    want_k = gam.view(KV, -1).amin(dim=1) ** 0.5
    want_q = gam / want_k.repeat_interleave(H // KV)
    assert ((fk / want_k - 1).abs() <= 32 * U).all()
    if H > KV:  # the head within tau: 1e20 * 2^63 = 9.2e38 is more than fp32 holds
        assert torch.isinf(fq[1])
        fq, want_q = torch.cat((fq[:1], fq[2:])), torch.cat((want_q[:1], want_q[2:]))
    assert ((fq / want_q - 1).abs() <= 32 * U).all()


def test_clipped_projection_gives_tau():
    # q = x W_q^T, k = x W_k^T: after the clip the largest logits are tau, up to the bf16 rounding of q and k
    T, H, KV, D, C = 500, 4, 2, 64, 96
    x = torch.randn((T, C), generator=gen(14), device="cuda")
    wq, wk = torch.randn((H * D, C), generator=gen(15), device="cuda"), torch.randn((KV * D, C), generator=gen(16), device="cuda")
    wq[:D] *= 1e-3  # one head far below tau
    proj = lambda w, h: (x.double() @ w.double().T).bfloat16().view(1, T, h, D)  # noqa: E731
    before = ma.qk_max_logit(proj(wq, H), proj(wk, KV))
    tau = 50.0
    assert float(before[0]) < tau < float(before[1:].min())
    ma.qk_clip(wq, wk, before, tau=tau, kv_heads=KV)
    after = ma.qk_max_logit(proj(wq, H), proj(wk, KV))
    # rounding q and k moves a logit by at most (2^-7 + 2^-16) of the sum of magnitudes, here below 40 times the logit
    assert abs(float(after[0]) / float(before[0]) - 1) < 0.4
    assert ((after[1:] - tau).abs() <= tau * 2.0 ** -7 * 40 * 2).all() and (after[1:] < before[1:]).all()


def test_arguments_that_do_not_fit():
    q = torch.zeros((1, 8, 4, 64), dtype=torch.bfloat16, device="cuda")
    off = torch.tensor([0, 8], dtype=torch.int32, device="cuda")
    w = torch.zeros((8, 4), device="cuda")
    for call, code in [
        (lambda: ma.qk_max_logit(q.half(), q), ma.MA_ERR_DTYPE), (lambda: ma.qk_max_logit(q.float(), q.float()), ma.MA_ERR_DTYPE),
        (lambda: ma.qk_max_logit(q[0], q[0]), ma.MA_ERR_SHAPE), (lambda: ma.qk_max_logit(q, q[:, :7]), ma.MA_ERR_SHAPE),
        (lambda: ma.qk_max_logit(q, q[:, :, :3]), ma.MA_ERR_SHAPE),
        (lambda: ma.qk_max_logit(q[..., :60], q[..., :60]), ma.MA_ERR_ALIGN),
        (lambda: ma.qk_max_logit(q.transpose(2, 3), q.transpose(2, 3)), ma.MA_ERR_SHAPE),
        (lambda: ma.qk_max_logit(q, q, out=torch.zeros(3, device="cuda")), ma.MA_ERR_SHAPE),
        (lambda: ma.qk_max_logit(q, q, accumulate=True), ma.MA_ERR_NULL),
        (lambda: ma.qk_max_logit(q[0], q[0], offsets=off.long()), ma.MA_ERR_SHAPE),
        (lambda: ma.qk_max_logit(q[0], q[0], offsets=off.cpu()), ma.MA_ERR_ARG),
        (lambda: ma.qk_max_logit(q, q, scale=0.0), ma.MA_ERR_ARG),
        (lambda: ma.qk_clip(w, w.clone(), torch.zeros(3, device="cuda")), ma.MA_ERR_SHAPE),
        (lambda: ma.qk_clip(w, w, torch.zeros(2, device="cuda")), ma.MA_ERR_ARG),
        (lambda: ma.qk_clip(w.half(), w.clone(), torch.zeros(2, device="cuda")), ma.MA_ERR_DTYPE),
        (lambda: ma.qk_clip(w.t(), w.clone().t(), torch.zeros(2, device="cuda")), ma.MA_ERR_SHAPE),
        (lambda: ma.qk_clip(w, w.clone(), torch.zeros(4, device="cuda"), kv_heads=3), ma.MA_ERR_SHAPE),
    ]:
        with pytest.raises(ma.MAError) as e:
            call()
        assert e.value.code == code
