"""Clipping, embedding and QK-Clip on buffers whose element offsets pass 32 bits (4 to 9 GB each).

Bounds as in the operators' own tests: the values are chosen so that each
result is exact (ones and powers of two), and compared for equality.
"""
import math

import pytest

torch = pytest.importorskip("torch")

import adamw_hybrid_optimizer_muon_b200 as ma

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _release():
    yield
    torch.cuda.synchronize()
    assert ma.ma_device_status() == ma.MA_OK
    torch.cuda.empty_cache()


def test_norm_and_clipping():
    n = (1 << 32) + 12345
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    for i in (0, 7, 1 << 31, (1 << 32) - 1, 1 << 32, n - 1, n - 2, 12344, (1 << 32) + 5):
        g[i] = 4.0
    c = ma.GradClip([g])
    assert float(c.norm()) == 12.0
    assert float(c.clip(6.0)) == 12.0
    assert int((g == 2.0).sum()) == 9 and float(g[n - 1]) == 2.0 and float(g[1 << 32]) == 2.0 and float(g[12345]) == 0.0


def test_lookup_and_gradient():
    V, D = 1_200_003, 2048  # 2.46e9 elements
    ids = torch.tensor([0, V - 1, 1048576, V - 1, 1048575, 5, V - 2], device="cuda")
    dy = torch.ones((7, D), dtype=torch.bfloat16, device="cuda")
    grad = torch.full((V, D), 3.0, dtype=torch.bfloat16, device="cuda")
    ma.embedding_grad(ids, dy, grad, scale=2.0)
    want = {0: 2.0, V - 1: 4.0, 1048576: 2.0, 1048575: 2.0, 5: 2.0, V - 2: 2.0}
    sums = torch.stack([grad[a:a + 100_000].sum(dim=1, dtype=torch.float32) for a in range(0, V - 100_000, 100_000)]
                       ).flatten()
    for v, x in want.items():
        assert bool((grad[v] == x).all()), v
    rest = torch.ones_like(sums, dtype=torch.bool)
    rest[[v for v in want if v < sums.numel()]] = False
    assert bool((sums[rest] == 0).all()) and bool((grad[sums.numel():V - 2] == 0).all())
    out = ma.embedding_lookup(ids, grad, scale=0.5)
    assert torch.equal(out, torch.tensor([1.0, 2, 1, 2, 1, 1, 1], device="cuda").bfloat16()[:, None].expand(7, D))
    # many tokens: the rows looked up pass 32 bits too
    many = torch.full((1_100_000,), V - 1, device="cuda")
    rows = ma.embedding_lookup(many, grad)
    assert bool((rows[-1] == 4.0).all()) and bool((rows[1_048_576] == 4.0).all())
    del grad
    small = torch.empty((3, D), device="cuda")
    ma.embedding_grad(torch.arange(1_100_000, device="cuda") % 2, rows, small)  # 550,000 times 4.0: exact in fp32
    assert bool((small[:2] == 2_200_000.0).all()) and bool((small[2] == 0).all())


def test_largest_logit():
    n, H, D, T = 1_050_000, 32, 128, 500  # 4.3e9 elements of queries
    q = torch.zeros((n, H, D), dtype=torch.bfloat16, device="cuda")
    k = torch.zeros((n, 1, D), dtype=torch.bfloat16, device="cuda")
    k[n - 30, 0, 3] = 2.0
    for h in range(H):
        q[n - 20, h, 3] = float(h + 1)
    q[n - 40] = 100.0  # before its key
    off = torch.arange(0, n + 1, T, dtype=torch.int32, device="cuda")
    got = ma.qk_max_logit(q, k, scale=1.0, offsets=off, max_len=T)
    assert torch.equal(got, torch.arange(1, H + 1, device="cuda") * 2.0)
    got = ma.qk_max_logit(q.view(n // T, T, H, D), k.view(n // T, T, 1, D), scale=1.0)
    assert torch.equal(got, torch.arange(1, H + 1, device="cuda") * 2.0)
    assert float(ma.qk_max_logit(q.view(n // T, T, H, D), k.view(n // T, T, 1, D), scale=1.0, causal=False).min()) == 200.0
    assert math.isfinite(float(got.max()))
