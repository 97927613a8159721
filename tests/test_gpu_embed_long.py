"""The table's gradient where the sort's blocks take several tiles each, and where runs are as long as they may be uncut.

Order. A run of up to kLong tokens is added in token order from zero, one fp32 addition a token: its sum is known to the
bit, and is another one when the sort is not stable. Counts (sums of ones) below 2^24 are exact in fp32. Other
tolerances: c - 1 fp32 additions of c values are off by at most (c - 1) 2^-24 of the sum of their magnitudes to first
order (twice that is granted), and a product and the output's rounding come after.
"""
import os
import re

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import adamw_hybrid_optimizer_muon_b200 as ma

pytestmark = pytest.mark.gpu

SRC = open(os.path.join(os.path.dirname(ma.__file__), "csrc", "embed.cu")).read()


def constant(name):
    return int(re.search(rf"constexpr int {name} = (\d+);", SRC).group(1))


LONG = constant("kLong")
TILE = constant("kTileThreads") * 2  # tokens a block ranks at a time
MOST = TILE * constant("kMaxTiles")  # tokens up to which a block ranks one tile
U = 2.0 ** -24


def sums_in_order(ids, dy, V):
    """Sums of each row's tokens in token order, an addition at a time, in dy's type."""
    order = torch.argsort(ids, stable=True)
    key = ids[order]
    count = torch.bincount(ids, minlength=V)
    nth = torch.arange(len(ids), device="cuda") - (count.cumsum(0) - count)[key]
    out = torch.zeros((V, dy.shape[1]), dtype=dy.dtype, device="cuda")
    for k in range(int(count.max())):
        at = order[nth == k]
        out[ids[at]] += dy[at]  # every row at most once
    return out, count


@pytest.mark.parametrize("n", [MOST + 1, 2 * MOST + 12345])
@pytest.mark.parametrize("V,D", [(5_000_003, 1), (4_000_000, 4)])
def test_blocks_that_rank_several_tiles_keep_the_order(n, V, D):
    assert re.search(r"constexpr int kTile = kTileThreads \* 2;", SRC)
    g = torch.Generator(device="cuda")
    g.manual_seed(n + D)
    ids = torch.randint(0, V, (n,), generator=g, device="cuda")
    dy = torch.randn((n, D), generator=g, device="cuda")
    want, count = sums_in_order(ids, dy, V)
    assert 4 < int(count.max()) <= LONG
    grad = torch.full((V, D), float("nan"), device="cuda")
    ma.embedding_grad(ids, dy, grad)
    assert torch.equal(grad, want)
    old = torch.randn((V, D), generator=g, device="cuda")
    acc = old.clone()
    ma.embedding_grad(ids.int(), dy, acc, accumulate=True)
    assert torch.equal(acc, torch.where(count[:, None] > 0, want + old, old))
    assert ma.ma_device_status() == ma.MA_OK


@pytest.mark.parametrize("n", [MOST + 1, 2 * MOST + 12345])
def test_blocks_that_rank_several_tiles_of_few_rows(n):
    V = 50000
    r = np.random.default_rng(n)
    ids = torch.from_numpy(np.minimum((V ** r.random(n)).astype(np.int64) - 1, V - 1)).cuda()  # often the first rows
    count = torch.bincount(ids, minlength=V)
    assert int(count.max()) < 1 << 24
    grad = torch.empty((V, 2), device="cuda")
    ma.embedding_grad(ids, torch.ones((n, 2), device="cuda"), grad)
    assert torch.equal(grad, count.float()[:, None].expand(V, 2))
    assert ma.ma_device_status() == ma.MA_OK


@pytest.mark.parametrize("n", [900, 8000, 9000, 60_000, 1_200_000])
@pytest.mark.parametrize("D", [8, 24, 514])
@pytest.mark.parametrize("dt", ["fp32", "bf16"])
def test_runs_just_below_and_above_the_length_where_they_are_cut(n, D, dt):
    # runs of LONG - 2 to LONG + 2 tokens beginning at every offset of the sums' tiles (8 to 512 tokens), with one to
    # nine single tokens before each
    D = D if n < 1_000_000 else min(D, 24)
    r = np.random.default_rng(n + D)
    m = n // 20
    lengths = np.stack([r.integers(LONG - 2, LONG + 3, m), *(r.integers(0, 2, (9, m)) * 1)], 1).reshape(-1)
    lengths = lengths[lengths > 0]
    lengths = lengths[:int(np.searchsorted(lengths.cumsum(), n, "right"))]
    V = len(lengths) + 50
    keys = np.repeat(np.sort(r.permutation(V)[:len(lengths)]), lengths)
    starts = (lengths.cumsum() - lengths)[lengths >= LONG - 2]
    assert n < 1_000_000 or len(set(starts % 512)) == 512
    ids = torch.from_numpy(r.permutation(keys)).cuda()
    t = {"fp32": torch.float32, "bf16": torch.bfloat16}[dt]
    dy = torch.randn((len(keys), D), device="cuda").to(t)
    grad = torch.full((V, D), 7.0, dtype=t, device="cuda")
    ma.embedding_grad(ids, dy, grad)
    count = torch.bincount(ids, minlength=V)[:, None].double()
    want = torch.zeros((V, D), dtype=torch.float64, device="cuda").index_add_(0, ids, dy.double())
    mag = torch.zeros_like(want).index_add_(0, ids, dy.double().abs())
    err = 2 * (count + 1) * U * mag
    assert torch.all((grad.double() - want).abs() <= err + torch.finfo(t).eps / 2 * (want.abs() + err))
    if dt == "fp32":
        exact, _ = sums_in_order(ids, dy, V)
        whole = (count <= LONG).squeeze(1)
        assert torch.equal(grad[whole], exact[whole])
    ones = torch.empty((V, D), device="cuda")
    ma.embedding_grad(ids, torch.ones_like(dy), ones)
    assert torch.equal(ones, count.float().expand(V, D))
    assert ma.ma_device_status() == ma.MA_OK
