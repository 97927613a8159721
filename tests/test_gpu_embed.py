"""Embedding lookup and its gradient on the GPU, against the formulas in fp64.

Tolerances, from the arithmetic. Lookup: one fp32 product (2^-24) and the
output's rounding (half a step). Gradient of a row with c tokens: c - 1 fp32
additions, whatever their order, are off by at most (c - 1) 2^-24 of the sum of
magnitudes (to first order; twice that is granted), one product, one addition
of the old value, and the output's rounding.
"""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import adamw_hybrid_optimizer_muon_b200 as ma

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def make_ids(kind, n, V, seed=0):
    r = np.random.default_rng([n, V, seed])
    if kind == "uniform":
        x = r.integers(0, V, n)
    elif kind == "zipf":
        x = r.permutation(V)[np.minimum((np.exp(r.random(n) * math.log(V + 1))).astype(np.int64) - 1, V - 1)]
    elif kind == "one":
        x = np.full(n, V - 1)
    elif kind == "two":
        x = np.where(r.random(n) < 0.5, 0, V - 1)
    elif kind == "descending":
        x = (V - 1 - np.arange(n)) % V
    return torch.from_numpy(x.astype(np.int64)).cuda()


def ref_grad(ids, dy, V, scale, padding=None):
    """(sum, sum of magnitudes, count) per row, in fp64."""
    keep = (ids >= 0) & (ids < V)
    if padding is not None:
        keep &= ids != padding
    ids, dy = ids[keep].long(), dy[keep].double()
    s = torch.zeros((V, dy.shape[1]), dtype=torch.float64, device="cuda").index_add_(0, ids, dy)
    a = torch.zeros_like(s).index_add_(0, ids, dy.abs())
    c = torch.bincount(ids, minlength=V).double()[:, None]
    return s * scale, a * abs(scale), c


def check_grad(got, s, a, c, old=None):
    want = s if old is None else s + old.double()
    half = torch.finfo(got.dtype).eps / 2
    err = 2 * (c + 1) * U * a + U * want.abs()
    tiny = torch.finfo(got.dtype).tiny * torch.finfo(got.dtype).eps
    bad = (got.double() - want).abs() > err + half * (want.abs() + err) + tiny
    assert not bad.any(), (int(bad.sum()), float((got.double() - want).abs().max()))


CASES = [  # tokens, rows, dim, ids
    (1, 1, 1, "one"), (1, 7, 8, "uniform"), (2, 3, 2, "one"), (31, 5, 6, "uniform"), (64, 64, 64, "descending"),
    (65, 100, 24, "zipf"), (301, 5003, 514, "zipf"), (1000, 10, 40, "uniform"), (1000, 2, 1001, "two"),
    (4097, 999, 130, "zipf"), (8191, 300, 16, "zipf"), (8192, 32000, 64, "uniform"), (8192, 32000, 72, "one"),
    (8193, 32000, 64, "zipf"), (8193, 1, 9, "one"), (20000, 65536, 32, "zipf"), (20000, 65535, 8, "descending"),
    (40000, 262143, 8, "zipf"), (40000, 262144, 16, "uniform"), (3000, 600000, 4, "uniform"), (100000, 50, 3, "zipf"),
    (100000, 70000, 128, "one"), (300000, 1000, 8, "two"), (5000, 130, 2056, "zipf"),
]


@pytest.mark.parametrize("n,V,D,kind", CASES)
@pytest.mark.parametrize("ydt,gdt", [("bf16", "bf16"), ("fp32", "fp32"), ("bf16", "fp32"), ("fp32", "bf16")])
def test_grad_matches_fp64(n, V, D, kind, ydt, gdt):
    g = gen(n + D)
    ids = make_ids(kind, n, V)
    dy = (torch.randn((n, D), generator=g, device="cuda") * 1e-2).to(DT[ydt])
    grad = torch.full((V, D), math.nan, dtype=DT[gdt], device="cuda")  # every row is written
    kept = ids.clone(), dy.clone()
    ma.embedding_grad(ids, dy, grad, scale=1.7)
    f = float(np.float32(1.7))
    s, a, c = ref_grad(ids, dy, V, f)
    check_grad(grad, s, a, c)
    assert torch.equal(ids, kept[0]) and torch.equal(dy, kept[1])
    old = (torch.randn((V, D), generator=g, device="cuda") * 1e-2).to(DT[gdt])
    acc = old.clone()
    ma.embedding_grad(ids.int(), dy, acc, scale=1.7, accumulate=True)
    check_grad(acc, s, a, c, old)
    untouched = (c == 0).squeeze(1)
    assert torch.equal(acc[untouched], old[untouched])
    again = torch.full_like(grad, 3.0)
    ma.embedding_grad(ids, dy, again, scale=1.7)
    assert torch.equal(again, grad)  # the same bits
    assert ma.ma_device_status() == ma.MA_OK


@pytest.mark.parametrize("n", [700, 9000])
def test_padding_and_ids_outside_the_table(n):
    V, D = 400, 40
    ids = make_ids("zipf", n, V)
    ids[::7] = -1
    ids[1::50] = 3
    dy = torch.randn((n, D), generator=gen(1), device="cuda")
    grad = torch.empty((V, D), device="cuda")
    ma.embedding_grad(ids, dy, grad, padding=-1)
    assert ma.ma_device_status() == ma.MA_OK
    check_grad(grad, *ref_grad(ids, dy, V, 1.0))
    ids = ids.clamp_(min=0)
    ma.embedding_grad(ids, dy, grad, padding=3)
    assert ma.ma_device_status() == ma.MA_OK
    check_grad(grad, *ref_grad(ids, dy, V, 1.0, padding=3))
    assert not grad[3].any()
    ids[5], ids[n - 1], ids[77] = V, -5, 1 << 40
    ma.embedding_grad(ids, dy, grad)
    assert ma.ma_device_status() == ma.MA_ERR_BOUNDS and ma.ma_device_status() == ma.MA_OK
    check_grad(grad, *ref_grad(ids, dy, V, 1.0))
    ids[:] = -1
    ma.embedding_grad(ids, dy, grad, padding=-1)
    assert not grad.any() and ma.ma_device_status() == ma.MA_OK


def test_nothing_to_do():
    grad = torch.ones((10, 8), device="cuda")
    none = torch.zeros(0, dtype=torch.int64, device="cuda")
    ma.embedding_grad(none, torch.zeros((0, 8), device="cuda"), grad, accumulate=True)
    assert (grad == 1).all()
    ma.embedding_grad(none, torch.zeros((0, 8), device="cuda"), grad)
    assert not grad.any()
    ma.embedding_grad(none, torch.zeros((0, 0), device="cuda"), torch.zeros((10, 0), device="cuda"))
    large = torch.ones((1 << 20, 3), dtype=torch.bfloat16, device="cuda")
    ma.embedding_grad(none, torch.zeros((0, 3), device="cuda"), large)
    assert not large.any()
    assert ma.embedding_lookup(none, grad).shape == (0, 8)
    assert ma.embedding_lookup(none + 0, torch.zeros((0, 8), device="cuda")).shape == (0, 8)


@pytest.mark.parametrize("D,off,ld", [(64, 0, 80), (64, 1, 72), (63, 0, 64), (64, 2, 66), (8, 8, 24)])
@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_strided_and_offset_rows(D, off, ld, dt):
    n, V = 777, 120
    g = gen(4)
    buf = lambda rows: (torch.randn(rows * ld + off + 8, generator=g, device="cuda")).to(DT[dt])  # noqa: E731
    view = lambda b, rows: torch.as_strided(b, (rows, D), (ld, 1), off)  # noqa: E731
    ids = make_ids("zipf", n, V)
    by, bg, bt, bo = buf(n), buf(V), buf(V), buf(n)
    kg, ko = bg.clone(), bo.clone()
    ma.embedding_grad(ids, view(by, n), view(bg, V), scale=0.5)
    check_grad(view(bg, V), *ref_grad(ids, view(by, n), V, 0.5))
    ma.embedding_lookup(ids, view(bt, V), scale=3.0, out=view(bo, n))
    want = view(bt, V)[ids].double() * 3
    assert ((view(bo, n).double() - want).abs() <= want.abs() * (U + torch.finfo(DT[dt]).eps / 2)).all()
    for b, k, rows in ((bg, kg, V), (bo, ko, n)):  # between the rows nothing changes
        mask = torch.ones_like(b, dtype=torch.bool)
        view(mask, rows)[:] = False
        assert torch.equal(b[mask], k[mask])


@pytest.mark.parametrize("n,V,D", [(1, 5, 1), (16, 65536, 1280), (77, 100, 513), (300, 50, 4096), (9, 10, 20000),
                                   (5000, 1000, 96), (3, 4, 2)])
@pytest.mark.parametrize("tdt,odt", [("fp32", "bf16"), ("fp32", "fp32"), ("bf16", "bf16"), ("bf16", "fp32")])
def test_lookup_matches_fp64(n, V, D, tdt, odt):
    table = torch.randn((V, D), generator=gen(5), device="cuda").to(DT[tdt])
    ids = make_ids("uniform", n, V)
    for i in (ids, ids.int()):
        out = ma.embedding_lookup(i, table, scale=45.25, dtype=DT[odt])
        want = table[ids].double() * 45.25
        assert out.dtype == DT[odt]
        assert ((out.double() - want).abs() <= want.abs() * (U + torch.finfo(DT[odt]).eps / 2 * (1 + U))).all()
    same = ma.embedding_lookup(ids, table)
    assert torch.equal(same, table[ids])  # scale 1: a copy
    assert ma.ma_device_status() == ma.MA_OK


def test_lookup_of_ids_outside_the_table():
    table = torch.randn((10, 40), device="cuda")
    ids = torch.tensor([[3, -1, 9], [-1, 0, 5]], device="cuda")
    out = ma.embedding_lookup(ids, table, padding=-1)
    assert ma.ma_device_status() == ma.MA_OK
    assert not out[0, 1].any() and not out[1, 0].any() and torch.equal(out[0, 2], table[9])
    assert torch.equal(ma.embedding_lookup(ids.clamp(min=0), table, padding=3)[0, 0], table[3])  # a row like any other
    ids[0, 0] = 10
    out = ma.embedding_lookup(ids, table, padding=-1)
    assert ma.ma_device_status() == ma.MA_ERR_BOUNDS
    assert not out[0, 0].any() and torch.equal(out[0, 2], table[9])
    assert ma.ma_device_status() == ma.MA_OK


def test_infinities_stay_in_their_rows():
    n, V, D = 500, 40, 16
    ids = make_ids("zipf", n, V)
    dy = torch.randn((n, D), device="cuda")
    bad = int(ids[10])
    dy[10, 3], dy[10, 4] = math.inf, math.nan
    grad = torch.empty((V, D), device="cuda")
    ma.embedding_grad(ids, dy, grad)
    fine = torch.isfinite(grad)
    assert not fine[bad, 3] and not fine[bad, 4] and int((~fine).sum()) == 2


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_autograd_matches_the_formula_and_differences(dtype):
    V, D, n = 50, 24, 200
    table = torch.nn.Parameter(torch.randn((V, D), generator=gen(6), device="cuda"))
    ids = make_ids("zipf", n, V).view(10, 20)
    w = torch.randn((10, 20, D), generator=gen(7), device="cuda")
    loss = (ma.embedding(ids, table, scale=2.0, dtype=DT[dtype]).float() * w).sum()
    loss.backward()
    dy = w.to(DT[dtype])
    check_grad(table.grad, *ref_grad(ids.view(-1), dy.view(-1, D), V, 2.0))
    first = table.grad.clone()
    (ma.embedding(ids, table, scale=2.0, dtype=DT[dtype]).float() * w).sum().backward()
    assert torch.equal(table.grad, 2 * first)  # accumulated by autograd
    # into the optimizer's buffer: no .grad, and sums over micro-batches
    buf = torch.zeros((V, D), device="cuda")
    other = torch.nn.Parameter(table.detach().clone())
    for _ in range(2):
        (ma.embedding(ids, other, scale=2.0, dtype=DT[dtype], grad=buf).float() * w).sum().backward()
    assert other.grad is None
    s, a, c = ref_grad(ids.view(-1), dy.view(-1, D), V, 2.0)
    check_grad(buf, 2 * s, 2 * a, 2 * c + 1)
    # a broadcast gradient (sum of the output)
    table.grad = None
    ma.embedding(ids, table, scale=2.0).sum().backward()
    assert torch.equal(table.grad, 2 * torch.bincount(ids.view(-1), minlength=V).float()[:, None].expand(V, D))
    if dtype == "fp32":  # differences along a direction: the loss is linear in the table
        d = torch.randn((V, D), generator=gen(8), device="cuda")
        f = lambda t: float((ma.embedding_lookup(ids, t, scale=2.0).double() * w.double()).sum())  # noqa: E731
        t0 = table.detach()
        slope = (f(t0 + d) - f(t0 - d)) / 2
        got = float((first.double() * d.double()).sum())
        size = float((first.double() * d.double()).abs().sum()) + 2 * float((w.double().abs()).sum()) * 4
        assert abs(got - slope) <= 64 * U * size


def test_streams_and_captured_replay():
    n, V, D = 9000, 500, 64
    ids, dy = make_ids("zipf", n, V), torch.randn((n, D), device="cuda")
    grad = torch.empty((V, D), device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ma.embedding_grad(ids, dy, grad, stream=s)
    out = ma.embedding_lookup(ids, grad, stream=s)
    s.synchronize()
    check_grad(grad, *ref_grad(ids, dy, V, 1.0))
    assert torch.equal(out, grad[ids])
    ws = torch.empty(ma.embed_grad_workspace_bytes(n, V, D), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ma.embedding_grad(ids, dy, grad, ws=ws)
        ma.embedding_lookup(ids, grad, out=out)
    for k in range(3):
        ids.copy_(make_ids("zipf", n, V, seed=k + 1))
        dy.normal_()
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        check_grad(grad, *ref_grad(ids, dy, V, 1.0))
        assert torch.equal(out, grad[ids])
    assert ma.ma_device_status() == ma.MA_OK


def test_runs_around_the_lengths_where_they_are_cut():
    # runs of 1 to 400 tokens, beginning at every offset of a tile, some after one another without a gap
    r = np.random.default_rng(3)
    lengths = [1, 63, 64, 65, 127, 128, 129, 130, 191, 192, 193, 255, 256, 257, 400] + list(r.integers(1, 300, 120))
    for n_extra in (0, 9000):  # the one-block sort takes the first, the sort by tiles both together
        V, D = 700, 24
        runs = r.permutation(lengths)[:40 if not n_extra else None]
        keys = np.repeat(np.sort(r.permutation(V)[:len(runs)]), runs)
        ids = torch.from_numpy(r.permutation(keys).astype(np.int64)).cuda()
        assert (len(keys) > 8192) == bool(n_extra)
        dy = torch.randn((len(keys), D), generator=gen(9), device="cuda")
        grad = torch.full((V, D), 7.0, device="cuda")
        ma.embedding_grad(ids, dy, grad)
        check_grad(grad, *ref_grad(ids, dy, V, 1.0))
        assert ma.ma_device_status() == ma.MA_OK


def test_many_tokens_reach_several_tiles_per_block():
    # more than 512 tiles of 4096 tokens: a block ranks several one after the other
    n, V, D = 512 * 4096 + 12345, 50000, 4
    ids = make_ids("zipf", n, V)
    dy = torch.ones((n, D), device="cuda")
    grad = torch.empty((V, D), device="cuda")
    ma.embedding_grad(ids, dy, grad)
    count = torch.bincount(ids, minlength=V)
    assert torch.equal(grad, count.float()[:, None].expand(V, D))  # counts below 2^24 are exact


def test_arguments_that_do_not_fit():
    ids = torch.zeros((3, 4), dtype=torch.int64, device="cuda")
    tab = torch.zeros((5, 8), device="cuda")
    for call, code in [
        (lambda: ma.embedding_lookup(ids.float(), tab), ma.MA_ERR_DTYPE),
        (lambda: ma.embedding_lookup(ids, tab.half()), ma.MA_ERR_DTYPE),
        (lambda: ma.embedding_lookup(ids, tab[0]), ma.MA_ERR_SHAPE),
        (lambda: ma.embedding_lookup(ids, tab.t()), ma.MA_ERR_SHAPE),
        (lambda: ma.embedding_lookup(ids, tab, out=torch.zeros((3, 4, 7), device="cuda")), ma.MA_ERR_SHAPE),
        (lambda: ma.embedding_lookup(ids, tab, out=torch.zeros((3, 4, 8), device="cuda").transpose(0, 1)
                                     .contiguous().transpose(0, 1)), ma.MA_ERR_SHAPE),
        (lambda: ma.embedding_grad(ids, torch.zeros((3, 4, 7), device="cuda"), tab), ma.MA_ERR_SHAPE),
        (lambda: ma.embedding_grad(ids, torch.zeros((3, 4, 8), device="cuda").half(), tab), ma.MA_ERR_DTYPE),
        (lambda: ma.embedding_grad(ids, torch.zeros((1, 1, 8), device="cuda").expand(3, 4, 8), tab), ma.MA_ERR_SHAPE),
        (lambda: ma.embedding_grad(ids, torch.zeros((3, 4, 8), device="cuda"), tab,
                                   ws=torch.zeros(16, dtype=torch.uint8, device="cuda")), ma.MA_ERR_WORKSPACE),
        (lambda: ma.embedding_lookup(ids, tab, out=tab.new_zeros(200)[:96].view(3, 4, 8), dtype=torch.bfloat16),
         ma.MA_ERR_SHAPE),
    ]:
        with pytest.raises(ma.MAError) as e:
            call()
        assert e.value.code == code


@pytest.mark.parametrize("n,D", [(2000, 40), (60000, 8), (500000, 8), (1000000, 16), (1000003, 1)])
def test_long_runs_of_every_length(n, D):
    # runs through zero to many tiles of the sum (8 to 512 tokens each), several of them side by side, first and last
    # in the batch's order, in rows whose ends are not at vectors' borders
    r = np.random.default_rng(n)
    lengths = []
    while sum(lengths) < n:
        lengths.append(int(min(n - sum(lengths), r.choice([1, 31, 33, 64, 257, 513, 600, 4097, 4700, n // 5]))))
    V = len(lengths) + 3
    rows = np.sort(r.permutation(V)[:len(lengths)])
    ids = torch.from_numpy(r.permutation(np.repeat(rows, lengths))).cuda()
    dy = torch.randn((n, D), generator=gen(n), device="cuda").bfloat16()
    for ld in (D, D + 3):
        full = torch.full((V, ld), 7.0, dtype=torch.bfloat16, device="cuda")
        grad = full[:, :D]
        ma.embedding_grad(ids, dy, grad)
        check_grad(grad, *ref_grad(ids, dy, V, 1.0))
        assert (full[:, D:] == 7).all()  # what lies between the rows stays
    assert ma.ma_device_status() == ma.MA_OK


@pytest.mark.parametrize("n", [5, 9000])
@pytest.mark.parametrize("D", [1, 3, 7, 8, 9, 15, 1283])
@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_zeros_of_rows_at_any_alignment(n, D, dt):
    V, off, ld = 500, 3, D + 5
    flat = torch.full((off + V * ld,), 7.0, dtype=DT[dt], device="cuda")
    grad = flat[off:off + V * ld].view(V, ld)[:, :D]
    ids = make_ids("uniform", n, V // 10)
    dy = torch.randn((n, D), generator=gen(n), device="cuda").to(DT[dt])
    ma.embedding_grad(ids, dy, grad)
    check_grad(grad, *ref_grad(ids, dy, V, 1.0))
    assert (flat[:off] == 7).all() and (flat[off:].view(V, ld)[:, D:] == 7).all()
    assert ma.ma_device_status() == ma.MA_OK


@pytest.mark.parametrize("n", [3, 700, 40000])
@pytest.mark.parametrize("D", [1, 8, 24, 1280, 1282, 2056, 5000])
def test_lookup_of_rows_that_do_not_fill_a_block(n, D):
    table = torch.randn((300, D), generator=gen(D), device="cuda").bfloat16()
    ids = make_ids("zipf", n, 300)
    assert torch.equal(ma.embedding_lookup(ids, table), table[ids])  # a scale of one: the same bits
    assert ma.ma_device_status() == ma.MA_OK


def test_captured_backward_while_an_eager_pass_lives():
    table = torch.randn((90, 24), generator=gen(30), device="cuda", requires_grad=True)
    ids = make_ids("zipf", 500, 90)
    w = torch.randn((500, 24), generator=gen(31), device="cuda")
    buf = torch.zeros((90, 24), device="cuda")
    loss = lambda: (ma.embedding(ids, table, grad=buf) * w).sum()  # noqa: E731
    loss().backward()  # the uncaptured passes: one done, one that still waits for its backward
    want = buf.clone()
    kept = loss()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        buf.zero_()
        loss().backward()
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(buf, want)
    kept.backward()
    torch.cuda.synchronize()
    s, a, c = ref_grad(ids, w, 90, 1.0)
    check_grad(buf, s, a, c, want)
    assert table.grad is None and ma.ma_device_status() == ma.MA_OK


def test_nothing_needs_a_gradient():
    table = torch.randn((9, 8), device="cuda")
    ids = make_ids("uniform", 5, 9)
    buf = torch.zeros((9, 8), device="cuda")
    assert not ma.embedding(ids, table, grad=buf).requires_grad
    table.requires_grad_()
    with torch.no_grad():
        assert not ma.embedding(ids, table, grad=buf).requires_grad
    assert ma.embedding(ids, table, grad=buf).requires_grad and ma.embedding(ids, table).requires_grad


@pytest.mark.parametrize("kind", ["zipf", "two", "uniform"])
@pytest.mark.parametrize("n,D", [(5000, 2058), (4200, 1027), (4200, 4099)])
@pytest.mark.parametrize("ydt,gdt", [("bf16", "fp32"), ("fp32", "bf16")])
def test_wide_rows_of_narrow_vectors(n, D, kind, ydt, gdt):
    # rows of more than 1024 vectors of one or two elements: a thread takes four of them
    V = 700
    ids = make_ids(kind, n, V)
    dy = (torch.randn((n, D), generator=gen(n), device="cuda") * 1e-2).to(DT[ydt])
    grad = torch.full((V, D), math.nan, dtype=DT[gdt], device="cuda")
    ma.embedding_grad(ids, dy, grad, scale=0.5)
    check_grad(grad, *ref_grad(ids, dy, V, 0.5))
    assert ma.ma_device_status() == ma.MA_OK


@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 65, 320])
@pytest.mark.parametrize("kind", ["one", "two", "zipf", "blocks"])
@pytest.mark.parametrize("D", [5, 72, 2058, 100003])
def test_short_batches(n, kind, D):
    # up to 32 tokens no run is cut, and no kernel adds up partial rows
    V = 40
    ids = make_ids(kind, n, V) if kind != "blocks" else torch.arange(n, device="cuda") // 40
    dy = torch.randn((n, D), generator=gen(n + D), device="cuda").bfloat16()
    grad = torch.full((V, D), math.nan, device="cuda")
    ma.embedding_grad(ids, dy, grad)
    s, a, c = ref_grad(ids, dy, V, 1.0)
    check_grad(grad, s, a, c)
    old = grad.clone()
    ma.embedding_grad(ids, dy, grad, accumulate=True)
    check_grad(grad, s, a, c, old)
    assert ma.ma_device_status() == ma.MA_OK
