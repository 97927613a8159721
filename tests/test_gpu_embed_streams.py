"""Lookups on several streams whose backward adds to one gradient buffer: no sum is lost.

Sums of ones: counts below 2^24 are exact in fp32, so the buffer has to hold them to the bit.
"""
import pytest

torch = pytest.importorskip("torch")

import adamw_hybrid_optimizer_muon_b200 as ma

pytestmark = pytest.mark.gpu


def branches(ids, table, grad, streams):
    """The sum of one lookup a stream, each joined to the current one."""
    here, outs = torch.cuda.current_stream(), []
    for x, s in zip(ids, streams):
        s.wait_stream(here)
        with torch.cuda.stream(s):
            outs.append(ma.embedding(x, table, grad=grad).sum())
        here.wait_stream(s)
    return sum(outs)


def counts(ids, V):
    return sum(torch.bincount(x, minlength=V) for x in ids).float()


@pytest.mark.parametrize("n,V,D", [(30000, 20000, 1024), (500, 64, 2048), (9000, 7, 33)])
def test_no_sum_is_lost(n, V, D):
    g = torch.Generator(device="cuda")
    g.manual_seed(n)
    table = torch.zeros((V, D), device="cuda", requires_grad=True)
    ids = [torch.randint(0, V, (n,), generator=g, device="cuda") for _ in range(3)]
    want = counts(ids, V)[:, None].expand(V, D)
    streams = [torch.cuda.Stream() for _ in ids]
    grad = torch.zeros((V, D), device="cuda")
    for _ in range(8):
        grad.zero_()
        branches(ids, table, grad, streams).backward()
        assert torch.equal(grad.clone(), want)  # read on the stream that called backward
    assert ma.ma_device_status() == ma.MA_OK


def test_views_of_one_buffer():
    V, D = 5000, 512
    table = torch.zeros((V, D), device="cuda", requires_grad=True)
    ids = [torch.arange(V, device="cuda").repeat(3) for _ in range(2)]
    flat = torch.zeros(V * D, device="cuda")
    streams = [torch.cuda.Stream() for _ in ids]
    for _ in range(8):
        flat.zero_()
        here = torch.cuda.current_stream()
        loss = 0
        for x, s in zip(ids, streams):
            s.wait_stream(here)
            with torch.cuda.stream(s):
                loss = loss + ma.embedding(x, table, grad=flat.view(V, D)).sum()
            here.wait_stream(s)
        loss.backward()
        assert torch.equal(flat, torch.full_like(flat, 6.0))


def test_captured_after_eager_and_eager_after_captured():
    V, D, n = 3000, 256, 20000
    table = torch.zeros((V, D), device="cuda", requires_grad=True)
    ids = [torch.randint(0, V, (n,), device="cuda") for _ in range(2)]
    want = counts(ids, V)[:, None].expand(V, D)
    grad = torch.zeros((V, D), device="cuda")
    streams = [torch.cuda.Stream() for _ in ids]

    def step():
        grad.zero_()
        branches(ids, table, grad, streams).backward()

    step()
    assert torch.equal(grad, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(4):
        grad.fill_(5.0)
        graph.replay()
        assert torch.equal(grad, want)
        step()
        assert torch.equal(grad, want)
    graph2 = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph2):
        step()
    grad.fill_(7.0)
    graph2.replay()
    assert torch.equal(grad, want)
    assert ma.ma_device_status() == ma.MA_OK
