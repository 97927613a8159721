"""Calls for the default stream, by its handle 0 or beside another stream."""
import pytest

torch = pytest.importorskip("torch")

import adamw_hybrid_optimizer_muon_b200 as ma

pytestmark = pytest.mark.gpu

LATER = 200_000_000  # cycles: about 0.1 s


def test_ids_copied_for_the_default_stream_are_read_there():
    # ids that are not contiguous are copied, behind what the default stream still has to do
    table = torch.arange(100, device="cuda", dtype=torch.float32)[:, None].repeat(1, 8)
    ids, dy = torch.zeros(64, dtype=torch.int64, device="cuda"), torch.ones((32, 8), device="cuda")
    grad = torch.zeros((100, 8), device="cuda")
    new = torch.arange(64, device="cuda") + 30
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(LATER)
    ids.copy_(new)
    with torch.cuda.stream(side):
        out = ma.embedding_lookup(ids[::2], table, stream=0)
        ma.embedding_grad(ids[::2], dy, grad, stream=0)
    torch.cuda.synchronize()
    assert torch.equal(out[:, 0], new[::2].float())
    assert torch.equal(grad[:, 0].nonzero()[:, 0], new[::2])


@pytest.mark.parametrize("first", ["default", "side"])
def test_sums_on_the_default_stream_and_another(first):
    V, D, n = 20000, 1024, 30000
    table, grad = torch.zeros((V, D), device="cuda", requires_grad=True), torch.zeros((V, D), device="cuda")
    ids = [torch.randint(0, V, (n,), device="cuda") for _ in range(2)]
    want = sum(torch.bincount(x, minlength=V) for x in ids).float()[:, None].expand(V, D)
    here, side = torch.cuda.current_stream(), torch.cuda.Stream()
    assert here.cuda_stream == 0
    for _ in range(8):
        grad.zero_()
        side.wait_stream(here)
        outs = []
        for x, s in zip(ids, (here, side) if first == "default" else (side, here)):
            with torch.cuda.stream(s):
                outs.append(ma.embedding(x, table, grad=grad).sum())
        here.wait_stream(side)
        sum(outs).backward()
        assert torch.equal(grad, want)
    assert ma.ma_device_status() == ma.MA_OK


def test_host_copies_on_the_default_stream_are_done_when_it_says_so():
    p = torch.ones(4096, device="cuda")
    opt = ma.MuonAdamW([(p, ma.ROLE_HIDDEN, 0)], [("adamw", ma.adamw_hparams())])
    host, dev = torch.ones(4096).pin_memory(), torch.zeros(4096, device="cuda")
    opt.step_from_host([host], [dev], copy_stream=0)
    torch.cuda.synchronize()
    torch.cuda._sleep(LATER)
    opt.step_from_host([host], [dev], copy_stream=0)
    assert not opt.host_copies_done.query()
    opt.host_copies_done.synchronize()
    assert torch.equal(dev.cpu(), host)
    torch.cuda.synchronize()
    assert ma.ma_device_status() == ma.MA_OK
