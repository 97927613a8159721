"""QK-Clip on data-parallel replicas: with each rank's own maximum the weights part, with the reduced one they stay alike.

Gloo ranks; the kernel is replaced by its formula in fp64."""
import datetime
import socket

import numpy as np
import pytest
import torch
import torch.distributed as dist
import torch.multiprocessing as mp

HEADS, KV, ROWS, COLS, TAU = 6, 3, 4, 5, 10.0


def clip(wq, wk, top):
    """Factors of the query and of the key heads, as the header defines them (alpha 1/2)."""
    g = torch.where((top > TAU) & torch.isfinite(top), TAU / top, torch.ones_like(top))
    fk = g.view(KV, -1).amin(1).sqrt()
    fq = g / fk.repeat_interleave(HEADS // KV)
    return wq * fq.repeat_interleave(ROWS)[:, None], wk * fk.repeat_interleave(ROWS)[:, None]


def rank_main(rank, world, port, q):
    dist.init_process_group("gloo", init_method=f"tcp://127.0.0.1:{port}", rank=rank, world_size=world,
                            timeout=datetime.timedelta(seconds=60))
    g = torch.Generator().manual_seed(3)
    wq = torch.randn((HEADS * ROWS, COLS), generator=g, dtype=torch.float64)
    wk = torch.randn((KV * ROWS, COLS), generator=g, dtype=torch.float64)
    top = torch.tensor([4.0, 9.0 + 8 * rank, 30.0, 50.0, float("inf") if rank else 2.0, 40.0 - 25 * rank])
    own = clip(wq, wk, top.double())
    dist.all_reduce(top, dist.ReduceOp.MAX)
    q.put((rank, [w.numpy() for w in own], [w.numpy() for w in clip(wq, wk, top.double())], top.numpy()))
    dist.barrier()
    dist.destroy_process_group()


@pytest.mark.parametrize("world", [2, 3])
def test_replicas_stay_alike_with_the_reduced_maximum(world):
    with socket.socket() as s:
        s.bind(("127.0.0.1", 0))
        port = s.getsockname()[1]
    ctx = mp.get_context("spawn")
    q = ctx.Queue()
    ps = [ctx.Process(target=rank_main, args=(r, world, port, q)) for r in range(world)]
    for p in ps:
        p.start()
    got = sorted(q.get(timeout=120) for _ in ps)
    for p in ps:
        p.join(timeout=60)
        assert p.exitcode == 0
    for rank, own, shared, top in got[1:]:
        assert not np.array_equal(own[0], got[0][1][0])  # each by its own batch: they part
        for a, b in zip(shared, got[0][2]):
            assert np.array_equal(a, b)
        assert np.array_equal(top, got[0][3])
    # head 0 is within TAU and shares its keys with head 1: its query weights make up for them
    wq, wk = got[0][2]
    g = torch.Generator().manual_seed(3)
    w0 = torch.randn((HEADS * ROWS, COLS), generator=g, dtype=torch.float64).numpy()
    k0 = torch.randn((KV * ROWS, COLS), generator=g, dtype=torch.float64).numpy()
    s0, s1 = w0[:ROWS] @ k0[:ROWS].T, wq[:ROWS] @ wk[:ROWS].T
    assert not np.array_equal(wq[:ROWS], w0[:ROWS]) and np.allclose(s0, s1, rtol=1e-12, atol=1e-12)
