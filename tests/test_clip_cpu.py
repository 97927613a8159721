"""Gradient norm and clipping: argument checks (before anything is launched) and the sharded step's norm on gloo ranks.

The refusals need no GPU: a call with bad arguments returns its status before
it looks for a device, so the pointers here are made up and never followed.
On CPU ranks the library's kernels are replaced by the formula in fp64; what is
tested is the exchange: which rank sums what, and that every rank gets the same
norm and coefficient, for the averaged gradients.
"""
import ctypes
import datetime
import math
import os
import socket

import numpy as np
import pytest
import torch
import torch.distributed as dist
import torch.multiprocessing as mp

import adamw_hybrid_optimizer_muon_b200 as ma

CLIP = 0x7000_0000_0000  # a made-up device address, 256-byte aligned
G0 = 0x6000_0000_0000


def _call(fn, n, ptrs, gdt, numel, scale=1.0, max_norm=1.0, clip=CLIP):
    arr = (ctypes.c_void_p * max(1, len(ptrs)))(*ptrs) if ptrs is not None else None
    dts = (ctypes.c_int32 * max(1, len(gdt)))(*gdt) if gdt is not None else None
    num = (ctypes.c_int64 * max(1, len(numel)))(*numel) if numel is not None else None
    return getattr(ma.lib(), fn)(n, arr, dts, num, scale, max_norm, clip, None)


BAD = [
    (dict(n=-1, ptrs=[G0], gdt=[0], numel=[4]), ma.MA_ERR_SHAPE),
    (dict(n=1, ptrs=None, gdt=[0], numel=[4]), ma.MA_ERR_NULL),
    (dict(n=1, ptrs=[G0], gdt=None, numel=[4]), ma.MA_ERR_NULL),
    (dict(n=1, ptrs=[G0], gdt=[0], numel=None), ma.MA_ERR_NULL),
    (dict(n=1, ptrs=[None], gdt=[0], numel=[4]), ma.MA_ERR_NULL),
    (dict(n=1, ptrs=[G0], gdt=[2], numel=[4]), ma.MA_ERR_DTYPE),
    (dict(n=1, ptrs=[G0], gdt=[0], numel=[-4]), ma.MA_ERR_SHAPE),
    (dict(n=1, ptrs=[G0], gdt=[0], numel=[(1 << 50) + 1]), ma.MA_ERR_SHAPE),
    (dict(n=1, ptrs=[G0 + 2], gdt=[0], numel=[4]), ma.MA_ERR_ALIGN),
    (dict(n=1, ptrs=[G0 + 1], gdt=[1], numel=[4]), ma.MA_ERR_ALIGN),
    (dict(n=1, ptrs=[G0], gdt=[0], numel=[4], clip=None), ma.MA_ERR_NULL),
    (dict(n=1, ptrs=[G0], gdt=[0], numel=[4], clip=CLIP + 16), ma.MA_ERR_ALIGN),
    (dict(n=1, ptrs=[CLIP + 256], gdt=[0], numel=[4]), ma.MA_ERR_ARG),  # a gradient inside the clip buffer
    (dict(n=1, ptrs=[CLIP - 8], gdt=[0], numel=[4]), ma.MA_ERR_ARG),
    (dict(n=1, ptrs=[G0], gdt=[0], numel=[4], scale=0.0), ma.MA_ERR_ARG),
    (dict(n=1, ptrs=[G0], gdt=[0], numel=[4], scale=-1.0), ma.MA_ERR_ARG),
    (dict(n=1, ptrs=[G0], gdt=[0], numel=[4], scale=math.inf), ma.MA_ERR_ARG),
    (dict(n=1, ptrs=[G0], gdt=[0], numel=[4], scale=math.nan), ma.MA_ERR_ARG),
    (dict(n=1, ptrs=[G0], gdt=[0], numel=[4], max_norm=-1.0), ma.MA_ERR_ARG),
    (dict(n=1, ptrs=[G0], gdt=[0], numel=[4], max_norm=math.nan), ma.MA_ERR_ARG),
]


@pytest.mark.parametrize("kw,code", BAD)
@pytest.mark.parametrize("fn", ["ma_grad_norm", "ma_grad_clip"])
def test_bad_arguments_are_refused(fn, kw, code):
    assert _call(fn, **kw) == code


def test_in_place_clipping_refuses_overlapping_gradients():
    kw = dict(n=2, ptrs=[G0, G0 + 8], gdt=[0, 0], numel=[4, 4])
    assert _call("ma_grad_clip", **kw) == ma.MA_ERR_ARG
    assert _call("ma_grad_clip", n=2, ptrs=[G0, G0], gdt=[1, 1], numel=[4, 4]) == ma.MA_ERR_ARG


def test_finalize_and_plan_arguments():
    L = ma.lib()
    assert L.ma_clip_finalize(1.0, -1.0, CLIP, None) == ma.MA_ERR_ARG
    assert L.ma_clip_finalize(1.0, 1.0, None, None) == ma.MA_ERR_NULL
    assert L.ma_clip_finalize(1.0, 1.0, CLIP + 8, None) == ma.MA_ERR_ALIGN
    assert L.ma_plan_set_clip(None, 1, 1.0, 1.0, CLIP) == ma.MA_ERR_NULL
    t = ma.Tensor()
    t.param, t.grad, t.state0, t.state1 = G0, G0 + 4096, G0 + 8192, G0 + 12288
    t.ndim, t.shape[0], t.role = 1, 1024, ma.ROLE_HIDDEN
    plan, _ = ma.ma_plan_create([t], ma.group_table([("adamw", ma.adamw_hparams())]))
    try:
        assert L.ma_plan_set_clip(plan, 1, 1.0, 1.0, CLIP) == ma.MA_OK
        assert L.ma_plan_set_clip(plan, 0, 1.0, 1.0, CLIP) == ma.MA_OK
        assert L.ma_plan_set_clip(plan, 2, 1.0, 1.0, CLIP) == ma.MA_ERR_ARG
        assert L.ma_plan_set_clip(plan, 1, 0.0, 1.0, CLIP) == ma.MA_ERR_ARG
        assert L.ma_plan_set_clip(plan, 1, 1.0, math.nan, CLIP) == ma.MA_ERR_ARG
        assert L.ma_plan_set_clip(plan, 1, 1.0, 1.0, CLIP + 128) == ma.MA_ERR_ALIGN
        for p in (t.param, t.grad, t.state0, t.state1):  # on a buffer the step uses
            assert L.ma_plan_set_clip(plan, 1, 1.0, 1.0, p) == ma.MA_ERR_ARG
        assert L.ma_plan_set_clip(plan, 1, 1.0, 1.0, None) == ma.MA_OK
    finally:
        ma.ma_plan_destroy(plan)


def test_steps_refuse_a_misaligned_clip_buffer():
    one = (ctypes.c_void_p * 1)(G0)
    num = (ctypes.c_int64 * 1)(64)
    hp, mh = ma.adamw_hparams(), ma.muon_hparams()
    assert ma.lib().adamw_step_fused_clipped(1, one, one, 0, one, one, num, ctypes.byref(hp), CLIP + 4,
                                             None) == ma.MA_ERR_ALIGN
    two = (ctypes.c_void_p * 1)(G0 + 4096)
    assert ma.lib().muon_step_batched_clipped(1, 8, 8, one, one, 0, two, ctypes.byref(mh), CLIP + 4, None, 0,
                                              None) == ma.MA_ERR_ALIGN


def test_host_tensors_are_refused():
    g = torch.zeros(8)
    for call in (lambda: ma.GradClip([g]), lambda: ma.ma_grad_norm([g], torch.zeros(ma.CLIP_BYTES // 4)),
                 lambda: ma.ma_grad_clip([g], torch.zeros(ma.CLIP_BYTES // 4), 1.0),
                 lambda: ma.ma_clip_finalize(torch.zeros(ma.CLIP_BYTES // 4))):
        with pytest.raises(ma.MAError) as e:
            call()
        assert e.value.code == ma.MA_ERR_ARG


def test_clip_bytes_match_the_header():
    import re
    src = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include",
                            "muonadamw.h")).read()
    assert ma.CLIP_BYTES == int(re.search(r"#define MA_CLIP_BYTES (\d+)", src).group(1))


# ---------------------------------------------------------------------------- the sharded step's norm

TABLE = [((100, 64), ma.ROLE_EMBED, 1), ((48, 96), ma.ROLE_HIDDEN, 0), ((96, 40), ma.ROLE_HIDDEN, 0),
         ((48, 96), ma.ROLE_HIDDEN, 0), ((48, 96), ma.ROLE_HIDDEN, 0), ((7,), ma.ROLE_HIDDEN, 1),
         ((), ma.ROLE_HIDDEN, 1)]


def _grads(step, rank):
    return [np.asarray(np.random.default_rng([step, rank, i]).standard_normal(s) * 1e-2, np.float32)
            for i, (s, _, _) in enumerate(TABLE)]


def _worker(rank, world, port, q):
    os.environ["MASTER_ADDR"], os.environ["MASTER_PORT"] = "127.0.0.1", str(port)
    dist.init_process_group("gloo", rank=rank, world_size=world, timeout=datetime.timedelta(seconds=60))
    try:
        from adamw_hybrid_optimizer_muon_b200.dist import DistMuonAdamW

        class FormulaDist(DistMuonAdamW):
            seen = []

            def _local_sumsq(self):
                self._clip.view(torch.float64)[1] = sum(float((pc.grad.double() ** 2).sum()) for pc in self.pieces())

            def _finish_norm(self, max_norm, scale):
                root = float(self._clip.view(torch.float64)[1]) ** 0.5
                self._clip[0] = scale * root
                self._clip[1] = scale if scale * root <= max_norm else max_norm / root

            def _local_step(self, b):
                self.seen.append(float(self._clip[1]) if self._clipping else None)

        params = [torch.zeros(s) for s, _, _ in TABLE]
        opt = FormulaDist([(p, role, g) for p, (_, role, g) in zip(params, TABLE)],
                          [("muon", ma.muon_hparams()), ("adamw", ma.adamw_hparams())], seg_cap=2048)
        out = []
        for step, kw in ((1, dict(max_norm=0.01)), (2, dict(max_norm=1e6)), (3, dict(max_norm=0.01, grad_scale=0.25)),
                         (4, {})):
            for v, g in zip(opt.grads, _grads(step, rank)):
                v.copy_(torch.from_numpy(g))
            opt.seen.clear()
            opt.step(**kw)
            out.append((float(opt.grad_norm), list(opt.seen)))
        with pytest.raises(ValueError):
            opt.step(max_norm=-1.0)
        with pytest.raises(ValueError):
            opt.step(grad_scale=0.0)
        q.put((rank, (out, opt.step_count)))
    finally:
        dist.destroy_process_group()


@pytest.mark.parametrize("world", [2, 3])
def test_sharded_norm_is_that_of_the_averaged_gradients(world):
    ctx = mp.get_context("spawn")
    q = ctx.Queue()
    s = socket.socket()
    s.bind(("127.0.0.1", 0))
    port = s.getsockname()[1]
    s.close()
    procs = [ctx.Process(target=_worker, args=(r, world, port, q)) for r in range(world)]
    for p in procs:
        p.start()
    res = dict(q.get(timeout=300) for _ in range(world))
    for p in procs:
        p.join(60)
    assert all(p.exitcode == 0 for p in procs)
    for step, (max_norm, scale) in ((1, (0.01, 1.0)), (2, (1e6, 1.0)), (3, (0.01, 0.25))):
        avg = [sum(np.float64(g) for g in gs) / world for gs in zip(*(_grads(step, r) for r in range(world)))]
        root = math.sqrt(sum(float((a ** 2).sum()) for a in avg))
        coef = scale * min(1.0, max_norm / (scale * root))
        for r in range(world):
            norm, seen = res[r][0][step - 1]
            # the fp32 average is off by a few roundings (world additions and a division) of 2^-24 per value
            assert abs(norm - scale * root) <= (world + 2) * 2.0 ** -24 * scale * root
            assert seen and all(abs(c - coef) <= (world + 3) * 2.0 ** -24 * coef for c in seen)
            assert res[r][0][step - 1] == res[0][0][step - 1]  # the same on every rank, and in every bucket
    for r in range(world):
        assert all(c is None for c in res[r][0][3][1])  # a step without max_norm is not clipped
        assert res[r][1] == 4                           # refused calls are no steps
