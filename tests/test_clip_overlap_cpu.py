"""Steps refuse a clip buffer inside what they write. Nothing is launched: the addresses are made up."""
import ctypes

import pytest

import adamw_hybrid_optimizer_muon_b200 as ma

BASE = 0x6000_0000_0000
P, G, M, V = (BASE + k * 65536 for k in range(4))
FAR = BASE + (1 << 30)


def one(p):
    return (ctypes.c_void_p * 1)(p)


def adamw(clip):
    return ma.lib().adamw_step_fused_clipped(1, one(P), one(G), 0, one(M), one(V), (ctypes.c_int64 * 1)(1024),
                                             ctypes.byref(ma.adamw_hparams()), clip, None)


def muon(clip):
    return ma.lib().muon_step_batched_clipped(1, 32, 32, one(P), one(G), 0, one(M), ctypes.byref(ma.muon_hparams()), clip,
                                              None, 0, None)


@pytest.mark.parametrize("clip", [P, P + 256, P + 4096 - 256, M, V + 512])
def test_adamw_refuses(clip):
    assert adamw(clip) == ma.MA_ERR_ARG


@pytest.mark.parametrize("clip", [P, P + 256, P + 4096 - 256, M])
def test_muon_refuses(clip):
    assert muon(clip) == ma.MA_ERR_ARG


def test_one_beside_them_is_not_refused_for_that():
    # the workspace is: the check after this one (a call of adamw_step_fused_clipped would be launched)
    for clip in (P + 4096, FAR, None):
        assert muon(clip) == ma.MA_ERR_WORKSPACE


WS = BASE + (1 << 29)


def test_muon_refuses_one_in_its_workspace():
    need = ma.muon_workspace_bytes(1, 32, 32, ma.muon_hparams())
    call = lambda clip: ma.lib().muon_step_batched_clipped(  # noqa: E731
        1, 32, 32, one(P), one(G), 0, one(M), ctypes.byref(ma.muon_hparams()), clip, WS, need, None)
    for clip in (WS, WS + need // 256 * 256 - 256):
        assert call(clip) == ma.MA_ERR_ARG


def test_a_plan_refuses_one_in_its_workspace():
    t = ma.Tensor()
    t.param, t.grad, t.state0, t.ndim, t.role = P, G, M, 2, ma.ROLE_HIDDEN
    t.shape[0], t.shape[1] = 32, 32
    groups = ma.group_table([("muon", ma.muon_hparams())])
    plan, need = ma.ma_plan_create([t], groups)
    arr = (ma.Group * 1)(*groups)
    try:
        for measure, clip in ((1, WS), (1, WS - 256), (0, WS), (1, WS + need // 256 * 256 - 256)):
            assert ma.lib().ma_plan_set_clip(plan, measure, 1.0, 1.0, clip) == ma.MA_OK
            for fn in ("muonadamw_step", "muonadamw_step_graph"):
                assert getattr(ma.lib(), fn)(plan, arr, WS, need, None) == ma.MA_ERR_ARG
    finally:
        ma.ma_plan_destroy(plan)
