"""Clip buffers that a kernel would write or read beyond, or that are not on the GPU, are refused before the library is
called. Nothing is launched: the library is a stand-in that fails the test when it is reached."""
import pytest
import torch

import adamw_hybrid_optimizer_muon_b200 as ma


class Unreached:
    def __getattr__(self, name):
        raise AssertionError(f"{name} was called")


@pytest.fixture
def no_library(monkeypatch):
    monkeypatch.setattr(ma, "lib", Unreached)
    monkeypatch.setattr(ma, "_lib_status_string", str)  # (the error's text comes from the library)


@pytest.fixture
def as_if_on_gpu(monkeypatch):
    """Host tensors pass for tensors of the current GPU, so that the checks after that one are reached."""
    monkeypatch.setattr(ma, "_on_current_gpu", lambda what, *tensors: None)
    monkeypatch.setattr(ma, "_on_gpu", lambda what, *tensors: None, raising=False)


SHORT = [torch.empty(4), torch.empty(ma.CLIP_BYTES // 4 - 1), torch.empty(ma.CLIP_BYTES // 4, dtype=torch.bfloat16),
         torch.empty(1).expand(ma.CLIP_BYTES // 4), torch.empty(ma.CLIP_BYTES // 4, 2)[:, 0]]
FILL = [lambda c, g: ma.ma_grad_norm([g], c), lambda c, g: ma.ma_grad_clip([g], c, 1.0),
        lambda c, g: ma.ma_plan_set_clip(0x1000, c, 1.0)]
# these read or write the first 16 bytes alone
HEAD = [lambda c, g: ma.ma_clip_finalize(c, 1.0), lambda c, g: ma.ma_plan_set_clip(0x1000, c, measure=False),
        lambda c, g: ma.adamw_step_fused([g], [g], [g], [g], ma.adamw_hparams(), stream=0, clip=c),
        lambda c, g: ma.muon_step_batched([g], [g], [g], ma.muon_hparams(), None, stream=0, shape=(2, 4), clip=c)]


@pytest.mark.parametrize("call", FILL)
@pytest.mark.parametrize("clip", SHORT)
def test_short_buffers_are_not_filled(no_library, as_if_on_gpu, call, clip):
    with pytest.raises(ma.MAError) as e:
        call(clip, torch.zeros(8))
    assert e.value.code == ma.MA_ERR_WORKSPACE


@pytest.mark.parametrize("call", HEAD)
@pytest.mark.parametrize("clip", [torch.empty(0), torch.empty(3), torch.empty(1).expand(4)])
def test_buffers_without_a_head_are_not_read(no_library, as_if_on_gpu, call, clip):
    with pytest.raises(ma.MAError) as e:
        call(clip, torch.zeros(8))
    assert e.value.code == ma.MA_ERR_WORKSPACE


@pytest.mark.parametrize("call", FILL + HEAD)
def test_host_buffers_are_refused(no_library, call):
    with pytest.raises(ma.MAError) as e:
        call(torch.zeros(ma.CLIP_BYTES // 4), torch.zeros(8))
    assert e.value.code == ma.MA_ERR_ARG


@pytest.mark.parametrize("call", HEAD[2:])
def test_whole_buffers_reach_the_library(no_library, as_if_on_gpu, call):
    with pytest.raises(AssertionError, match="was called"):
        call(torch.zeros(ma.CLIP_BYTES // 4), torch.zeros(8))
