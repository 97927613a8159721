"""GradClip on gradients whose memory was replaced. No GPU: host tensors, and a stand-in for the library that reads the
tables it is given."""
import ctypes

import pytest
import torch

import adamw_hybrid_optimizer_muon_b200 as ma


class Library:
    calls = []

    def ma_grad_norm(self, n, ptrs, gdt, numel, scale, max_norm, clip, stream):
        read = lambda a, t: list((t * n).from_address(a if isinstance(a, int) else ctypes.addressof(a)))  # noqa: E731
        self.calls.append((read(ptrs, ctypes.c_uint64), read(gdt, ctypes.c_int32), read(numel, ctypes.c_int64)))
        return 0

    def ma_grad_clip(self, *args):
        return self.ma_grad_norm(*args)


@pytest.fixture(params=["module", "methods"])
def calls(request, monkeypatch):
    if request.param == "methods":
        monkeypatch.setattr(ma, "_MARSHAL", ma._Methods)
    else:
        assert ma._marshal() is not ma._Methods
    monkeypatch.setattr(ma, "_on_current_gpu", lambda what, *tensors: None)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: -1)
    monkeypatch.setattr(ma, "clip_buffer", lambda device=None: torch.zeros(ma.CLIP_BYTES // 4))
    monkeypatch.setattr(ma, "lib", Library)
    monkeypatch.setattr(ma, "_lib_status_string", str)
    monkeypatch.setattr(Library, "calls", [])
    return Library.calls


def tables(grads):
    code = {torch.float32: ma.MA_F32, torch.bfloat16: ma.MA_BF16}
    return [g.data_ptr() for g in grads], [code[g.dtype] for g in grads], [g.numel() for g in grads]


def test_replaced_memory_is_seen(calls):
    grads = [torch.zeros(n) for n in (5, 1, 700)]
    clip = ma.GradClip(grads)
    clip.norm(stream=0)
    old = tables(grads)
    grads[1].data = torch.ones(9)                            # elsewhere, and of another size
    clip.norm(stream=0)
    grads[2].set_(torch.zeros(700))                          # elsewhere
    clip.clip(1.0, stream=0)
    grads[0].data = torch.zeros(5, dtype=torch.bfloat16)     # elsewhere, and of another type
    clip.norm(stream=0)
    assert calls[0] == old and calls[-1] == tables(grads)
    assert all(a[0] != b[0] for a, b in zip(calls, calls[1:]))
    grads[2].resize_(3)                                      # where it was, and shorter
    clip.norm(stream=0)
    assert calls[-1] == tables(grads)
    clip.norm(stream=0)
    assert calls[-1] == calls[-2]


def test_what_does_not_fit_any_more_is_refused(calls):
    grads = [torch.zeros(8), torch.zeros(8)]
    clip = ma.GradClip(grads)
    grads[1].data = torch.zeros((4, 4))[:, ::2]
    with pytest.raises(ma.MAError):
        clip.norm(stream=0)
    grads[1].data = torch.zeros(8, dtype=torch.float64)
    with pytest.raises(ma.MAError):
        clip.norm(stream=0)
    assert not calls


def test_no_gradients(calls):
    clip = ma.GradClip([])
    clip.norm(stream=0)
    assert calls == [([], [], [])]
