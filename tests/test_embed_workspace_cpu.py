"""The workspace given to embedding_grad: its bytes have to be there. Nothing is launched."""
import pytest
import torch

import adamw_hybrid_optimizer_muon_b200 as ma


class Unreached:
    def __getattr__(self, name):
        raise AssertionError(f"{name} was called")


@pytest.mark.parametrize("ws", [torch.empty(1, dtype=torch.uint8).expand(1 << 24),
                                torch.empty((1 << 12, 2), dtype=torch.uint8)[:, :1]])
def test_a_workspace_that_is_not_contiguous_is_refused(monkeypatch, ws):
    # by its element count the first has 16 MB, and one byte of memory
    monkeypatch.setattr(ma, "_on_current_gpu", lambda what, *tensors: None)
    monkeypatch.setattr(ma, "_lib_status_string", str)
    monkeypatch.setattr(ma, "lib", Unreached)
    ids, dy, grad = torch.zeros(4, dtype=torch.int64), torch.zeros(4, 8), torch.zeros(5, 8)
    with pytest.raises(ma.MAError) as e:
        ma.embedding_grad(ids, dy, grad, ws=ws, stream=0)
    assert e.value.code == ma.MA_ERR_WORKSPACE
