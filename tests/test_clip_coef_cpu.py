"""The sharded step's coefficient, beside its norm."""
import pytest
import torch

from adamw_hybrid_optimizer_muon_b200.dist import DistMuonAdamW


def test_the_sharded_step_gives_norm_and_coefficient():
    opt = object.__new__(DistMuonAdamW)
    opt._clip = None
    for name in ("grad_norm", "grad_coef"):
        with pytest.raises(RuntimeError):
            getattr(opt, name)
    opt._clip = torch.tensor([3.0, 0.25, 0.0, 0.0])
    assert float(opt.grad_norm) == 3.0 and float(opt.grad_coef) == 0.25
