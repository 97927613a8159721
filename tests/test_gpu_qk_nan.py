"""The maximum with what is there already: a NaN of either sign stays one, whatever the call adds to it."""
import math

import pytest

torch = pytest.importorskip("torch")

import adamw_hybrid_optimizer_muon_b200 as ma

pytestmark = pytest.mark.gpu

NANS = [0x7FC00000, -0x400000, 0x7FFFFFFF, -1, 0x7F800001, -0x7FFFFF]  # quiet and signalling, positive and negative


@pytest.mark.parametrize("absolute", [False, True])
@pytest.mark.parametrize("T", [1, 300, 2000])
def test_a_nan_that_is_there_stays(T, absolute):
    H, D = len(NANS) + 3, 64
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    q = torch.randn((2, T, H, D), generator=g, device="cuda").bfloat16()
    k = torch.randn((2, T, H, D), generator=g, device="cuda").bfloat16()
    q[:, :, 1::2] = -q[:, :, 1::2].abs()  # and heads whose logits are all negative
    k[:, :, 1::2] = k[:, :, 1::2].abs()
    fresh = ma.qk_max_logit(q, k, absolute=absolute)
    assert absolute or bool((fresh[1::2] < 0).all())
    out = torch.empty(H, device="cuda")
    out.view(torch.int32).copy_(torch.tensor(NANS + [0, 0, 0], dtype=torch.int32))
    out[len(NANS):] = torch.tensor([-math.inf, 1e30, -1e30])
    before = out.clone()
    got = ma.qk_max_logit(q, k, absolute=absolute, out=out, accumulate=True)
    n = len(NANS)
    assert bool(torch.isnan(before[:n]).all()) and bool(torch.isnan(got[:n]).all()), got
    assert torch.equal(got[n:], torch.maximum(before[n:], fresh[n:]))
    again = ma.qk_max_logit(q, k, absolute=absolute, out=out, accumulate=True)
    assert bool(torch.isnan(again[:n]).all()) and torch.equal(again[n:], got[n:])
    assert ma.ma_device_status() == ma.MA_OK
