"""A step's coefficient tells whether its gradients were dropped; its norm, a float, is also infinite where it is beyond fp32."""
import math

import pytest

torch = pytest.importorskip("torch")

import adamw_hybrid_optimizer_muon_b200 as ma

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("graph", [False, True])
def test_a_norm_beyond_fp32_is_a_step_and_a_gradient_that_is_not_finite_is_none(graph):
    n, value, beta1 = 4096, 3e38, 0.5
    p, g = torch.ones(n, device="cuda"), torch.full((n,), value, device="cuda")
    opt = ma.MuonAdamW([(p, ma.ROLE_HIDDEN, 0)], [("adamw", ma.adamw_hparams(lr=0.01, beta1=beta1, weight_decay=0.0))])
    with pytest.raises(RuntimeError):
        opt.grad_coef
    opt.step([g], graph=graph, max_norm=1.0)
    want = 1 / (float(g[0]) * math.sqrt(n))
    assert math.isinf(float(opt.grad_norm))
    coef = float(opt.grad_coef)
    assert abs(coef - want) <= 2.0 ** -150 + want * 2.0 ** -23  # half a step of a subnormal number
    # exp_avg = (1 - beta1) * g * coef: three roundings
    m = opt.state[0][0].double()
    assert torch.all((m - (1 - beta1) * float(g[0]) * coef).abs() <= 4 * 2.0 ** -24 * m.abs())
    assert torch.all(p != 1)
    kept, m_kept = p.clone(), opt.state[0][0].clone()
    g[7] = math.inf
    opt.step([g], graph=graph, max_norm=1.0)
    assert math.isinf(float(opt.grad_norm)) and float(opt.grad_coef) == 0
    assert torch.equal(opt.state[0][0], m_kept * beta1)  # a step with zero gradients
    assert torch.all(torch.isfinite(p)) and not torch.equal(p, kept)
    g[7] = 1.0
    opt.step([g], graph=graph, grad_scale=0.25)
    assert float(opt.grad_coef) == 0.25
    assert ma.ma_device_status() == ma.MA_OK
