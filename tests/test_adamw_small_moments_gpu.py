"""Second moments that are hardly above zero, and an eps of no help: the quotient is that of fp32 operations."""
import pytest
import torch

import gemm_blockwise_dequant_gb300 as qg
from test_adamw_gpu import BETAS, LR

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("state", ["f32", "e4m3"])
@pytest.mark.parametrize("eps", [0.0, 1e-22])
def test_small_gradients(state, eps):
    # blocks of one magnitude each, from 1 to where (1 - beta2) g^2 has a bit or two
    size = 2.0 ** -torch.arange(0, 69, device="cuda").float().repeat_interleave(256)
    g = size * torch.where(torch.rand(size.numel(), generator=torch.Generator(device="cuda").manual_seed(4), device="cuda") < 0.5, -1.0, 1.0)
    p = torch.zeros_like(g)
    t = qg.QGAdamWList([p], [g], state=state)
    qg.qg_adamw_step(t, lr=LR, step=1, betas=BETAS, eps=eps)
    v = (1 - BETAS[1]) * g.square()
    assert (v > 0).all() and (v < 2.0 ** -126).any()
    want = -LR * g.double() / ((v.double() / (1 - BETAS[1])).sqrt() + eps)
    # the root, both bias corrections, a reciprocal and four products: eight roundings and the approximations' units
    assert ((p.double() - want).abs() <= 2.0 ** -20 * want.abs()).all()
    if state == "f32":
        assert torch.equal(t.exp_avg_sq[0], v)


def test_a_second_moment_below_zero_has_no_root():
    """Of a state that something spoiled: it shows in its own parameter and nowhere else."""
    g, m, v = torch.zeros(5000, device="cuda"), torch.full((5000,), 1e-3, device="cuda"), torch.full((5000,), 1e-6, device="cuda")
    v[7], v[4999], v[2000] = -1e-6, -1e-30, -0.0
    p = torch.ones(5000, device="cuda")
    t = qg.QGAdamWList([p], [g], exp_avg=[m], exp_avg_sq=[v])
    qg.qg_adamw_step(t, lr=LR, step=1, betas=BETAS)
    assert p.isnan().nonzero().flatten().tolist() == [7, 4999]
    assert float(p[2000]) < -1  # m' over eps
