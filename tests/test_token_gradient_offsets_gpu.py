"""The gradient of logits far from zero: exact for the lse that it is given, and off by no more than that lse's rounding to fp32."""
import pytest
import torch

import gemm_blockwise_dequant_gb300 as qg
from test_token_logprobs_gpu import DT, UNIT, call, logits, score64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("x", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("offset", [-60000.0, -300.0, 300.0, 16384.0, 60000.0])
@pytest.mark.parametrize("inv_t", [0.01, 1.0, 50.0])
def test_rows_far_from_zero(x, offset, inv_t):
    T, V = 5, 3001
    X, target = logits(T, V, "f32", seed=7)
    X = (X + offset).to(DT[x])
    g = torch.Generator(device="cuda").manual_seed(1)
    d, h = torch.randn(T, generator=g, device="cuda"), torch.randn(T, generator=g, device="cuda")
    lp, entropy, lse, _, _ = call(X, target, inv_t)
    dX = torch.empty_like(X)
    qg.qg_token_logprobs_grad(X, target, lse, d, dX, entropy=entropy, d_entropy=h, inv_temperature=inv_t)
    hot = torch.nn.functional.one_hot(target, V)
    dd, hh = d.double()[:, None], h.double()[:, None]

    def near(logp, entropy, more):
        p = logp.exp()
        want = inv_t * (dd * (hot - p) - hh * p * (logp + entropy[:, None]))
        # p: the rounding of z - lse (not of their magnitudes) and the exponential; then one rounding to the type
        size = inv_t * p * (dd.abs() + hh.abs() * (logp.abs() + entropy.abs()[:, None] + 1))
        off = size * (2.0 ** -20 + 2.0 ** -22 * logp.abs() + more) + UNIT[DT[x]] * 1.01 * want.abs() + 2.0 ** -23 * inv_t * dd.abs() + (2.0 ** -25 if x == "f16" else 1e-36)
        return ((dX.double() - want).abs() <= off).all()

    assert near(X.double() * inv_t - lse.double()[:, None], entropy.double(), 0.0)
    _, entropy64, lse64, logp = score64(X, target, inv_t)
    # the forward pass's lse and entropy are off by a rounding of the value and 2^-18
    far = torch.expm1(1.01 * (2.0 ** -24 * lse64.abs() + 2.0 ** -18))[:, None]
    assert near(logp, entropy64, 2 * far)
