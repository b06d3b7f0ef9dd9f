"""Log probabilities at any temperature that the call takes: logits that are ruled out, and rows of odd widths (what fills their last vectors
counts for nothing), against fp64."""
import math

import pytest
import torch

from test_token_logprobs_gpu import DT, call, check, logits

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("x", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,V", [(1, 100352), (6, 1003), (330, 5003)])
@pytest.mark.parametrize("inv_t", [1e-2, 1.5e-3, 1.2e-3, 1e-3, 2e-4, 1e-4, 1e-5, 1e-6, 1e-12, 1e-30, 3e-37, 1e-38, 1e-45])
def test_high_temperatures(x, T, V, inv_t):
    X, target = logits(T, V, x, seed=V, shift=1)
    g = torch.Generator(device="cuda").manual_seed(T)
    out = torch.rand(T, V, generator=g, device="cuda") < 0.9
    out[T // 2] = False            # a row without a mask
    out[:, 5] = False
    X.masked_fill_(out, -math.inf)
    X[T - 1, 7] = 16000.0          # far above the others
    target[:] = 5
    check(X, target, inv_t, 6, call(X, target, inv_t, 6))


@pytest.mark.parametrize("x", ["f32", "bf16"])
@pytest.mark.parametrize("T", [1, 330])
@pytest.mark.parametrize("inv_t", [1e6, 1e34, 1e36, 2e36, 2e38])
def test_low_temperatures(x, T, inv_t):
    """Logits that are as small as the factor is large."""
    X, target = logits(T, 2005, "f32", seed=T)
    X = (X / inv_t).to(DT[x])
    X[:, ::3] = -math.inf
    target = target.clamp(max=2003) // 3 * 3 + 1
    check(X, target, inv_t, 6, call(X, target, inv_t, 6))


@pytest.mark.parametrize("x", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("largest", [60.0, 0.0, 2.0 ** -13])
@pytest.mark.parametrize("inv_t", [3e5, 1e8, 2e9, 1e12, 1e20, 2.2e38])
def test_nearly_no_temperature(x, inv_t, largest):
    """The largest logits share the probability, the others have none."""
    X, target = logits(5, 3001, x, seed=1)
    X -= 100
    X[:, 1::2] = -math.inf
    X[:, 40] = X[:, 3000] = largest
    X[2, 40] = -math.inf
    target[:] = 3000
    got = call(X, target, inv_t, 1)
    two = torch.tensor([2.0, 2.0, 1.0, 2.0, 2.0], device="cuda").log()
    assert torch.equal(got[3][:, 0].cpu(), torch.tensor([40, 40, 3000, 40, 40]))
    # the logarithm of two and nothing else
    assert ((got[0] + two).abs() <= 2.0 ** -22).all() and ((got[1] - two).abs() <= 2.0 ** -22).all() and ((got[4][:, 0] + two).abs() <= 2.0 ** -22).all()
