"""Norms of gradients with many zeros: those of tensors that nothing reached, beside values whose squares are below fp32's range or above it."""
import math

import pytest
import torch

import gemm_blockwise_dequant_gb300 as qg

pytestmark = pytest.mark.gpu


def norm_of(grads):
    t = qg.QGAdamWList([torch.zeros_like(g) for g in grads], grads)
    norm = torch.full((1,), -1.0, device="cuda")
    qg.qg_adamw_step(t, lr=1e-3, step=1, max_norm=1.0, norm=norm)
    return float(norm)


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("value", [1e-3, 6e-8, 1e-22, 1e-30, 1e-38, 1e22, 3e38])
def test_zeros_among_values(dtype, shift, value):
    if dtype == torch.float16 and not 6e-8 <= value <= 1:
        pytest.skip("no value of the type")
    room = torch.zeros(70_000 + shift, dtype=dtype, device="cuda")
    g = room[shift:]
    g[::2].fill_(-0.0)
    assert norm_of([g, torch.zeros(5000, dtype=dtype, device="cuda")]) == 0
    g[torch.tensor([3, 4095, 4096, 20_000, 69_999], device="cuda")] = value
    g[40_000:40_008] = -value
    # sums of eight squares in fp32, the rest in fp64
    assert abs(norm_of([g]) / (float(g[3]) * math.sqrt(13)) - 1) <= 2.0 ** -21 or value == 3e38 and math.isinf(norm_of([g]))
    if value == 1e22:  # beside each other
        g[8:16] = 1e-30
        assert abs(norm_of([g]) / (float(g[3]) * math.sqrt(13)) - 1) <= 2.0 ** -21


@pytest.mark.parametrize("bad", [math.inf, math.nan])
def test_what_is_not_finite_among_zeros(bad):
    g = torch.zeros(70_000, device="cuda")
    g[60_000] = bad
    assert not math.isfinite(norm_of([g]))
