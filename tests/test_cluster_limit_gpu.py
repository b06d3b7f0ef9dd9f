"""The adapter and activation-gradient launches of few rows where no cluster of 16 CTAs fits on the device: narrower ones give
the same results up to the order of the sums."""
import pytest
import torch

from lora_util import DT, lora_case
from test_dgrad_gpu import check as check_dgrad
from test_lora_gpu import check_apply, check_grad, forward_v, qg  # noqa: F401  (qg: the fixture)

pytestmark = pytest.mark.gpu


@pytest.fixture(params=[1, 2, 4, 8, 16])
def limit(qg, request):
    before = qg.qg_test_cluster_limit(request.param)
    yield request.param
    qg.qg_test_cluster_limit(before)


@pytest.mark.parametrize("x,w", [("bf16", "bf16"), ("f16", "f16"), ("f32", "f16")])
def test_adapters(qg, limit, x, w):
    for lens, ids in (([1], [1]), ([3, 0, 17], [0, 1, -1])):
        c = lora_case(lens, ids, na=2, r=24, N=9000, K=8192, x=x, w=w, seed=71)
        check_apply(qg, c, c["Yin"].to(DT[x]), DT[x])
        check_grad(qg, c, forward_v(c), c["dXin"], torch.float32)


@pytest.mark.parametrize("x", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M,N,K", [(1, 8192, 256), (77, 4100, 128), (128, 5000, 512)])
def test_activation_gradient(qg, limit, x, M, N, K):
    check_dgrad(qg, M, N, K, "u4", "tensor", x=x, seed=72)
    check_dgrad(qg, M, N, K, "nf4", x=x, seed=73)


def test_limits_that_are_refused(qg):
    for widest in (0, -1, 3, 32):
        with pytest.raises(ValueError):
            qg.qg_test_cluster_limit(widest)
    assert qg.qg_test_cluster_limit(16) == 16
