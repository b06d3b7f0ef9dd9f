"""The fine-tuning example end to end: the loss falls, the gradients agree with autograd over the dequantized weights,
and requests served together get what each gets alone."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ex():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gemm_blockwise_dequant_gb300 import build

    build.build()
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import qlora

    return qlora


def test_training_and_serving(ex):
    net = ex.Network()
    losses, norms = ex.train(net)
    assert losses[-1] < 0.7 * losses[0] and all(n > 0 for n in norms)
    together, alone = ex.serve(net)
    # the same sums in another split of the batch: both rounded to bf16 along the way
    assert float((together.float() - alone.float()).abs().max()) <= 2.0 ** -6 * float(alone.float().abs().max())


def test_gradients_against_autograd(ex):
    import gemm_blockwise_dequant_gb300 as qg

    net = ex.Network(hidden=128, inner=192, seed=3)
    g = torch.Generator(device="cuda").manual_seed(4)
    for layer in (net.up, net.down):
        layer.B.data.copy_((torch.randn(layer.B.shape, generator=g, device="cuda") * 0.05).bfloat16())
    offsets, ids = ex.requests([30, 0, 17, 9], [1, 0, 0, -1])
    X = torch.randn(56, 128, generator=g, device="cuda").bfloat16().requires_grad_()
    R = torch.randn(56, 128, generator=g, device="cuda")
    got = torch.autograd.grad((net(X, offsets, ids).float() * R).sum(), [X] + net.parameters())

    def dense(layer):
        N, K = layer.W.shape[0], layer.W.shape[1] * 2
        w = torch.empty(N, K, device="cuda")
        qg.qg_dequant_codebook4(layer.W, layer.codebook, layer.absmax, w, block_size=ex.BLOCK)
        return w.double()

    x = X.detach().double().requires_grad_()
    params = [p.detach().double().requires_grad_() for p in net.parameters()]

    def apply(h, w, A, B):
        outs = []
        for i, a in enumerate(ids.tolist()):
            t = h[offsets[i]:offsets[i + 1]]
            y = t @ w.t()
            outs.append(y + 2.0 * (t @ A[a].t()) @ B[a].t() if a >= 0 else y)
        return torch.cat(outs)

    h = torch.nn.functional.silu(apply(x, dense(net.up), params[0], params[1]))
    want = torch.autograd.grad((apply(h, dense(net.down), params[2], params[3]) * R.double()).sum(), [x] + params)
    for a, b in zip(got, want):  # a handful of roundings to bf16 (2^-8 each) on the way through both layers
        assert float((a.double() - b).norm()) <= 6 * 2.0 ** -8 * float(b.norm())
