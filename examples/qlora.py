"""Fine-tuning and serving of low-rank adapters over a frozen 4-bit model, on one GPU.

A two-layer network keeps its weights as 4-bit codes into a codebook times a block absmax.  A training step runs

    forward    qgemm_codebook4 (shared projection, fp32 out) and qg_lora_apply beside it
    backward   qgemm_codebook4_dgrad (through the frozen weight) and qg_lora_grad
    clipping   qg_clip_grad_norm over all adapters' gradients, before a plain gradient step

and the serving step pushes requests with different adapters (and one without) through the same network at once.

    python examples/qlora.py            # prints the loss of every step and checks the served rows
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import gemm_blockwise_dequant_gb300 as qg  # noqa: E402
from workloads import nf4_codebook  # noqa: E402

BLOCK = 64


def quantize(w, codebook):
    """[N, K] values to packed 4-bit codes [N, K/2] and the absmax of every 64 of them [N, K/64]."""
    N, K = w.shape
    blocks = w.float().reshape(N, K // BLOCK, BLOCK)
    absmax = blocks.abs().amax(dim=2)
    codes = ((blocks / absmax[:, :, None])[..., None] - codebook).abs().argmin(dim=-1).reshape(N, K).to(torch.uint8)
    return (codes[:, 0::2] | (codes[:, 1::2] << 4)).contiguous(), absmax.contiguous()


class Adapted(torch.autograd.Function):
    """Y = X . W^T + scaling (X A^T) B^T with W frozen and quantized; gradients of X, A and B."""

    @staticmethod
    def forward(ctx, X, A, B, layer, offsets, ids):
        base = torch.empty(X.shape[0], B.shape[1], device=X.device)  # fp32: the sum below is rounded once
        qg.qgemm_codebook4(X, layer.W, layer.codebook, layer.absmax, base, block_size=BLOCK)
        Y = torch.empty_like(base, dtype=X.dtype)
        V = torch.empty(X.shape[0], A.shape[1], device=X.device)
        qg.qg_lora_apply(X, offsets, ids, A, B, layer.scaling, base, Y, V=V)
        ctx.save_for_backward(X, A, B, V, offsets, ids)
        ctx.layer = layer
        return Y

    @staticmethod
    def backward(ctx, dY):
        X, A, B, V, offsets, ids = ctx.saved_tensors
        layer, dY = ctx.layer, dY.contiguous()
        dX, dA, dB = torch.empty_like(X), torch.empty_like(A), torch.empty_like(B)
        qg.qgemm_codebook4_dgrad(dY, layer.W, layer.codebook, layer.absmax, dX, block_size=BLOCK)
        qg.qg_lora_grad(dY, X, V, offsets, ids, A, B, layer.scaling, dX, dX, dA, dB)
        return dX, dA, dB, None, None, None


class Layer:
    """A quantized projection [N, K] and `adapters` adapters of rank `rank` for it."""

    def __init__(self, N, K, adapters, rank, codebook, generator):
        rnd = lambda *s: torch.randn(*s, generator=generator, device="cuda")
        self.codebook = codebook
        self.W, self.absmax = quantize(rnd(N, K) * K ** -0.5, codebook)
        self.A = (rnd(adapters, rank, K) * K ** -0.5).bfloat16().requires_grad_()
        self.B = torch.zeros(adapters, N, rank, dtype=torch.bfloat16, device="cuda").requires_grad_()
        self.scaling = torch.full((adapters,), 2.0, device="cuda")

    def __call__(self, X, offsets, ids):
        return Adapted.apply(X, self.A, self.B, self, offsets, ids)


class Network:
    def __init__(self, hidden=256, inner=512, adapters=2, rank=8, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        codebook = torch.from_numpy(nf4_codebook()).cuda()
        self.up = Layer(inner, hidden, adapters, rank, codebook, g)
        self.down = Layer(hidden, inner, adapters, rank, codebook, g)

    def __call__(self, X, offsets, ids):
        return self.down(torch.nn.functional.silu(self.up(X, offsets, ids)), offsets, ids)

    def parameters(self):
        return [self.up.A, self.up.B, self.down.A, self.down.B]


def requests(lengths, adapters):
    """Device offsets of the requests' rows and their adapters (-1: none)."""
    offsets = torch.zeros(len(lengths) + 1, dtype=torch.int64)
    offsets[1:] = torch.tensor(lengths).cumsum(0)
    return offsets.cuda(), torch.tensor(adapters, dtype=torch.int32, device="cuda")


def train(net, steps=40, lr=0.2, max_norm=1.0, seed=1):
    """Fits both adapters at once, each to a task of its own; returns the losses and the gradient norms."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    hidden = net.down.W.shape[0]
    lengths = [96, 160]  # the first request trains adapter 0, the second adapter 1
    offsets, ids = requests(lengths, [0, 1])
    X = torch.randn(sum(lengths), hidden, generator=g, device="cuda").bfloat16()
    left, right = (torch.randn(2, hidden, 4, generator=g, device="cuda") * hidden ** -0.5 for _ in range(2))
    tasks = 2.0 * left @ right.transpose(1, 2)  # what each task adds: four directions of its own
    with torch.no_grad():
        plain = net(X, offsets, torch.full_like(ids, -1)).float()
        target = torch.cat([plain[a:b] + X[a:b].float() @ tasks[i] for i, (a, b) in enumerate(((0, 96), (96, 256)))])
    norm, losses, norms = torch.empty(1, device="cuda"), [], []
    for _ in range(steps):
        loss = (net(X, offsets, ids).float() - target).square().sum(dim=1).mean()
        grads = list(torch.autograd.grad(loss, net.parameters()))
        qg.qg_clip_grad_norm(grads, max_norm, norm)
        with torch.no_grad():
            for p, d in zip(net.parameters(), grads):
                p -= lr * d
        losses.append(float(loss.detach()))
        norms.append(float(norm))
    return losses, norms


@torch.no_grad()
def serve(net, seed=2):
    """One decode step of six requests with adapters 0, 1 and none; returns what it gives and what each gives alone."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    adapters = [0, 1, -1, 1, 0, 1]
    X = torch.randn(len(adapters), net.down.W.shape[0], generator=g, device="cuda").bfloat16()
    together = net(X, *requests([1] * len(adapters), adapters))
    alone = torch.cat([net(X[i:i + 1], *requests([1], [a])) for i, a in enumerate(adapters)])
    return together, alone


def main():
    net = Network()
    losses, norms = train(net)
    for i, (loss, norm) in enumerate(zip(losses, norms)):
        print("step %2d  loss %.4f  gradient norm %.3f" % (i, loss, norm))
    together, alone = serve(net)
    print("served together and alone differ by at most %.3g of %.3g" % (float((together.float() - alone.float()).abs().max()), float(alone.abs().max())))
    return losses, together, alone


if __name__ == "__main__":
    main()
