"""Fine-tuning calls one behind another on a stream, each reading what the one before wrote, with nothing waited for on the
host: every result is what the calls give one at a time."""
import pytest
import torch

from lora_util import DT, lora_case
from test_dgrad_gpu import run, weight
from test_lora_gpu import forward_v, qg  # noqa: F401  (qg: the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("x", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("sizes", [[300], [100000, 7, 4097], [3000000, 12345]])
def test_clipping_in_place(qg, x, sizes):
    """Each pass over the same buffers sees the values that the one before left there."""
    g = torch.Generator(device="cuda").manual_seed(81)
    start = [torch.randn(n, generator=g, device="cuda").to(DT[x]) for n in sizes]
    bounds = [2.0 ** -k for k in range(10)]

    def passes(wait):
        ts = [t.clone() for t in start]
        lst, norms = qg.QGGradList(ts), torch.zeros(len(bounds), device="cuda")
        torch.cuda.synchronize()
        for i, b in enumerate(bounds):
            qg.qg_clip_grad_norm(lst, b, norms[i:i + 1])
            if wait:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        return ts + [norms]

    alone = passes(True)
    for i, b in enumerate(bounds[:-1]):  # the next norm is the bound, to one rounding of each value (and fp16's subnormals)
        assert abs(float(alone[-1][i + 1]) - b) <= b * 2.0 ** -8 + 2.0 ** -25 * sum(sizes) ** 0.5
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(alone, passes(False)))


@pytest.mark.parametrize("x", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T", [1, 37, 200, 2100])
def test_a_training_step(qg, x, T):
    """Adapters over a base, the gradient through the weight, the adapters' gradients onto it, clipping; then the same with
    other inputs in the same buffers."""
    N, K, r = 5128, 2880, 64
    cs = [lora_case([T - T // 3, T // 3], [1, 0], na=2, r=r, N=N, K=K, x=x, seed=s) for s in (82, 83)]
    p, _ = weight(N, K, "nf4", "none", 64, 84)
    X, dY, base = (torch.empty_like(cs[0][n]) for n in ("X", "dY", "Yin"))
    Y, V, dX = torch.empty_like(dY), torch.empty(T, r, device="cuda"), torch.empty_like(X)
    dA, dB, norm = torch.empty_like(cs[0]["A"]), torch.empty_like(cs[0]["B"]), torch.empty(1, device="cuda")
    lst = qg.QGGradList([dA, dB])

    def steps(wait):
        kept = []
        for i in range(6):
            c = cs[i % 2]
            hold = lambda: torch.cuda.synchronize() if wait else None
            for d, s in ((X, c["X"]), (dY, c["dY"]), (base, c["Yin"])):
                d.copy_(s)
            hold()
            qg.qgemm_codebook4(X, p["W"], p["codebook"], p["absmax"], base, block_size=64)
            hold()
            qg.qg_lora_apply(X, c["offsets"], c["ids"], c["A"], c["B"], c["scaling"], base, Y, V=V)
            hold()
            run(qg, p, dY, dX)
            hold()
            qg.qg_lora_grad(dY, X, V, c["offsets"], c["ids"], c["A"], c["B"], c["scaling"], dX, dX, dA, dB)
            hold()
            qg.qg_clip_grad_norm(lst, 1.0, norm)
            hold()
            kept.append([t.clone() for t in (Y, V, dX, dA, dB, norm)])
        torch.cuda.synchronize()
        return kept

    alone = steps(True)
    assert not torch.equal(alone[0][0], alone[1][0])
    for _ in range(2):
        for a, b in zip(alone, steps(False)):
            assert all(torch.equal(u, v) for u, v in zip(a, b))
