"""Experts whose weights a kernel replaces just ahead of the layer (swapped in, quantized anew): calls one behind another on a stream, and
replayed, see what was written last of the codes, scales and zero points of both products."""
import pytest
import torch

import gemm_blockwise_dequant_gb300 as qg
from test_moe_tokens_gpu import choose, layer, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits,bs", [(2, 32), (2, 64), (4, 32), (4, 128), (8, 32), (8, 64)])
@pytest.mark.parametrize("T,E,k,H,I", [(1, 4, 2, 256, 256), (3, 8, 4, 384, 640), (40, 6, 3, 512, 256)])
def test_weights_written_between_calls(bits, bs, T, E, k, H, I):
    sets = [layer(E, H, I, bits, bs, True, True, seed=s) for s in range(3)]
    X = torch.randn(T, H, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").half()
    ids, weights = choose(T, E, k)
    want = []
    for w in sets:
        want.append(run(X, ids, weights, w, bits, bs))
        torch.cuda.synchronize()
    live = {n: t.clone() for n, t in sets[0].items()}
    room = torch.empty(qg.qmoe_tokens_workspace_bytes(T, k, H, I), dtype=torch.uint8, device="cuda")
    got = torch.empty(60, *X.shape, dtype=X.dtype, device="cuda")

    def rounds():
        for i in range(60):
            # the second product's last, so that they are what was written just before
            for n in sorted(live):
                live[n].copy_(sets[i % 3][n])
            run(X, ids, weights, live, bits, bs, y=got[i], workspace=room)

    rounds()
    for i in range(60):
        assert torch.equal(got[i], want[i % 3]), i
    got.zero_()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rounds()
    for _ in range(2):
        got.zero_()
        graph.replay()
        for i in range(60):
            assert torch.equal(got[i], want[i % 3]), i
