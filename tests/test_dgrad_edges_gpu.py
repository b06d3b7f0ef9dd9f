"""The activation gradients of fp32 dY at the ends of fp32's range, and beside parameters that are not finite."""
import pytest
import torch

from test_dgrad_gpu import qg, run, weight  # noqa: F401  (qg: the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M", [40, 300])
@pytest.mark.parametrize("kind,zp", [("u4", "tensor"), ("nf4", "none")])
def test_rows_over_the_whole_range_of_fp32(qg, kind, zp, M):
    """Each row keeps its precision from 1e-37 to 1e36; the weights bring none of them out of fp32's range."""
    p, w = weight(64, 256, kind, zp, 64, 31)
    g = torch.Generator(device="cuda").manual_seed(32)
    dY = torch.randn(M, 64, generator=g, device="cuda") * torch.logspace(-37, 36, M, dtype=torch.float64, device="cuda").float()[:, None]
    dX = torch.empty(M, 256, device="cuda")
    run(qg, p, dY, dX)
    want = dY.double() @ w
    assert float(want.abs().max()) < 3e38
    assert bool(((dX.double() - want).norm(dim=1) <= 1e-5 * want.norm(dim=1)).all())


@pytest.mark.parametrize("M", [40, 300])
def test_large_weights_and_small_rows(qg, M):
    """Weights around 1e35 against rows around 1e-30: neither power of two alone may take the sums out of range."""
    p, w = weight(64, 256, "nf4", "none", 64, 33)
    p["absmax"] = p["absmax"] * 1e35
    g = torch.Generator(device="cuda").manual_seed(34)
    dY = torch.randn(M, 64, generator=g, device="cuda") * 1e-30
    dX = torch.empty(M, 256, device="cuda")
    run(qg, p, dY, dX)
    want = dY.double() @ (w * 1e35)
    assert bool(((dX.double() - want).norm(dim=1) <= 1e-5 * want.norm(dim=1)).all())
