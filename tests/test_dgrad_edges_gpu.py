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


@pytest.mark.parametrize("M", [40, 300])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
@pytest.mark.parametrize("kind,zp,size", [("nf4", "none", 1e6), ("nf4", "none", 1e-6), ("u4", "tensor", 2.0 ** -7), ("u8", "none", 2.0 ** -7)])
def test_a_parameter_that_is_not_finite_stays_in_its_block(qg, kind, zp, size, bad, M):
    """One block's absmax or scale is infinite or NaN: the columns of the other blocks keep their precision."""
    p, w = weight(64, 256, kind, zp, 64, 35)
    name = "absmax" if kind == "nf4" else "scales"
    p[name] = (p[name] * size).contiguous()
    w = w * size
    if kind != "nf4":  # the products with 2^-7 are rounded where they are subnormal in fp16: take what is there
        z = p["zp"].double().repeat_interleave(64, 1) if zp == "tensor" else float(1 << (p["bits"] - 1))
        one = torch.ones_like(p["scales"])
        q = dict(p, scales=one, zp=None if zp == "none" else torch.zeros_like(one))
        eye = torch.eye(64, device="cuda")
        codes = torch.empty(64, 256, device="cuda")
        run(qg, q, eye, codes)
        w = (codes.double() + (float(1 << (p["bits"] - 1)) if zp == "none" else 0.0) - z) * p["scales"].double().repeat_interleave(64, 1)
    p[name][10, 2] = bad
    g = torch.Generator(device="cuda").manual_seed(36)
    dY = torch.randn(M, 64, generator=g, device="cuda")
    dX = torch.empty(M, 256, device="cuda")
    run(qg, p, dY, dX)
    keep = torch.ones(256, dtype=torch.bool, device="cuda")
    keep[128:192] = False
    want = dY.double() @ torch.where(keep, w, 0.0)
    assert bool(((dX.double()[:, keep] - want[:, keep]).norm(dim=1) <= 1e-5 * want[:, keep].norm(dim=1)).all())
    assert not bool(torch.isfinite(dX[:, ~keep]).all())
