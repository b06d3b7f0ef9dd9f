"""qg_lora_apply and qg_lora_grad at the ends of their ranges: no adapters, no outputs, single rows of odd strides, and sums over
very many rows of one sign."""
import pytest
import torch

from lora_util import DT, check, grad64, lora_case, scale_of
from test_lora_gpu import check_apply, check_grad, forward_v, qg  # noqa: F401  (qg: the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [1, 40, 2048])
@pytest.mark.parametrize("x", ["bf16", "f16", "f32"])
def test_no_adapters_at_all(qg, x, T):
    """Without an adapter there is nothing to add: Y is Y_in, V is zero and dX is dX_in, whatever the number of rows."""
    c = lora_case([T // 2, T - T // 2], [-1, -1], na=1, r=64, N=8192, K=4096, x=x, seed=61)
    c["A"], c["B"], c["scaling"] = c["A"][:0], c["B"][:0], None
    base = c["Yin"].to(DT[x])
    Y, V = torch.empty_like(base), torch.full((T, 64), float("nan"), device="cuda")
    qg.qg_lora_apply(c["X"], c["offsets"], c["ids"], c["A"], c["B"], None, base, Y, V=V)
    assert torch.equal(Y, base) and not V.any()
    dX = torch.empty_like(c["dXin"])
    qg.qg_lora_grad(c["dY"], c["X"], V, c["offsets"], c["ids"], c["A"], c["B"], None, c["dXin"], dX, torch.empty_like(c["A"]), torch.empty_like(c["B"]))
    assert torch.equal(dX, c["dXin"])


@pytest.mark.parametrize("T", [1, 40, 2048])
@pytest.mark.parametrize("x", ["bf16", "f16", "f32"])
def test_gradient_of_no_outputs(qg, x, T):
    """N = 0: the sums over outputs are empty, so dX is dX_in and dA is zero."""
    c = lora_case([T], [0], na=2, r=64, N=0, K=32768, x=x, seed=62, extra=3)
    V = torch.ones(T + 3, 64, device="cuda")
    dX = torch.full_like(c["dXin"], float("nan"))
    dA = torch.full(c["A"].shape, 5.0, device="cuda")
    dB = torch.empty(c["B"].shape, device="cuda")
    call = lambda base, out, **kw: qg.qg_lora_grad(c["dY"], c["X"], V, c["offsets"], c["ids"], c["A"], c["B"], c["scaling"], base, out, dA, dB, **kw)
    call(None, None, accumulate=True)
    assert bool((dA == 5).all())
    call(c["dXin"], dX)
    assert torch.equal(dX[:T], c["dXin"][:T]) and bool(dX[T:].isnan().all()) and not dA.any()
    call(None, dX)
    assert not dX[:T].any() and bool(dX[T:].isnan().all())


@pytest.mark.parametrize("x", ["bf16", "f16", "f32"])
def test_a_single_row_has_no_stride(qg, x):
    """One row out of a matrix whose rows begin at odd places: what lies behind it is never read."""
    c = lora_case([1], [1], na=2, r=16, N=72, K=64, x=x, seed=63)
    odd = lambda t: torch.cat([t, torch.full((1, 5), float("nan"), dtype=t.dtype, device="cuda")], 1).repeat(3, 1)[:1, :t.shape[1]]
    for name in ("X", "dY", "dXin"):
        c[name] = odd(c[name])
    assert c["X"].stride(0) == 69
    check_apply(qg, c, odd(c["Yin"].to(DT[x])), DT[x])
    V = forward_v(c)
    (wx, wa, wb), (mx, ma, mb) = grad64(c, V, c["dXin"])
    dX, dA, dB = torch.empty(1, 64, dtype=DT[x], device="cuda"), torch.empty_like(c["A"]), torch.empty_like(c["B"])
    qg.qg_lora_grad(c["dY"], c["X"], V, c["offsets"], c["ids"], c["A"], c["B"], c["scaling"], c["dXin"], dX, dA, dB)
    check(dX, wx, mx)
    check(dA, wa, ma)
    check(dB, wb, mb)


@pytest.mark.parametrize("x", ["bf16", "f16"])
def test_many_rows_of_one_sign(qg, x):
    """2^20 rows whose products all have one sign, 16-bit gradients: random signs would hide an accumulator that rounds one way."""
    T, na, r, n = 1 << 20, 64, 8, 512
    g = torch.Generator(device="cuda").manual_seed(64)
    pos = lambda *s, std=1.0: (torch.randn(*s, generator=g, device="cuda") * std).abs()
    c = dict(T=T, N=n, K=n, r=r, na=na, lens=[T], ids_host=[5], off_host=[0, T], x=DT[x], w=DT[x])
    c["X"], c["dY"] = pos(T, n).to(DT[x]), pos(T, n).to(DT[x])
    c["A"], c["B"] = pos(na, r, n).to(DT[x]), pos(na, n, r, std=0.1).to(DT[x])
    c["scaling"] = torch.full((na,), 2.0 ** -15, device="cuda")
    c["offsets"], c["ids"] = torch.tensor([0, T], device="cuda"), torch.tensor([5], dtype=torch.int32, device="cuda")
    V = pos(T, r)
    dA, dB = torch.empty_like(c["A"]), torch.empty_like(c["B"])
    qg.qg_lora_grad(c["dY"], c["X"], V, c["offsets"], c["ids"], c["A"], c["B"], c["scaling"], None, None, dA, dB)
    s, dy = scale_of(c, 5), c["dY"].double()
    wa = (s * (dy @ c["B"][5].double())).t() @ c["X"].double()
    wb = s * (dy.t() @ V.double())
    check(dA[5], wa, wa)
    check(dB[5], wb, wb)
    for d in (dA, dB):
        d[5] = 0
        assert not d.any()
