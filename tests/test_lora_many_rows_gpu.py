"""qg_lora_apply and qg_lora_grad on batches of many rows (the tensor-core kernels of 16-bit activations) against fp64."""
import pytest
import torch

from lora_util import DT, apply64, check, grad64, lora_case
from test_lora_gpu import check_apply, check_grad, forward_v, qg, run_apply  # noqa: F401  (qg: the fixture)

pytestmark = pytest.mark.gpu

LAYOUTS = {
    "one request": ([1000], [0]),
    "packed": ([512, 0, 130, 259, 1, 64, 128, 127], [1, 0, 2, -1, 1, 0, 2, 1]),
    "short and long": ([700] + [3] * 8, [2, 0, 1, -1, 0, 1, 2, 0, 1]),
    "none": ([600, 100], [-1, -1]),
}


@pytest.mark.parametrize("layout", list(LAYOUTS))
@pytest.mark.parametrize("x", ["bf16", "f16", "f32"])
def test_layouts(qg, x, layout):
    lens, ids = LAYOUTS[layout]
    c = lora_case(lens, ids, na=4, r=16, N=328, K=520, x=x, seed=21, extra=9)
    check_apply(qg, c, c["Yin"].to(DT[x]), DT[x])
    check_grad(qg, c, forward_v(c), c["dXin"], DT[x])
    check_grad(qg, c, forward_v(c), None, torch.float32)


@pytest.mark.parametrize("r", [8, 16, 24, 32, 48, 64, 72, 104, 128])
@pytest.mark.parametrize("x", ["bf16", "f16"])
def test_ranks(qg, x, r):
    c = lora_case([300, 450], [0, 1], na=2, r=r, N=392, K=640, x=x, seed=22)
    check_apply(qg, c, c["Yin"].to(DT[x]), DT[x])
    check_grad(qg, c, forward_v(c), c["dXin"], DT[x])
    check_grad(qg, c, forward_v(c), c["dXin"], torch.float32)


@pytest.mark.parametrize("N,K", [(1, 8), (8, 64), (64, 72), (256, 256), (257, 200), (1000, 136), (72, 2056), (3000, 1024)])
@pytest.mark.parametrize("x", ["bf16", "f16", "f32"])
def test_widths(qg, x, N, K):
    c = lora_case([190, 65, 390], [1, -1, 0], na=2, r=8, N=N, K=K, x=x, seed=23, extra=2)
    check_apply(qg, c, c["Yin"].to(DT[x]), DT[x])
    check_grad(qg, c, forward_v(c), c["dXin"], torch.float32)


def test_strides_bases_and_no_input_gradient(qg):
    c = lora_case([533, 77], [0, 1], na=2, r=16, N=96, K=160, x="bf16", seed=24, pad=24)
    for base in (None, c["Yin"], c["Yin"].bfloat16()):
        check_apply(qg, c, base, torch.bfloat16)
        check_apply(qg, c, base if base is None or base.dtype == torch.float32 else None, torch.float32)
        Y, _ = run_apply(qg, c, base, torch.bfloat16, v=False)
        wy, _, mag = apply64(c, base)
        check(Y, wy, mag)
    check_grad(qg, c, forward_v(c), c["dXin"], torch.bfloat16)
    check_grad(qg, c, forward_v(c), None, torch.bfloat16, want_dx=False)
    out = torch.randn(c["T"], 96, device="cuda").bfloat16()
    keep = out.clone()
    qg.qg_lora_apply(c["X"], c["offsets"], c["ids"], c["A"], c["B"], c["scaling"], out, out)
    wy, _, mag = apply64(c, keep)
    check(out, wy, mag)


@pytest.mark.parametrize("x", ["bf16", "f16"])
def test_other_rows_and_adapters_do_not_leak(qg, x):
    lens, ids = [300, 61, 200, 77], [0, -1, 2, 0]
    c = lora_case(lens, ids, na=4, r=24, N=136, K=160, x=x, seed=25, extra=40)
    V = forward_v(c)
    for t in (slice(300, 361), slice(638, 678)):
        c["X"][t], c["dY"][t], V[t] = float("nan"), float("inf"), float("nan")
    c["A"][1], c["B"][3] = float("nan"), float("inf")
    check_apply(qg, c, c["Yin"].to(DT[x]), DT[x])
    _, dA, dB = check_grad(qg, c, V, c["dXin"], torch.float32)
    assert not dA[1].any() and not dB[1].any() and not dA[3].any() and not dB[3].any()


def test_scales_of_half(qg):
    """fp16 keeps V and G scaled by each adapter's largest value: sums far outside fp16's range, in two adapters whose
    values are 2^20 apart."""
    c = lora_case([400, 400], [0, 1], na=2, r=16, N=64, K=256, x="f16", seed=26)
    c["scaling"] = torch.tensor([2.0 ** 12, 2.0 ** -8], device="cuda")
    check_grad(qg, c, forward_v(c), None, torch.float32)
    c["dY"] = (c["dY"].float() * 2.0 ** -12).half()
    check_grad(qg, c, forward_v(c) * 2.0 ** 18, None, torch.float32)
    check_grad(qg, c, forward_v(c) * 2.0 ** -30, None, torch.float32)
    zero = torch.zeros(800, 16, device="cuda")
    _, _, dB = check_grad(qg, c, zero, None, torch.float32)
    assert not dB.any()


def test_accumulate_repeat_and_many_adapters(qg):
    n = 12
    c = lora_case([60 + 7 * i for i in range(n)], [(5 * i) % 7 for i in range(n)], na=8, r=8, N=200, K=64, x="bf16", seed=27)
    V = forward_v(c)
    (_, wa, wb), (_, ma, mb) = grad64(c, V, None)
    dA, dB = torch.full(c["A"].shape, 2.0, device="cuda"), torch.full(c["B"].shape, -3.0, device="cuda")
    for _ in range(2):
        qg.qg_lora_grad(c["dY"], c["X"], V, c["offsets"], c["ids"], c["A"], c["B"], c["scaling"], None, None, dA, dB, accumulate=True)
    check(dA, 2 * wa + 2, 2 * ma + 2)
    check(dB, 2 * wb - 3, 2 * mb + 3)
    first = run_apply(qg, c, None, torch.bfloat16), check_grad(qg, c, V, c["dXin"], torch.bfloat16)
    for _ in range(2):
        again = run_apply(qg, c, None, torch.bfloat16), check_grad(qg, c, V, c["dXin"], torch.bfloat16)
        assert all(torch.equal(a, b) for x, y in zip(first, again) for a, b in zip(x, y))


def test_offsets_that_break_the_rule_compute_nothing(qg):
    for off in ([0, 500, 400], [0, 300, 1001], [2, 300, 900]):
        c = lora_case([400, 600], [0, 1], na=2, r=8, N=16, K=32, x="f16", seed=28)
        c["offsets"] = torch.tensor(off, dtype=torch.int64, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        Y, V = run_apply(qg, c, None, torch.float16, status=status)
        assert int(status) == 1 and bool(Y.isnan().all()) and bool(V.isnan().all())
        status.zero_()
        dX = torch.full((1000, 32), float("nan"), dtype=torch.float16, device="cuda")
        dA, dB = torch.full_like(c["A"], 7), torch.full_like(c["B"], 7)
        qg.qg_lora_grad(c["dY"], c["X"], torch.zeros(1000, 8, device="cuda"), c["offsets"], c["ids"], c["A"], c["B"], None, None, dX,
                        dA, dB, status=status)
        assert int(status) == 1 and bool(dX.isnan().all()) and bool((dA == 7).all()) and bool((dB == 7).all())
    assert qg.qg_read_device_fault() == 0


@pytest.mark.parametrize("x", ["bf16", "f32"])
def test_more_rows_than_a_grid_dimension(qg, x):
    c = lora_case([40000, 0, 25000, 5500], [0, 1, -1, 1], na=2, r=8, N=24, K=32, x=x, seed=29)
    check_apply(qg, c, c["Yin"].to(DT[x]), DT[x])
    check_grad(qg, c, forward_v(c), c["dXin"], torch.float32)


@pytest.mark.parametrize("x", ["bf16", "f16"])
def test_offsets_beyond_32_bits(qg, x):
    """Rows 2^24 values apart: the last ones lie past 2^32 bytes and values."""
    T, ld = 300, 1 << 24
    big = torch.empty(T * ld, dtype=DT[x], device="cuda").view(T, ld)
    c = lora_case([250, 50], [0, 1], na=2, r=16, N=40, K=64, x=x, seed=30)
    for name, at in (("X", 0), ("dY", 128), ("dXin", 256)):
        part = big[:, at:at + c[name].shape[1]]
        part.copy_(c[name])
        c[name] = part
    check_apply(qg, c, None, DT[x])
    V = forward_v(c)
    dA, dB = torch.empty_like(c["A"]), torch.empty_like(c["B"])
    dX = big[:, 512:576]
    qg.qg_lora_grad(c["dY"], c["X"], V, c["offsets"], c["ids"], c["A"], c["B"], c["scaling"], c["dXin"], dX, dA, dB)
    (wx, wa, wb), (mx, ma, mb) = grad64(c, V, c["dXin"])
    check(dX, wx, mx)
    check(dA, wa, ma)
    check(dB, wb, mb)


def test_an_infinity_does_not_scale_the_others(qg):
    """fp16: one infinite value of V must not push the other columns' values, far beyond fp16's range, over it."""
    c = lora_case([200], [0], na=1, r=8, N=32, K=64, x="f16", seed=31)
    V = forward_v(c) * 2.0 ** 20
    V[7, 3] = float("inf")
    dA, dB = torch.empty(1, 8, 64, device="cuda"), torch.empty(1, 32, 8, device="cuda")
    qg.qg_lora_grad(c["dY"], c["X"], V, c["offsets"], c["ids"], c["A"], c["B"], c["scaling"], None, None, dA, dB)
    (_, wa, wb), (_, ma, mb) = grad64(c, V, None)
    keep = [j for j in range(8) if j != 3]
    check(dA, wa, ma)
    check(dB[:, :, keep], wb[:, :, keep], mb[:, :, keep])
    assert not bool(torch.isfinite(dB[:, :, 3]).any())


@pytest.mark.parametrize("lens,r,N,K", [([1000, 30, 470], 64, 6001, 4096), ([33, 1, 300], 24, 523, 512), ([1] * 40, 8, 262, 1024)])
@pytest.mark.parametrize("x", ["bf16", "f16", "f32"])
def test_outputs_of_odd_widths(qg, x, lens, r, N, K):
    """Rows that begin at no 16-byte boundary: every type of base and output, in place, and rows without an adapter."""
    c = lora_case(lens, [(i % 3) - 1 for i in range(len(lens))], na=2, r=r, N=N, K=K, x=x, seed=25, extra=3)
    for y in {DT[x], torch.float32}:
        for base in (None, c["Yin"], c["Yin"].to(y)):
            check_apply(qg, c, base, y)
    out = c["Yin"].to(DT[x])
    keep = out.clone()
    qg.qg_lora_apply(c["X"], c["offsets"], c["ids"], c["A"], c["B"], c["scaling"], out, out)
    wy, _, mag = apply64(c, keep)
    n = c["off_host"][-1]
    check(out[:n], wy[:n], mag[:n])
    assert torch.equal(out[n:], keep[n:])


@pytest.mark.parametrize("lens,N,K,pad", [([300, 0, 211], 1001, 264, 0), ([300, 0, 211], 1002, 264, 0), ([40, 3], 331, 520, 1),
                                          ([200, 9], 330, 520, 2), ([17], 6, 8, 0)])
@pytest.mark.parametrize("x,r", [("bf16", 16), ("f16", 40), ("f32", 16), ("f32", 64)])
def test_gradients_of_odd_widths(qg, x, r, lens, N, K, pad):
    """Rows of dY that begin at 2-byte and 4-byte boundaries, with odd and even widths."""
    c = lora_case(lens, [1, 0, 1][:len(lens)], na=2, r=r, N=N, K=K, x=x, seed=26, extra=2)
    if pad:
        c["dY"] = torch.nn.functional.pad(c["dY"], (0, pad), value=float("nan"))[:, :N]
    for g in {DT[x], torch.float32}:
        check_grad(qg, c, forward_v(c), c["dXin"], g)
