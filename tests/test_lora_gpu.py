"""qg_lora_apply and qg_lora_grad against plain fp64 forms: types, ranks, request layouts, strides, rows that belong to
no request or to a request without an adapter, and their refusals."""
import pytest
import torch

from lora_util import DT, apply64, check, grad64, lora_case, spans

pytestmark = pytest.mark.gpu

TYPES = [("bf16", "bf16"), ("f16", "f16"), ("f32", "f32"), ("f32", "f16"), ("f32", "bf16")]
LAYOUTS = {
    "one row": ([1], [0]),
    "decode": ([1] * 9, [2, 0, -1, 1, 1, 0, 2, -1, 0]),
    "ragged": ([5, 0, 17, 64, 0, 31, 1], [1, 0, 0, -1, 2, 2, 1]),
    "long": ([300, 129], [2, 0]),
    "one adapter often": ([16, 16, 33, 40], [1, 1, 1, 1]),
    "no adapter": ([3, 20], [-1, -5]),
}


@pytest.fixture(scope="module")
def qg():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gemm_blockwise_dequant_gb300 as qg
    from gemm_blockwise_dequant_gb300 import build

    build.build()
    qg.lib()
    return qg


def run_apply(qg, c, Yin, y, v=True, **kw):
    Y = torch.full((c["T"], c["N"]), float("nan"), dtype=y, device="cuda")
    V = torch.full((c["T"], c["r"]), float("nan"), device="cuda") if v else None
    qg.qg_lora_apply(c["X"], c["offsets"], c["ids"], c["A"], c["B"], c["scaling"], Yin, Y, V=V, **kw)
    return Y, V


def owned(c):
    return slice(0, c["off_host"][-1])


def check_apply(qg, c, Yin, y):
    Y, V = run_apply(qg, c, Yin, y)
    wy, wv, mag = apply64(c, Yin)
    t = owned(c)
    check(Y[t], wy[t], mag[t])
    vm = torch.zeros_like(wv)
    for s, a in spans(c):
        if a >= 0:
            vm[s] = c["X"][s].double().abs() @ c["A"][a].double().abs().t()
    check(V[t], wv[t], vm[t])
    assert bool(Y[c["off_host"][-1]:].isnan().all())  # rows of no request: untouched
    return Y, V


def check_grad(qg, c, V, dXin, g, want_dx=True):
    dX = torch.full((c["T"], c["K"]), float("nan"), dtype=c["x"], device="cuda") if want_dx else None
    dA = torch.full(c["A"].shape, float("nan"), dtype=g, device="cuda")
    dB = torch.full(c["B"].shape, float("nan"), dtype=g, device="cuda")
    if dXin is not None and want_dx:
        dX = torch.empty_like(dXin) if dXin.is_contiguous() else torch.nn.functional.pad(dX, (0, dXin.stride(0) - c["K"]), value=float("nan"))[:, :c["K"]]
        dX.fill_(float("nan"))
    qg.qg_lora_grad(c["dY"], c["X"], V, c["offsets"], c["ids"], c["A"], c["B"], c["scaling"], dXin if want_dx else None, dX, dA, dB)
    (wx, wa, wb), (mx, ma, mb) = grad64(c, V, dXin)
    t = owned(c)
    if want_dx:
        check(dX[t], wx[t], mx[t])
        assert bool(dX[c["off_host"][-1]:].isnan().all())
    check(dA, wa, ma)
    check(dB, wb, mb)
    return dX, dA, dB


def forward_v(c):
    return apply64(c, None)[1].float()


@pytest.mark.parametrize("layout", list(LAYOUTS))
@pytest.mark.parametrize("x,w", TYPES)
def test_types_and_layouts(qg, x, w, layout):
    lens, ids = LAYOUTS[layout]
    c = lora_case(lens, ids, na=3, r=16, N=264, K=512, x=x, w=w, seed=1, extra=3)
    check_apply(qg, c, c["Yin"].to(DT[x]), DT[x])
    check_grad(qg, c, forward_v(c), c["dXin"], DT[w])


@pytest.mark.parametrize("r", [8, 16, 24, 32, 40, 64, 72, 128])
@pytest.mark.parametrize("x", ["bf16", "f16", "f32"])
def test_ranks(qg, x, r):
    c = lora_case([40, 1, 70], [0, 1, 0], na=2, r=r, N=136, K=320, x=x, seed=2)
    check_apply(qg, c, c["Yin"].to(DT[x]), DT[x])
    check_grad(qg, c, forward_v(c), c["dXin"], torch.float32)


@pytest.mark.parametrize("N,K", [(1, 8), (7, 16), (8, 8), (64, 24), (257, 40), (333, 1000), (1000, 136), (2047, 64), (48, 2104)])
@pytest.mark.parametrize("x", ["bf16", "f16", "f32"])
def test_sizes(qg, x, N, K):
    c = lora_case([19, 2, 45], [1, -1, 0], na=2, r=8, N=N, K=K, x=x, seed=3, extra=1)
    check_apply(qg, c, c["Yin"].to(DT[x]), DT[x])
    check_grad(qg, c, forward_v(c), c["dXin"], DT[x])


@pytest.mark.parametrize("x,w", [("bf16", "bf16"), ("f32", "f16")])
def test_row_strides_and_base_types(qg, x, w):
    c = lora_case([33, 7], [0, 1], na=2, r=16, N=96, K=160, x=x, w=w, seed=4, pad=24)
    assert c["X"].stride(0) == 184 and c["dY"].stride(0) == 120
    for y in (DT[x], torch.float32):
        for base in (None, c["Yin"], c["Yin"].to(y)):
            check_apply(qg, c, base, y)
    check_grad(qg, c, forward_v(c), c["dXin"], torch.float32)
    check_grad(qg, c, forward_v(c), None, torch.float32)
    check_grad(qg, c, forward_v(c), None, torch.float32, want_dx=False)
    # a slice of a wider output, in place, and at an odd column
    for at in (96, 97):
        wide = torch.randn(c["T"], 301, device="cuda").to(DT[x])
        keep = wide.clone()
        out = wide[:, at:at + 96]
        qg.qg_lora_apply(c["X"], c["offsets"], c["ids"], c["A"], c["B"], c["scaling"], out, out)
        wy, _, mag = apply64(c, keep[:, at:at + 96])
        check(out, wy, mag)
        assert torch.equal(wide[:, :at], keep[:, :at]) and torch.equal(wide[:, at + 96:], keep[:, at + 96:])


def test_no_scaling_means_one(qg):
    c = lora_case([21], [0], na=1, r=8, N=64, K=64, x="bf16", seed=5, scaling=False)
    check_apply(qg, c, None, torch.bfloat16)
    check_grad(qg, c, forward_v(c), None, torch.bfloat16)


@pytest.mark.parametrize("x", ["bf16", "f16", "f32"])
def test_other_rows_and_adapters_do_not_leak(qg, x):
    """NaN and infinity in rows without an adapter, in rows of no request and in adapters no request uses."""
    c = lora_case([9, 6, 20], [0, -1, 2], na=4, r=16, N=72, K=96, x=x, seed=6, extra=13)
    V = forward_v(c)
    for t in (slice(9, 15), slice(35, 48)):
        c["X"][t], c["dY"][t], V[t] = float("nan"), float("inf"), float("nan")
    c["A"][1], c["B"][3] = float("nan"), float("inf")
    check_apply(qg, c, c["Yin"].to(DT[x]), DT[x])
    _, dA, dB = check_grad(qg, c, V, c["dXin"], torch.float32)
    assert not dA[1].any() and not dB[1].any() and not dA[3].any() and not dB[3].any()


@pytest.mark.parametrize("x", ["bf16", "f16", "f32"])
def test_infinities_of_a_row_stay_in_it(qg, x):
    c = lora_case([20], [0], na=1, r=16, N=64, K=64, x=x, seed=7)
    c["X"][5, 3] = float("inf")
    Y, V = run_apply(qg, c, c["Yin"].to(DT[x]), DT[x])
    rows = torch.ones(20, dtype=torch.bool)
    rows[5] = False
    wy, _, mag = apply64(c, c["Yin"].to(DT[x]))
    check(Y[rows], wy[rows], mag[rows])
    assert not bool(torch.isfinite(Y[5]).any())


def test_large_and_small_values_in_half(qg):
    """V beyond fp16's range and far below its normal range: it is kept in fp32 between the products."""
    for big in (2.0 ** 12, 2.0 ** -12):
        c = lora_case([40], [0], na=1, r=16, N=64, K=256, x="f16", seed=8)
        c["X"] = (c["X"].float() * big).half()
        c["A"] = (c["A"].float() * (big if big < 1 else 16)).half()
        c["B"] = (c["B"].float() / (2.0 ** 14 if big > 1 else 1)).half()
        check_apply(qg, c, None, torch.float32)
        c["dY"] = (c["dY"].float() * big).half()
        check_grad(qg, c, forward_v(c), None, torch.float32)


def test_accumulate_and_repeat(qg):
    c = lora_case([50, 30, 1], [0, 1, 0], na=3, r=8, N=40, K=64, x="bf16", seed=9)
    V = forward_v(c)
    (_, wa, wb), (_, ma, mb) = grad64(c, V, None)
    dA, dB = torch.full(c["A"].shape, 2.0, device="cuda"), torch.full(c["B"].shape, -3.0, device="cuda")
    for _ in range(2):
        qg.qg_lora_grad(c["dY"], c["X"], V, c["offsets"], c["ids"], c["A"], c["B"], c["scaling"], None, None, dA, dB, accumulate=True)
    check(dA, 2 * wa + 2, 2 * ma + 2)
    check(dB, 2 * wb - 3, 2 * mb + 3)
    assert bool((dA[2] == 2).all()) and bool((dB[2] == -3).all())
    outs = [run_apply(qg, c, None, torch.bfloat16) for _ in range(3)]
    grads = [check_grad(qg, c, V, c["dXin"], torch.float32) for _ in range(3)]
    for o in outs[1:]:
        assert all(torch.equal(p, q) for p, q in zip(o, outs[0]))
    for o in grads[1:]:
        assert all(torch.equal(p, q) for p, q in zip(o, grads[0]))


def test_gradient_against_differences(qg):
    """The loss sum(R * Y) is linear in A, B and X each, so its central difference along any direction is exact up to
    rounding: fp32 sums of ~2^10 terms leave about 2^-20 of the loss's terms, divided by the step 2^-4."""
    c = lora_case([13, 20], [1, 0], na=2, r=8, N=48, K=64, x="f32", seed=10)
    g = torch.Generator(device="cuda").manual_seed(11)
    R = torch.randn(33, 48, generator=g, device="cuda")
    c["dY"] = R

    def loss(**other):
        d = dict(c, **other)
        Y, _ = run_apply(qg, d, None, torch.float32)
        return float((Y.double() * R.double()).sum()), float((Y.double() * R.double()).abs().sum())

    dX, dA, dB = check_grad(qg, c, forward_v(c), None, torch.float32)
    for name, grad in (("X", dX), ("A", dA), ("B", dB)):
        D = torch.randn(c[name].shape, generator=g, device="cuda")
        h = 2.0 ** -4
        up, mag = loss(**{name: c[name] + h * D})
        down, _ = loss(**{name: c[name] - h * D})
        slope = float((grad.double() * D.double()).sum())
        assert abs((up - down) / (2 * h) - slope) <= 2.0 ** -20 * mag / h * 4 + 1e-5 * abs(slope)


def test_many_requests_and_large_offsets(qg):
    """More requests than threads of a block, and rows whose byte offset passes 2^31."""
    n = 1500
    lens = [(i * 7) % 4 for i in range(n)]
    c = lora_case(lens, [(i * 5) % 6 - 1 for i in range(n)], na=5, r=8, N=24, K=32, x="f16", seed=12)
    check_apply(qg, c, c["Yin"].half(), torch.float16)
    check_grad(qg, c, forward_v(c), c["dXin"], torch.float16)
    T, ld = 70, 1 << 24  # 70 rows 2^24 values (32 MB) apart
    big = torch.empty(T * ld, dtype=torch.float16, device="cuda").view(T, ld)
    c = lora_case([60, 10], [0, 1], na=2, r=8, N=40, K=64, x="f16", seed=13)
    big[:, :64].copy_(c["X"])
    c["X"] = big[:, :64]
    big[:, 128:168].copy_(c["dY"])
    c["dY"] = big[:, 128:168]
    check_apply(qg, c, None, torch.float16)
    check_grad(qg, c, forward_v(c), None, torch.float16)


def test_another_stream(qg):
    c = lora_case([40, 60], [0, 1], na=2, r=16, N=512, K=512, x="bf16", seed=14)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    Y = torch.zeros(100, 512, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    qg.qg_lora_apply(c["X"], c["offsets"], c["ids"], c["A"], c["B"], c["scaling"], None, Y, stream=s)
    s.synchronize()
    wy, _, mag = apply64(c, None)
    check(Y, wy, mag)


def test_offsets_that_break_the_rule_compute_nothing(qg):
    for off in ([0, 5, 4], [1, 3, 6], [0, 3, 11], [0, -2, 4]):
        c = lora_case([4, 6], [0, 1], na=2, r=8, N=16, K=32, x="bf16", seed=15)
        c["offsets"] = torch.tensor(off, dtype=torch.int64, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        Y, _ = run_apply(qg, c, None, torch.bfloat16, v=False, status=status)
        assert int(status) == 1 and bool(Y.isnan().all())
        status.zero_()
        dX = torch.full((10, 32), float("nan"), dtype=torch.bfloat16, device="cuda")
        dA, dB = torch.full_like(c["A"], 7), torch.full_like(c["B"], 7)
        qg.qg_lora_grad(c["dY"], c["X"], torch.zeros(10, 8, device="cuda"), c["offsets"], c["ids"], c["A"], c["B"], None, None,
                        dX, dA, dB, status=status)
        assert int(status) == 1 and bool(dX.isnan().all())


def test_strange_adapter_counts_as_none(qg):
    c = lora_case([4, 6], [0, 2], na=2, r=8, N=16, K=32, x="bf16", seed=16)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    Y, _ = run_apply(qg, c, c["Yin"], torch.bfloat16, status=status)
    assert int(status) == 1
    wy, _, mag = apply64(c, c["Yin"])
    check(Y, wy, mag)


def test_no_rows(qg):
    c = lora_case([0, 0], [0, 1], na=2, r=8, N=16, K=32, x="bf16", seed=17)
    run_apply(qg, c, None, torch.bfloat16)
    _, dA, dB = check_grad(qg, c, forward_v(c), None, torch.bfloat16)
    assert not dA.any() and not dB.any()


def test_refusals(qg):
    c = lora_case([4, 6], [0, 1], na=2, r=8, N=16, K=32, x="bf16", seed=18)
    Y = torch.zeros(10, 16, dtype=torch.bfloat16, device="cuda")
    call = lambda **o: qg.qg_lora_apply(*[dict(c, **o)[n] for n in ("X", "offsets", "ids", "A", "B", "scaling")],
                                        o.get("Yin", None), o.get("Y", Y), raw=True)
    assert call() == qg.QG_OK
    half = lambda t: t.half()
    assert call(A=half(c["A"]), B=half(c["B"])) == qg.QG_ERR_UNSUPPORTED          # 16-bit activations, other adapters
    assert call(A=c["A"][:, :4].contiguous(), B=c["B"][:, :, :4].contiguous()) == qg.QG_ERR_UNSUPPORTED  # rank 4
    assert call(A=c["A"][:, :, :20].contiguous(), X=c["X"][:, :20]) == qg.QG_ERR_UNSUPPORTED             # K 20
    assert call(Yin=torch.zeros(10, 16, dtype=torch.float16, device="cuda")) == qg.QG_ERR_UNSUPPORTED    # base in another 16-bit type
    assert call(X=torch.zeros(10, 33, dtype=torch.bfloat16, device="cuda")[:, :32]) == qg.QG_ERR_INVALID_ARG  # rows at 66 bytes
    with pytest.raises(ValueError):
        call(X=c["X"][:, ::2])
    with pytest.raises(ValueError):
        call(offsets=c["offsets"].int())
    with pytest.raises(ValueError):
        call(Y=torch.zeros(9, 16, dtype=torch.bfloat16, device="cuda"))
    assert not Y.any() or bool(torch.isfinite(Y).all())
