"""qg_lora_apply and qg_lora_grad where the products over rows are two launches (the first one on the tensor cores), against
fp64.  Every case asserts that it takes that path, by the workspace that only this path needs."""
import pytest
import torch

from lora_util import DT, apply64, check, grad64, lora_case
from test_lora_gpu import check_apply, check_grad, forward_v, qg, run_apply  # noqa: F401  (qg: the fixture)

pytestmark = pytest.mark.gpu

LENS, IDS = [1000, 130, 0, 700, 333, 37], [0, -1, 1, 1, 0, 2]  # whole and ragged tiles, some of fewer than 32 rows


def case(qg, lens, ids, *, r, N, K, x, **kw):
    c = lora_case(lens, ids, r=r, N=N, K=K, x=x, **kw)
    assert qg.qg_lora_apply_workspace_bytes(c["T"], len(lens), r, N, K) > 0 and c["T"] // 128 >= len(lens) and x != "f32"
    assert c["X"].stride(0) % 8 == 0 and c["dY"].stride(0) % 8 == 0
    return c


def wide_enough(T, r):
    """N and K, multiples of 8 but not of 32, with which T rows of rank r go in two launches."""
    need = 1.2e9 / (T * (r + 16))
    K = int(0.4 * need) // 32 * 32 + 40
    return (int(need) - K) // 32 * 32 + 56, K


def same_as_before(c, V, dX_in, first, qg, g):
    again = check_grad(qg, c, V, dX_in, g)
    return all(torch.equal(a.nan_to_num(7.0), b.nan_to_num(7.0)) for a, b in zip(first, again))


@pytest.mark.parametrize("T,N,K,r", [(2048, 9216, 2304, 64), (2048, 8192, 2880, 64), (2048, 5120, 11008, 32), (1024, 5120, 13824, 64),
                                     (1024, 4096, 17920, 64), (2048, 8192, 4104, 64), (2048, 16384, 4160, 16), (4100, 12288, 4160, 8)])
@pytest.mark.parametrize("x", ["bf16", "f16"])
def test_input_gradient_with_a_base(qg, x, T, N, K, r):
    """dX_in beside an odd number of 32-column groups a CTA, or a last group that is not whole: the warps are then at
    different loops over their base rows."""
    lens = [T // 2 - 3, 20, T // 4, T - (T // 2 - 3) - 20 - T // 4 - 31, 31]
    c = case(qg, lens, [0, 1, -1, 1, 0], na=2, r=r, N=N, K=K, x=x, seed=41)
    V = forward_v(c)
    first = check_grad(qg, c, V, c["dXin"], DT[x])
    for _ in range(3):
        assert same_as_before(c, V, c["dXin"], first, qg, DT[x])
    dX = c["dXin"].clone()
    qg.qg_lora_grad(c["dY"], c["X"], V, c["offsets"], c["ids"], c["A"], c["B"], c["scaling"], dX, dX, torch.empty_like(c["A"]), torch.empty_like(c["B"]))
    assert torch.equal(dX, first[0])


@pytest.mark.parametrize("r", [8, 16, 24, 32, 48, 64, 72, 104, 128])
@pytest.mark.parametrize("x", ["bf16", "f16"])
def test_ranks(qg, x, r):
    N, K = wide_enough(sum(LENS) + 5, r)
    c = case(qg, LENS, IDS, na=4, r=r, N=N, K=K, x=x, seed=42, extra=5)
    for base in (None, c["Yin"], c["Yin"].to(DT[x])):
        Y, _ = check_apply(qg, c, base, DT[x])
        assert torch.equal(run_apply(qg, c, base, DT[x], v=False)[0].nan_to_num(7.0), Y.nan_to_num(7.0))
    check_apply(qg, c, c["Yin"], torch.float32)
    V = forward_v(c)
    check_grad(qg, c, V, c["dXin"], DT[x])
    check_grad(qg, c, V, None, torch.float32)
    check_grad(qg, c, V, None, torch.float32, want_dx=False)


@pytest.mark.parametrize("N,K", [(8192, 8224), (8200, 8208), (8211, 8216), (24, 16400), (16400, 8), (16384, 64)])
@pytest.mark.parametrize("x", ["bf16", "f16"])
def test_widths(qg, x, N, K):
    c = lora_case(LENS, IDS, na=3, r=24, N=N, K=K, x=x, seed=43)
    assert qg.qg_lora_apply_workspace_bytes(c["T"], len(LENS), 24, N, K) > 0
    check_apply(qg, c, c["Yin"].to(DT[x]), DT[x])
    check_apply(qg, c, c["Yin"], DT[x])
    check_grad(qg, c, forward_v(c), c["dXin"], DT[x])


@pytest.mark.parametrize("x", ["bf16", "f16"])
def test_strides_and_in_place(qg, x):
    c = case(qg, LENS, IDS, na=3, r=32, N=7976, K=4064, x=x, seed=44, pad=24)
    assert c["X"].stride(0) == 4088 and c["dY"].stride(0) == 8000
    check_apply(qg, c, c["Yin"].to(DT[x]), DT[x])
    check_grad(qg, c, forward_v(c), c["dXin"], DT[x])
    for at in (16, 21):
        wide = torch.randn(c["T"], 8100, device="cuda").to(DT[x])
        keep = wide.clone()
        out = wide[:, at:at + 7976]
        qg.qg_lora_apply(c["X"], c["offsets"], c["ids"], c["A"], c["B"], c["scaling"], out, out)
        wy, _, mag = apply64(c, keep[:, at:at + 7976])
        check(out, wy, mag)
        assert torch.equal(wide[:, :at], keep[:, :at]) and torch.equal(wide[:, at + 7976:], keep[:, at + 7976:])


@pytest.mark.parametrize("x", ["bf16", "f16"])
def test_other_rows_and_adapters_do_not_leak(qg, x):
    c = case(qg, LENS, [0, -1, 2, 2, 0, -1], na=4, r=24, N=8200, K=8208, x=x, seed=45, extra=40)
    V = forward_v(c)
    for t in (slice(1000, 1130), slice(2163, 2240)):
        c["X"][t], c["dY"][t], V[t] = float("nan"), float("inf"), float("nan")
    c["A"][1], c["B"][3] = float("nan"), float("inf")
    check_apply(qg, c, c["Yin"].to(DT[x]), DT[x])
    for g in (DT[x], torch.float32):
        _, dA, dB = check_grad(qg, c, V, None, g)
        assert not dA[1].any() and not dB[1].any() and not dA[3].any() and not dB[3].any()


def test_scales_of_half(qg):
    """Sums far outside fp16's range, in adapters whose values are 2^20 apart."""
    c = case(qg, [1200, 1000], [0, 1], na=2, r=16, N=12288, K=8192, x="f16", seed=46)
    c["scaling"] = torch.tensor([2.0 ** 12, 2.0 ** -8], device="cuda")
    V = forward_v(c)
    check_grad(qg, c, V, None, torch.float32)
    c["dY"] = (c["dY"].float() * 2.0 ** -12).half()
    check_grad(qg, c, V * 2.0 ** 18, None, torch.float32)
    check_grad(qg, c, V * 2.0 ** -30, None, torch.float32)


@pytest.mark.parametrize("x", ["bf16", "f16"])
def test_accumulate_and_many_adapters(qg, x):
    n = 12
    lens, ids = [140 + 17 * i for i in range(n)], [(5 * i) % 7 for i in range(n)]
    c = case(qg, lens, ids, na=8, r=32, N=6000, K=4104, x=x, seed=47)
    V = forward_v(c)
    (_, wa, wb), (_, ma, mb) = grad64(c, V, None)
    dA, dB = torch.full(c["A"].shape, 2.0, device="cuda"), torch.full(c["B"].shape, -3.0, device="cuda")
    for _ in range(2):
        qg.qg_lora_grad(c["dY"], c["X"], V, c["offsets"], c["ids"], c["A"], c["B"], c["scaling"], None, None, dA, dB, accumulate=True)
    check(dA, 2 * wa + 2, 2 * ma + 2)
    check(dB, 2 * wb - 3, 2 * mb + 3)
    check_apply(qg, c, c["Yin"].to(DT[x]), DT[x])


@pytest.mark.parametrize("x", ["bf16", "f16"])
def test_calls_one_behind_another_in_one_workspace(qg, x):
    """Two inputs in turn, with nothing waited for: each call gives what it gives alone."""
    cs = [case(qg, LENS, IDS, na=3, r=64, N=5128, K=2888, x=x, seed=s) for s in (48, 49)]
    vs = [forward_v(c) for c in cs]
    T, S = cs[0]["T"], len(LENS)
    ws = torch.empty(max(qg.qg_lora_grad_workspace_bytes(T, S, 3, 64, 5128, 2888), qg.qg_lora_apply_workspace_bytes(T, S, 64, 5128, 2888)),
                     dtype=torch.uint8, device="cuda")

    def calls(i):
        c, out = cs[i], [torch.empty(T, 5128, dtype=DT[x], device="cuda"), torch.empty_like(cs[i]["dXin"])]
        grads = [torch.empty_like(c["A"]), torch.empty_like(c["B"])]
        qg.qg_lora_apply(c["X"], c["offsets"], c["ids"], c["A"], c["B"], c["scaling"], None, out[0], workspace=ws)
        qg.qg_lora_grad(c["dY"], c["X"], vs[i], c["offsets"], c["ids"], c["A"], c["B"], c["scaling"], c["dXin"], out[1], *grads, workspace=ws)
        return out + grads

    alone = []
    for i in range(2):
        alone.append(calls(i))
        torch.cuda.synchronize()
    behind = [calls(i % 2) for i in range(8)]
    for i, out in enumerate(behind):
        assert all(torch.equal(a, b) for a, b in zip(out, alone[i % 2]))


@pytest.mark.parametrize("x", ["bf16", "f16"])
def test_offsets_that_break_the_rule_compute_nothing(qg, x):
    for off in ([0, 1500, 1400], [0, 300, 2201], [2, 300, 900]):
        c = case(qg, [1200, 1000], [0, 1], na=2, r=16, N=12288, K=8192, x=x, seed=50)
        c["offsets"] = torch.tensor(off, dtype=torch.int64, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        Y, V = run_apply(qg, c, None, DT[x], status=status)
        assert int(status) == 1 and bool(Y.isnan().all()) and bool(V.isnan().all())
        status.zero_()
        dX = torch.full((2200, 8192), float("nan"), dtype=DT[x], device="cuda")
        dA, dB = torch.full_like(c["A"], 7), torch.full_like(c["B"], 7)
        qg.qg_lora_grad(c["dY"], c["X"], torch.zeros(2200, 16, device="cuda"), c["offsets"], c["ids"], c["A"], c["B"], None, None, dX, dA, dB,
                        status=status)
        assert int(status) == 1 and bool(dX.isnan().all()) and bool((dA == 7).all()) and bool((dB == 7).all())
    assert qg.qg_read_device_fault() == 0


@pytest.mark.parametrize("x", ["bf16", "f16"])
def test_many_rows(qg, x):
    c = case(qg, [40000, 0, 25000, 5500], [0, 1, -1, 1], na=2, r=8, N=424, K=328, x=x, seed=51)
    check_apply(qg, c, c["Yin"].to(DT[x]), DT[x])
    check_grad(qg, c, forward_v(c), c["dXin"], torch.float32)
