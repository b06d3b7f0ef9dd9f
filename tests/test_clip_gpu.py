"""qg_clip_grad_norm against fp64: sizes, alignments and types of the tensors, values whose squares leave fp32's range,
norms that are zero, infinite or NaN, and its refusals."""
import math

import pytest
import torch

from lora_util import DT, UNIT

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qg():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gemm_blockwise_dequant_gb300 as qg
    from gemm_blockwise_dequant_gb300 import build

    build.build()
    qg.lib()
    return qg


def make(sizes, types, seed=0, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [(torch.randn(n, generator=g, device="cuda") * std).to(DT[types[i % len(types)]]) for i, n in enumerate(sizes)]


def norm64(ts):
    return math.sqrt(sum(float((t.double() ** 2).sum()) for t in ts))


def check(qg, ts, outs, max_norm, eps=1e-6):
    want = norm64(ts)
    keep = [t.clone() for t in ts]
    norm = torch.full((1,), -1.0, device="cuda")
    qg.qg_clip_grad_norm(qg.QGGradList(ts, outs), max_norm, norm, eps=eps)
    # sums of 16 squares in fp32 (2^-24 each), the rest in fp64, half of that by the root, one rounding
    assert abs(float(norm) - want) <= 2.0 ** -20 * want
    c = min(1.0, max_norm / (want + eps))
    for k, o in zip(keep, outs or ts):
        w = k.double() * c
        e = (o.double() - w).abs()
        # the factor to 2^-20, one rounding (half a unit of the smallest subnormal where there is one)
        tiny = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134, torch.float32: 2.0 ** -150}[o.dtype]
        assert bool((e <= (UNIT[o.dtype] + 2.0 ** -19) * w.abs() + tiny).all())
    if outs:
        assert all(torch.equal(t, k) for t, k in zip(ts, keep))
    return float(norm)


SIZES = [[1], [7, 1, 300], [4096], [4095, 4097, 8191, 0, 5], [100003, 3, 1 << 20, 64, 0, 0, 17], [0, 0, 12], [33] * 700]


@pytest.mark.parametrize("sizes", SIZES, ids=[str(len(s)) + "x" + str(sum(s)) for s in SIZES])
@pytest.mark.parametrize("types", [["f32"], ["f16"], ["bf16"], ["bf16", "f32", "f16"]], ids=lambda t: "+".join(t))
def test_sizes_and_types(qg, sizes, types):
    ts = make(sizes, types, seed=1)
    outs = [torch.full_like(t, float("nan")) for t in ts]
    check(qg, ts, outs, 1.0)
    check(qg, ts, outs, 1e9)   # no clipping: a copy
    assert all(torch.equal(t, o) for t, o in zip(ts, outs))
    check(qg, ts, None, 0.5)   # in place


@pytest.mark.parametrize("x", ["f32", "f16", "bf16"])
def test_alignments(qg, x):
    """Slices of flat buffers that start at any element, in and out at different ones."""
    sizes = [5000, 4096, 33, 12289]
    for a, b in ((1, 0), (0, 3), (5, 5), (2, 6)):
        flat, flat_out = make([sum(sizes) + 16], [x], seed=2)[0], torch.zeros(sum(sizes) + 16, dtype=DT[x], device="cuda")
        ts = list(flat[a:a + sum(sizes)].split(sizes))
        outs = list(flat_out[b:b + sum(sizes)].split(sizes))
        check(qg, ts, outs, 2.0)
        assert not flat_out[:b].any() and not flat_out[b + sum(sizes):].any()
        check(qg, ts, None, 2.0)


def test_squares_beyond_fp32(qg):
    for std in (1e25, 1e-25, 1e-42):
        ts = make([1000, 5000], ["f32"], seed=3, std=1.0)
        ts = [(t.double() * std).float() for t in ts]
        want = norm64(ts)
        norm = torch.zeros(1, device="cuda")
        outs = [torch.empty_like(t) for t in ts]
        qg.qg_clip_grad_norm(qg.QGGradList(ts, outs), want * 0.5, norm, eps=0.0)
        assert abs(float(norm) - want) <= max(2.0 ** -20 * want, 2.0 ** -149)
    one = [torch.zeros(5000, device="cuda"), torch.zeros(77, device="cuda")]
    one[1][3] = 3e-30
    norm = torch.zeros(1, device="cuda")
    qg.qg_clip_grad_norm(one, 1.0, norm)
    assert abs(float(norm) / 3e-30 - 1) < 1e-6


def test_zero_infinite_and_nan(qg):
    norm = torch.full((1,), -1.0, device="cuda")
    z = [torch.zeros(100, device="cuda")]
    qg.qg_clip_grad_norm(z, 1.0, norm)
    assert float(norm) == 0 and not z[0].any()
    for bad in (float("inf"), float("-inf"), float("nan")):
        for x in ("f32", "f16", "bf16"):
            ts = make([5000, 60], [x], seed=4)
            ts[0][4321] = bad
            qg.qg_clip_grad_norm(ts, 1.0, norm)
            want = math.inf if abs(bad) == math.inf else math.nan
            assert float(norm) == want or (math.isnan(want) and math.isnan(float(norm)))
            if want == math.inf:
                assert not ts[1].any() and bool(ts[0][4321].isnan()) and not ts[0][:4321].any()
            else:
                assert bool(ts[0].isnan().all()) and bool(ts[1].isnan().all())


def test_max_norm_zero_and_infinite(qg):
    ts = make([3000], ["f32"], seed=5)
    keep = ts[0].clone()
    norm = torch.zeros(1, device="cuda")
    qg.qg_clip_grad_norm(ts, math.inf, norm)
    assert torch.equal(ts[0], keep) and float(norm) > 0
    qg.qg_clip_grad_norm(ts, 0.0, norm)
    assert not ts[0].any()


def test_repeats_and_streams(qg):
    ts = make([100000, 31, 5000], ["bf16"], seed=6)
    outs = [torch.empty_like(t) for t in ts]
    lst = qg.QGGradList(ts, outs)
    seen = []
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for i in range(5):
        norm = torch.zeros(1, device="cuda")
        torch.cuda.synchronize()
        qg.qg_clip_grad_norm(lst, 1.0, norm, stream=s if i % 2 else None)
        torch.cuda.synchronize()
        seen.append((float(norm), [o.clone() for o in outs]))
    assert all(a[0] == seen[0][0] and all(torch.equal(p, q) for p, q in zip(a[1], seen[0][1])) for a in seen)


def test_large(qg):
    """More than 2^31 bytes in one tensor."""
    n = (1 << 30) + 12345
    t = torch.full((n,), 0.5, dtype=torch.bfloat16, device="cuda")
    t[-1] = 64.0
    norm = torch.zeros(1, device="cuda")
    qg.qg_clip_grad_norm([t], 1e3, norm)
    want = math.sqrt((n - 1) * 0.25 + 64.0 ** 2)
    assert abs(float(norm) - want) <= 2.0 ** -20 * want
    c = 1e3 / want
    assert abs(float(t[0]) - 0.5 * c) <= 0.5 * c * 2.0 ** -8 and abs(float(t[-1]) - 64 * c) <= 64 * c * 2.0 ** -8
    assert bool((t[:-1] == t[0]).all())


def test_empty_list_and_refusals(qg):
    norm = torch.full((1,), 5.0, device="cuda")
    qg.qg_clip_grad_norm([], 1.0, norm)
    assert float(norm) == 0.0
    t = torch.zeros(8, device="cuda")
    for m, e in ((-1.0, 1e-6), (math.nan, 1e-6), (1.0, -1.0), (1.0, math.nan)):
        assert qg.qg_clip_grad_norm([t], m, norm, eps=e, raw=True) == qg.QG_ERR_INVALID_ARG
    assert qg.qg_clip_grad_norm([t], 1.0, norm, workspace=torch.zeros(0, dtype=torch.uint8, device="cuda"), raw=True) == qg.QG_ERR_WORKSPACE_TOO_SMALL
    with pytest.raises(ValueError):
        qg.QGGradList([torch.zeros(4, 4, device="cuda").t()[:2]])
    with pytest.raises(ValueError):
        qg.QGGradList([t], [t.half()])
