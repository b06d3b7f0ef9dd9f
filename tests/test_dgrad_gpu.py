"""qgemm_nbits_dgrad, qgemm_nbits_uniform_zp_dgrad and qgemm_codebook4_dgrad against fp64 products with the dequantized
weight, and against the forward pass by the adjoint identity."""
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


def weight(N, K, kind, zp, bs, seed):
    """Codes, parameters and the weight in fp64 (unpacked bit by bit)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    bits = 4 if kind == "nf4" else int(kind[1])
    W = torch.randint(0, 256, (N, K * bits // 8), generator=g, device="cuda", dtype=torch.uint8)
    bit = ((W[:, :, None].int() >> torch.arange(8, device="cuda")) & 1).reshape(N, K, bits)
    q = (bit << torch.arange(bits, device="cuda")).sum(-1)
    p = dict(bits=bits, bs=bs, W=W, kind=kind)
    if kind == "nf4":
        p["codebook"] = torch.sort(torch.randn(16, generator=g, device="cuda")).values
        p["absmax"] = torch.rand(N, K // bs, generator=g, device="cuda") + 0.1
        w = p["codebook"].double()[q] * p["absmax"].double().repeat_interleave(bs, 1)
    else:
        p["scales"] = (torch.rand(N, K // bs, generator=g, device="cuda") * 0.05 + 0.01).half()
        p["zp"] = {"none": None, "uniform": 1.5,
                   "tensor": torch.randint(0, 1 << bits, (N, K // bs), generator=g, device="cuda").half()}[zp]
        z = float(1 << (bits - 1)) if zp == "none" else 1.5 if zp == "uniform" else p["zp"].double().repeat_interleave(bs, 1)
        w = (q.double() - z) * p["scales"].double().repeat_interleave(bs, 1)
    return p, w


def run(qg, p, dY, dX, **kw):
    if p["kind"] == "nf4":
        return qg.qgemm_codebook4_dgrad(dY, p["W"], p["codebook"], p["absmax"], dX, block_size=p["bs"], **kw)
    if isinstance(p["zp"], float):
        return qg.qgemm_nbits_uniform_zp_dgrad(dY, p["W"], p["scales"], p["zp"], dX, bits=p["bits"], block_size=p["bs"], **kw)
    return qg.qgemm_nbits_dgrad(dY, p["W"], p["scales"], p["zp"], dX, bits=p["bits"], block_size=p["bs"], **kw)


def check(qg, M, N, K, kind="u4", zp="tensor", bs=64, x="bf16", out=None, seed=0):
    p, w = weight(N, K, kind, zp, bs, seed)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    dY = torch.randn(M, N, generator=g, device="cuda").to(DT[x])
    dX = torch.full((M, K), float("nan"), dtype=DT[out or x], device="cuda")
    run(qg, p, dY, dX)
    want, mag = dY.double() @ w, dY.double().abs() @ w.abs()
    e = (dX.double() - want).abs()
    # one rounding of the result; the weight rounded to a 16-bit dY's type (fp32: both kept to 2^-20); at most 2^-24
    # of the terms' magnitude for each of the sequential additions (N / 16 of them, the tensor cores' K step)
    wr = UNIT[DT[x]] if x != "f32" else 2.0 ** -20
    room = UNIT[dX.dtype] * want.abs() + (wr + 2.0 ** -24 * (N / 16 + 8)) * mag
    assert bool((e <= room).all()), float((e / room).max())
    # independent roundings of the weights add up as their squares: the norm is within both roundings
    assert float(e.norm()) <= (UNIT[dX.dtype] + wr + 4e-6) * float(want.norm()) * (1 if M * K > 64 else 8)
    return dX


@pytest.mark.parametrize("kind,zp", [("u2", "none"), ("u2", "uniform"), ("u2", "tensor"), ("u3", "tensor"), ("u3", "none"), ("u4", "none"),
                                     ("u4", "uniform"), ("u4", "tensor"), ("u8", "none"), ("u8", "uniform"), ("u8", "tensor"), ("nf4", "none")])
@pytest.mark.parametrize("x", ["f16", "bf16", "f32"])
def test_formats(qg, kind, zp, x):
    check(qg, 70, 200, 256, kind, zp, x=x, seed=1)


@pytest.mark.parametrize("bs", [32, 64, 128, 256])
@pytest.mark.parametrize("kind", ["u2", "u4", "u8", "nf4"])
def test_block_sizes(qg, kind, bs):
    check(qg, 130, 136, 768, kind, bs=bs, x="f16", seed=2)
    check(qg, 40, 72, 512, kind, bs=bs, x="bf16", seed=3)


@pytest.mark.parametrize("M,N,K", [(1, 1, 64), (1, 8, 64), (2, 7, 128), (3, 64, 64), (9, 63, 320), (16, 65, 192), (127, 129, 448), (128, 128, 256),
                                   (129, 16, 1088), (257, 72, 512), (300, 1000, 96 * 2), (513, 264, 832), (5, 2001, 64)])
@pytest.mark.parametrize("x,out", [("f16", "f16"), ("bf16", "f32"), ("f32", "f32"), ("f32", "bf16")])
def test_sizes(qg, M, N, K, x, out):
    check(qg, M, N, K, "u4", "tensor", x=x, out=out, seed=4)
    check(qg, M, N, K, "u2", "uniform", bs=32, x=x, out=out, seed=5)


@pytest.mark.parametrize("K", [32, 96, 160, 224, 416])
@pytest.mark.parametrize("kind", ["u2", "u4", "u8", "nf4"])
def test_rows_of_any_block_count(qg, kind, K):
    """Weight and parameter rows that are no multiple of 16 bytes."""
    check(qg, 33, 48, K, kind, bs=32, x="bf16", seed=6)
    check(qg, 33, 48, K, kind, bs=32, x="f32", seed=7)


@pytest.mark.parametrize("x", ["f16", "bf16", "f32"])
def test_many_tiles(qg, x):
    check(qg, 700, 1100, 2304, "u2", "uniform", x=x, seed=8)
    check(qg, 1030, 520, 1344, "nf4", x=x, seed=9)


@pytest.mark.parametrize("kind,zp", [("u2", "uniform"), ("u4", "tensor"), ("u8", "none"), ("nf4", "none")])
def test_adjoint_of_the_forward_pass(qg, kind, zp):
    """sum(dY * forward(X)) = sum(X * dX): what a difference of the (linear) forward pass along X gives.  Both sides are
    fp32 sums whose terms are right to 2^-20 of their magnitude."""
    M, N, K = 24, 96, 512
    p, w = weight(N, K, kind, zp, 64, 10)
    g = torch.Generator(device="cuda").manual_seed(11)
    X, dY = torch.randn(M, K, generator=g, device="cuda"), torch.randn(M, N, generator=g, device="cuda")
    Y, dX = torch.empty(M, N, device="cuda"), torch.empty(M, K, device="cuda")
    if kind == "nf4":
        qg.qgemm_codebook4(X, p["W"], p["codebook"], p["absmax"], Y, block_size=64)
    elif zp == "uniform":
        qg.qgemm_nbits_uniform_zp(X, p["W"], p["scales"], 1.5, Y, bits=p["bits"], block_size=64)
    else:
        qg.qgemm_nbits(X, p["W"], p["scales"], p["zp"], Y, bits=p["bits"], block_size=64)
    run(qg, p, dY, dX)
    left, right = (dY.double() * Y.double()), (X.double() * dX.double())
    assert abs(float(left.sum() - right.sum())) <= 2.0 ** -18 * float((dY.double().abs() @ w.abs() * X.double().abs()).sum())


@pytest.mark.parametrize("M", [40, 300])
def test_long_sums(qg, M):
    """Contractions of 8192 rows of the weight and more stay as exact as short ones."""
    for N in (8192, 20000):
        check(qg, M, N, 128, "u4", "tensor", x="f32", seed=20)
        p, w = weight(N, 128, "nf4", "none", 64, 21)
        dY = torch.randn(M, N, device="cuda")
        dX = torch.empty(M, 128, device="cuda")
        run(qg, p, dY, dX)
        want = dY.double() @ w
        assert float((dX.double() - want).norm()) <= 2e-6 * float(want.norm())  # 48 truncating additions of 1.5e-8, then fp32


def test_special_values(qg):
    """Infinities and NaN of dY stay in their row; large and small rows keep their precision in fp32."""
    p, w = weight(64, 128, "u4", "tensor", 64, 12)
    for x in ("f16", "bf16", "f32"):
        dY = torch.randn(40, 64, device="cuda").to(DT[x])
        dY[3, 5], dY[7, 1] = float("inf"), float("nan")
        dX = torch.empty(40, 128, dtype=DT[x], device="cuda")
        run(qg, p, dY, dX)
        rows = torch.ones(40, dtype=torch.bool, device="cuda")
        rows[3] = rows[7] = False
        assert bool(torch.isfinite(dX[rows]).all()) and bool(dX[7].isnan().all()) and not bool(torch.isfinite(dX[3]).any())
    dY = torch.randn(40, 64, device="cuda") * torch.logspace(-30, 30, 40, device="cuda")[:, None]
    dX = torch.empty(40, 128, device="cuda")
    run(qg, p, dY, dX)
    want = dY.double() @ w
    assert bool(((dX.double() - want).norm(dim=1) <= 1e-5 * want.norm(dim=1)).all())


def test_repeats_are_identical_and_other_streams_work(qg):
    p, w = weight(520, 640, "u2", "uniform", 64, 13)
    for x in ("f16", "f32"):
        dY = torch.randn(300, 520, device="cuda").to(DT[x])
        outs = []
        s = torch.cuda.Stream()
        torch.cuda.synchronize()
        for i in range(4):
            dX = torch.empty(300, 640, dtype=DT[x], device="cuda")
            torch.cuda.synchronize()
            run(qg, p, dY, dX, stream=s if i == 3 else None)
            s.synchronize()
            outs.append(dX)
        assert all(torch.equal(o, outs[0]) for o in outs)


def test_empty_and_refused(qg):
    p, _ = weight(64, 128, "u4", "tensor", 64, 14)
    dX = torch.full((4, 128), 7.0, device="cuda")
    run(qg, p, torch.empty(0, 64, device="cuda"), dX[:0])
    e = torch.empty(0, 64, dtype=torch.uint8, device="cuda"), torch.empty(0, 2, dtype=torch.float16, device="cuda")
    qg.qgemm_nbits_dgrad(torch.empty(4, 0, device="cuda"), e[0], e[1], None, dX, bits=4, block_size=64)
    assert not dX.any()
    dY = torch.zeros(4, 64, device="cuda")
    call = lambda **o: qg.qgemm_nbits_dgrad(o.get("dY", dY), o.get("W", p["W"]), o.get("scales", p["scales"]), None, o.get("dX", dX),
                                            bits=o.get("bits", 4), block_size=o.get("bs", 64), raw=True)
    assert call() == qg.QG_OK
    assert call(bs=16, scales=torch.zeros(64, 8, dtype=torch.float16, device="cuda")) == qg.QG_ERR_UNSUPPORTED
    assert call(bits=5, W=torch.zeros(64, 80, dtype=torch.uint8, device="cuda")) == qg.QG_ERR_UNSUPPORTED
    off = torch.zeros(64 * 64 + 1, dtype=torch.uint8, device="cuda")[1:].view(64, 64)
    assert call(W=off) == qg.QG_ERR_INVALID_ARG
    with pytest.raises(ValueError):
        call(dY=torch.zeros(4, 63, device="cuda"))
    with pytest.raises(ValueError):
        call(dX=torch.zeros(128, 4, device="cuda").t())
