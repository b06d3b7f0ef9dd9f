"""The mixture-of-experts layer over a few tokens and the choice of its experts, against fp64."""
import math

import pytest
import torch

import gemm_blockwise_dequant_gb300 as qg

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
UNIT = {t: torch.finfo(t).eps / 2 for t in DT.values()}


def layer(E, H, I, bits, bs, zp=False, bias=False, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    top = 0.32 / (1 << bits)
    w = {}
    for name, n, k in (("fc1", 2 * I, H), ("fc2", H, I)):
        w[name + "_w"] = torch.randint(0, 256, (E, n, k * bits // 8), generator=g, device="cuda", dtype=torch.uint8)
        w[name + "_scales"] = (torch.rand(E, n, k // bs, generator=g, device="cuda") * top + 0.2 * top).half()
        # zero points in quarters: no whole numbers
        w[name + "_zp"] = (torch.randint(0, 4 << bits, (E, n, k // bs), generator=g, device="cuda") / 4).half() if zp else None
        w[name + "_bias"] = (torch.randn(E, n, generator=g, device="cuda") * 0.1).half() if bias else None
    return w


def weight64(w, name, e, bits, bs):
    codes, scales, zp = w[name + "_w"][e], w[name + "_scales"][e].double(), w[name + "_zp"]
    q = (codes[..., None] >> torch.arange(0, 8, bits, device="cuda", dtype=torch.uint8)) & ((1 << bits) - 1)
    q = q.reshape(*scales.shape, bs).double()
    z = zp[e].double()[..., None] if zp is not None else float(1 << (bits - 1))
    return ((q - z) * scales[..., None]).flatten(1)


def layer64(x, ids, weights, w, bits, bs, interleaved=0, half=2.0 ** -11):
    """(y, what y may be off before its rounding)."""
    E, H = w["fc1_w"].shape[0], x.shape[1]
    y = torch.zeros(x.shape[0], H, dtype=torch.float64, device="cuda")
    off = torch.zeros_like(y)
    # fp32 sums of a block by the MMAs and of the blocks: 2^-18 of the magnitudes; fp16 of a row: 2^-11 of h (x is exact but
    # where it is 2^-29 of its row's largest); half: of h where it is one fp16
    sums = 2.0 ** -18
    for e in range(E):
        t, j = (ids == e).nonzero(as_tuple=True)
        if t.numel() == 0:
            continue
        a = x[t].double()
        W1, W2 = weight64(w, "fc1", e, bits, bs), weight64(w, "fc2", e, bits, bs)
        b1, b2 = (w[n + "_bias"][e].double() if w[n + "_bias"] is not None else torch.zeros(1, device="cuda", dtype=torch.float64) for n in ("fc1", "fc2"))
        mid = 2.0 ** bits  # the sums are of codes less the midpoint and of zero points less it
        s1 = w["fc1_scales"][e].double().repeat_interleave(bs, dim=1) * mid
        s2 = w["fc2_scales"][e].double().repeat_interleave(bs, dim=1) * mid
        g, eg = a @ W1.t() + b1, sums * (a.abs() @ s1.t())
        n = g.shape[1] // 2
        pick = (lambda v: (v[:, 0::2], v[:, 1::2])) if interleaved else (lambda v: (v[:, :n], v[:, n:]))
        (gate, up), (eg0, eg1) = pick(g), pick(eg)
        act = gate * torch.sigmoid(gate)
        h = act * up
        eh = 1.1 * eg0 * up.abs() + act.abs() * eg1 + half * h.abs() + 2.0 ** -19 * h.abs()
        o, eo = h @ W2.t() + b2, eh @ W2.abs().t() + sums * (h.abs() @ s2.t())
        c = weights[t, j].double()[:, None]
        y.index_add_(0, t, c * o)
        off.index_add_(0, t, c.abs() * (eo + 2.0 ** -21 * o.abs()))
    return y, off


def choose(T, E, k, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    ids = torch.rand(T, E, generator=g, device="cuda").argsort(dim=1)[:, :k].to(torch.int32).contiguous()
    return ids, torch.rand(T, k, generator=g, device="cuda")


def run(x, ids, weights, w, bits, bs, y=None, **more):
    y = torch.full_like(x, float("nan")) if y is None else y
    qg.qmoe_tokens_fused(x, ids, weights, **w, bits=bits, block_size=bs, y=y, **more)
    return y


def check(got, x, ids, weights, w, bits, bs, interleaved=0):
    y, off = layer64(x, ids, weights, w, bits, bs, interleaved)
    off = off + UNIT[got.dtype] * 1.01 * y.abs() + (2.0 ** -25 if got.dtype == torch.float16 else 0)
    assert ((got.double() - y).abs() <= off).all()
    # the bound above is one of the worst case; the typical error is far below
    assert (got.double() - y).norm() <= (4 * UNIT[got.dtype] + 2.0 ** -11) * y.norm()


@pytest.mark.parametrize("bits", [2, 4, 8])
@pytest.mark.parametrize("bs", [32, 64, 128, 256])
@pytest.mark.parametrize("zp,bias", [(False, False), (True, True)])
@pytest.mark.parametrize("T,E,k,x", [(1, 5, 2, "f16"), (7, 8, 3, "bf16"), (30, 6, 4, "f16")])
def test_layer(bits, bs, zp, bias, T, E, k, x):
    H, I = (512, 768) if bs == 256 else (384, 640)
    w = layer(E, H, I, bits, bs, zp, bias, seed=bits + bs)
    g = torch.Generator(device="cuda").manual_seed(T)
    X = torch.randn(T, H, generator=g, device="cuda").to(DT[x])
    ids, weights = choose(T, E, k, seed=T)
    check(run(X, ids, weights, w, bits, bs), X, ids, weights, w, bits, bs)


@pytest.mark.parametrize("H,I,bs", [(32, 32, 32), (96, 32, 32), (32, 160, 32), (64, 64, 64), (2880, 2880, 32), (2048, 768, 64), (608, 1376, 32), (448, 192, 64)])
@pytest.mark.parametrize("bits,x", [(2, "bf16"), (4, "f16"), (8, "f16")])
def test_widths(H, I, bs, bits, x):
    E, k, T = 6, 2, 5
    w = layer(E, H, I, bits, bs, True, False, seed=H)
    X = torch.randn(T, H, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").to(DT[x])
    ids, weights = choose(T, E, k)
    check(run(X, ids, weights, w, bits, bs), X, ids, weights, w, bits, bs)


@pytest.mark.parametrize("T,E,k", [(64, 128, 8), (64, 16, 16), (1, 1, 1), (128, 8, 2), (100, 10, 10), (3, 512, 16), (1024, 4, 1)])
def test_numbers_of_tokens_and_experts(T, E, k):
    w = layer(E, 256, 128, 4, 32, False, True, seed=T)
    X = torch.randn(T, 256, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").bfloat16()
    ids, weights = choose(T, E, k)
    check(run(X, ids, weights, w, 4, 32), X, ids, weights, w, 4, 32)


def test_all_tokens_at_one_expert_and_an_expert_twice():
    w = layer(9, 256, 256, 4, 64, True, True)
    X = torch.randn(61, 256, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").half()
    ids, weights = choose(61, 9, 4)
    ids[:] = 7
    weights[:, 2] = 0
    check(run(X, ids, weights, w, 4, 64), X, ids, weights, w, 4, 64)


@pytest.mark.parametrize("interleaved", [0, 1])
@pytest.mark.parametrize("y", ["f32", "f16", "bf16"])
def test_interleaved_halves_and_types_of_y(interleaved, y):
    w = layer(4, 320, 224, 4, 32, False, True)
    X = torch.randn(9, 320, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").half()
    ids, weights = choose(9, 4, 2)
    out = torch.empty(9, 320, dtype=DT[y], device="cuda")
    check(run(X, ids, weights, w, 4, 32, y=out, swiglu_interleaved=interleaved), X, ids, weights, w, 4, 32, interleaved)


def test_long_rows_take_fewer_rows_at_a_time():
    """An inner width whose rows fit the shared memory one or a few at a time."""
    for H, I, T in ((128, 17920, 20), (17920, 64, 9)):
        w = layer(3, H, I, 4, 64)
        X = torch.randn(T, H, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").bfloat16()
        ids, weights = choose(T, 3, 2)
        check(run(X, ids, weights, w, 4, 64), X, ids, weights, w, 4, 64)


def test_one_token_is_what_the_single_token_decode_gives():
    w = layer(8, 512, 384, 4, 32, True, True)
    X = torch.randn(1, 512, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").half()
    ids, weights = choose(1, 8, 4)
    one = torch.empty(512, dtype=torch.float16, device="cuda")
    qg.qmoe_decode_fused(X[0], ids[0], weights[0], num_experts=8, **w, bits=4, block_size=32, y=one)
    got = run(X, ids, weights, w, 4, 32)[0]
    assert float((got.double() - one.double()).norm() / one.double().norm()) <= 2.0 ** -10


@pytest.mark.parametrize("x", ["f16", "bf16"])
def test_rows_of_any_magnitude_and_rows_that_are_not_finite(x):
    w = layer(4, 256, 192, 4, 32, True)
    X = torch.randn(12, 256, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    scale = torch.tensor([1, 1e-4, 3e3, 1, 1, 0, 1e-7, 1, 1, 1, 1, 1], device="cuda")[:, None]
    if x == "bf16":
        scale[1], scale[2], scale[6] = 1e-30, 1e15, 1e-38
    X = (X * scale).to(DT[x])
    X[3, 10], X[4, 11] = math.inf, math.nan
    X[8, 5] = 60000.0  # the others far below it
    ids, weights = choose(12, 4, 2)
    out = torch.empty(12, 256, device="cuda")
    got = run(X, ids, weights, w, 4, 32, y=out)
    bad = torch.tensor([i in (3, 4) for i in range(12)], device="cuda")
    assert not torch.isfinite(got[bad]).all(dim=1).any()
    fine = [i for i in range(12) if i not in (3, 4)]
    y, off = layer64(X[fine], ids[fine], weights[fine], w, 4, 32)
    # values below 2^-29 of a row's largest are kept to 2^-40 of it
    assert ((got[fine].double() - y).abs() <= off + UNIT[torch.float32] * y.abs() + 1e-38).all()
    assert not got[5].any()


def test_ids_that_are_no_expert():
    w = layer(5, 128, 128, 4, 32)
    X = torch.randn(6, 128, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").half()
    ids, weights = choose(6, 5, 2)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    run(X, ids, weights, w, 4, 32, status=status)
    assert int(status) == 0
    ids[1, 0], ids[2, 0], ids[2, 1], ids[5, 1] = -1, 5, 1 << 20, -(1 << 31)
    got = run(X, ids, weights, w, 4, 32, status=status)
    assert int(status) == 1
    check(got, X, ids, weights, w, 4, 32)
    assert not got[2].any()
    ids[:] = -1
    assert not run(X, ids, weights, w, 4, 32).any()


def test_repeated_captured_and_on_another_stream():
    w = layer(16, 512, 256, 4, 32, True, True)
    X = torch.randn(10, 512, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").half()
    ids, weights = choose(10, 16, 4)
    first = run(X, ids, weights, w, 4, 32)
    for _ in range(3):
        assert torch.equal(first, run(X, ids, weights, w, 4, 32))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = torch.empty_like(X)
    run(X, ids, weights, w, 4, 32, y=y, stream=side)
    side.synchronize()
    assert torch.equal(first, y)
    logits = torch.zeros(10, 16, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qg.qmoe_route_topk(logits, ids, weights)
        run(X, ids, weights, w, 4, 32, y=y)
    for seed in (3, 4):
        logits.normal_(generator=torch.Generator(device="cuda").manual_seed(seed))
        graph.replay()
        again_ids, again_weights = torch.empty_like(ids), torch.empty_like(weights)
        qg.qmoe_route_topk(logits, again_ids, again_weights)
        assert torch.equal(ids, again_ids) and torch.equal(weights, again_weights)
        assert torch.equal(y, run(X, again_ids, again_weights, w, 4, 32))


@pytest.mark.parametrize("x", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,E,k,pad", [(1, 1, 1, 0), (5, 128, 8, 3), (64, 512, 16, 0), (33, 100, 7, 1), (300, 16, 16, 0)])
@pytest.mark.parametrize("renormalize", [False, True])
def test_route(x, T, E, k, pad, renormalize):
    g = torch.Generator(device="cuda").manual_seed(T + E)
    logits = (torch.randn(T, E + pad, generator=g, device="cuda") * 2).to(DT[x])[:, :E]
    logits[0] = 0.25  # ties: the lowest indexes
    ids, weights = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
    qg.qmoe_route_topk(logits, ids, weights, renormalize=renormalize)
    order = logits.double().sort(dim=1, descending=True, stable=True)
    assert torch.equal(ids.long(), order.indices[:, :k])
    want = order.values[:, :k].softmax(dim=1) if renormalize else order.values.softmax(dim=1)[:, :k]
    # an exponential and a quotient, and the sum of up to 512 terms in some twenty additions
    assert ((weights - want).abs() <= 2.0 ** -19 * want).all()


def test_route_of_masked_infinite_and_nan_logits():
    logits = torch.randn(6, 40, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    logits[0, 3:] = -math.inf
    logits[1] = -math.inf
    logits[2, 5] = math.nan
    logits[3, 6] = math.inf
    logits[4] = torch.finfo(torch.float32).min
    logits[5, ::2] = -math.inf
    ids, weights = torch.empty(6, 5, dtype=torch.int32, device="cuda"), torch.empty(6, 5, device="cuda")
    for renormalize in (True, False):
        qg.qmoe_route_topk(logits, ids, weights, renormalize=renormalize)
        assert sorted(ids[0, :3].tolist()) == [0, 1, 2] and ids[0, 3:].tolist() == [3, 4] and not weights[0, 3:].any()
        assert abs(float(weights[0].sum()) - 1) < 1e-6
        assert ids[1].tolist() == [0, 1, 2, 3, 4] and not weights[1].any()
        assert int(ids[2, 0]) == 5 and weights[2].isnan().all()
        assert int(ids[3, 0]) == 6 and weights[3, 0].isnan()
        assert ids[4].tolist() == [0, 1, 2, 3, 4] and torch.allclose(weights[4], torch.full((5,), 0.2 if renormalize else 0.025, device="cuda"))
        assert (ids[5] % 2 == 1).all()


@pytest.mark.parametrize("zp", [False, True])
@pytest.mark.parametrize("bits,bs", [(2, 32), (2, 64), (4, 32), (4, 128), (8, 32), (8, 64)])
@pytest.mark.parametrize("T,E,k", [(1, 3, 2), (5, 4, 3), (9, 3, 3), (40, 5, 2)])
def test_the_inner_activations_keep_their_bits(T, E, k, bits, bs, zp):
    """An fp32 y is as far off as two fp16 terms of h and the sums are, an fp16 y hardly further than its rounding."""
    H, I = 384, 640
    w = layer(E, H, I, bits, bs, zp, True, seed=T)
    X = torch.randn(T, H, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda").half()
    ids, weights = choose(T, E, k, seed=T)
    y, off = layer64(X, ids, weights, w, bits, bs, half=2.0 ** -21)
    got = run(X, ids, weights, w, bits, bs, y=torch.empty(T, H, device="cuda"))
    assert ((got.double() - y).abs() <= off + 2.0 ** -23 * y.abs()).all()
    # sums that are off by no more than 2^-18 of their terms' magnitudes; those are some ten times the sum
    assert (got.double() - y).norm() <= 2.0 ** -14 * y.norm()
    rounded, best = run(X, ids, weights, w, bits, bs), y.half()
    assert (rounded.double() - y).norm() <= 1.05 * (best.double() - y).norm()


def test_long_rows_in_two_terms():
    """Rows of which a pair's two just fit, or one alone does."""
    for I in (17920, 26624, 28672):
        w = layer(3, 128, I, 4, 64)
        X = torch.randn(5, 128, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").half()
        ids, weights = choose(5, 3, 2)
        out = torch.empty(5, 128, device="cuda")
        check(run(X, ids, weights, w, 4, 64, y=out), X, ids, weights, w, 4, 64)
