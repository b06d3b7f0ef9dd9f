"""Log probabilities of given tokens, entropy and alternatives, and the gradient of the logits, against fp64."""
import math

import pytest
import torch

import gemm_blockwise_dequant_gb300 as qg

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
UNIT = {t: torch.finfo(t).eps / 2 for t in DT.values()}


def logits(T, V, x, seed=0, shift=0, pad=0, std=3.0):
    """[T, V] values whose first row begins `shift` values after a 256-byte boundary, rows `pad` values apart."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    flat = (torch.randn(shift + T * (V + pad), generator=g, device="cuda") * std).to(DT[x])
    X = flat[shift:].view(T, V + pad)[:, :V]
    X[torch.arange(T, device="cuda"), torch.randint(0, V, (T,), generator=g, device="cuda")] += 6
    return X, torch.randint(0, V, (T,), generator=g, device="cuda")


def score64(X, target, inv_t):
    z = X.double() * inv_t
    lse = torch.logsumexp(z, dim=1)
    logp = z - lse[:, None]
    p = logp.exp()
    entropy = -torch.where(p > 0, p * logp, 0.0).sum(dim=1)
    lp = torch.where(target >= 0, logp.gather(1, target.clamp(min=0)[:, None])[:, 0], 0.0)
    return lp, entropy, lse, logp


def order64(X, k):
    """Ids of the k largest of each row, the lower index first among equals, NaN above all."""
    x = torch.where(X.isnan(), math.inf, X.double())
    first = torch.sort(X.isnan().int(), dim=1, descending=True, stable=True).indices
    within = torch.sort(x.gather(1, first), dim=1, descending=True, stable=True).indices
    return first.gather(1, within)[:, :k]


def call(X, target, inv_t=1.0, k=0, **more):
    T = X.shape[0]
    out = [torch.full((T,), float("nan"), device="cuda") for _ in range(3)]
    ids = torch.full((T, k), -7, dtype=torch.int64, device="cuda") if k else None
    top = torch.full((T, k), float("nan"), device="cuda") if k else None
    qg.qg_token_logprobs(X, target, out[0], entropy=out[1], lse=out[2], top_ids=ids, top_logprobs=top, inv_temperature=inv_t, **more)
    return out + [ids, top]


def slack(V):
    """Of log S: every addition of a thread's run and of the joins 2^-24 of the sum, every exponential 2^-21."""
    return (V / 512 + 64) * 2.0 ** -24 + 2.0 ** -21


def check(X, target, inv_t, k, got):
    lp, entropy, lse, logp = score64(X, target, inv_t)
    V = X.shape[1]
    # differences of logits and their products with two rounded constants: 3 roundings of the magnitude
    far = lambda t: 4 * 2.0 ** -24 * t.abs().clamp(max=1e30)
    assert ((got[0] - lp).abs() <= slack(V) + far(lp) + far(lp + lse - X.double().amax(1) * inv_t)).all()
    assert ((got[2] - lse).abs() <= slack(V) + far(lse) + far(X.double().amax(1) * inv_t)).all()
    assert ((got[1] - entropy).abs() <= slack(V) * (2 + 2 * entropy) + far(entropy)).all()
    if k:
        ids = order64(X, k)
        assert torch.equal(got[3], ids)
        want = logp.gather(1, ids)
        fine = want > -math.inf
        assert torch.equal(got[4] > -math.inf, fine)
        assert ((got[4] - want).abs()[fine] <= (slack(V) + far(want) + 2.0 ** -22 * (1 + lse.abs())[:, None])[fine]).all()


@pytest.mark.parametrize("x", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,V,k,shift,pad", [(1, 1, 1, 0, 0), (1, 100352, 20, 0, 0), (3, 32003, 64, 1, 0), (70, 5003, 7, 3, 5), (400, 999, 33, 0, 0),
                                             (17, 64, 64, 5, 1), (2, 33000, 0, 0, 8), (305, 20000, 5, 2, 2), (1, 300001, 64, 7, 0), (9, 9, 3, 1, 1)])
def test_forward(x, T, V, k, shift, pad):
    X, target = logits(T, V, x, seed=T + V, shift=shift, pad=pad)
    target[::5] = -100
    check(X, target, 1.25, k, call(X, target, 1.25, k))


@pytest.mark.parametrize("x", ["f32", "bf16"])
@pytest.mark.parametrize("T,V", [(2, 50000), (330, 9001)])
def test_ties_and_order_of_values(x, T, V):
    """Equal logits in their thousands, ascending and descending rows: the list of candidates fills again and again."""
    X, target = logits(T, V, x, seed=3)
    ramp = torch.arange(V, device="cuda", dtype=torch.float32)
    X[0] = 0.5
    X[1] = (ramp / 64).to(DT[x])
    if T > 2:
        X[2] = (-ramp / 8).to(DT[x])
        X[3] = (ramp % 7).to(DT[x])
        X[4] = -0.0
        X[4, 1::2] = 0.0
    for k in (1, 13, 64):
        check(X, target, 1.0, k, call(X, target, 1.0, k))


@pytest.mark.parametrize("x", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T", [1, 400])
def test_masked_rows(x, T):
    V, k = 4099, 20
    X, target = logits(T, V, x, seed=5, shift=1)
    X[:, 11:] = -math.inf           # eleven tokens are allowed: nine alternatives have probability 0
    target[:] = 3
    target[::3] = 4000              # a token that is ruled out: -inf
    got = call(X, target, 1.0, k)
    lp, entropy, lse, logp = score64(X, target, 1.0)
    assert torch.equal(got[0] == -math.inf, target == 4000)
    check(X, torch.full_like(target, 3), 1.0, k, call(X, torch.full_like(target, 3), 1.0, k))
    X[0] = -math.inf                # nothing is left
    got = call(X, target, 1.0, k)
    assert float(got[0][0]) == -math.inf and float(got[1][0]) == 0 and float(got[2][0]) == -math.inf
    assert got[3][0].tolist() == list(range(k)) and (got[4][0] == -math.inf).all()
    got = call(X, torch.full_like(target, -1), 1.0, k)
    assert float(got[0][0]) == 0
    low = torch.finfo(DT[x]).min    # masks of the type's lowest value: as if masked, all of them equal
    X[0] = low
    X[0, 5] = 1.0
    got = call(X, torch.full_like(target, 5), 1.0, k)
    assert float(got[0][0]) == 0 and float(got[1][0]) == 0 and float(got[2][0]) == 1.0
    assert got[3][0].tolist() == [5, 0, 1, 2, 3, 4] + list(range(6, k))
    X[0] = low
    got = call(X, torch.full_like(target, 5), 1.0, k)
    assert abs(float(got[1][0]) - math.log(V)) < 1e-4 and abs(float(got[0][0]) + math.log(V)) < 1e-4


@pytest.mark.parametrize("x", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("offset", [-60000.0, -16384.0, -300.0, 16384.0, 30000.0, 60000.0])
@pytest.mark.parametrize("inv_t", [0.01, 1.0, 50.0])
def test_rows_far_from_zero(x, offset, inv_t):
    """Logits with a common offset, some of them ruled out, at high and low temperatures."""
    X, target = logits(3, 5003, "f32", seed=7)
    X = (X + offset).to(DT[x])
    X[:, ::3] = -math.inf
    target = target // 3 * 3 + 1
    check(X, target.clamp(max=5002), inv_t, 6, call(X, target.clamp(max=5002), inv_t, 6))


@pytest.mark.parametrize("x", ["f32", "f16", "bf16"])
def test_infinite_and_nan_logits(x):
    X, target = logits(6, 10007, x, seed=6)
    X[1, 9000] = math.nan
    X[2, 17] = math.inf
    X[3, 5], X[3, 4] = math.inf, math.nan
    X[4, 3] = -math.inf
    k = 4
    got = call(X, target, 1.0, k)
    assert torch.equal(got[3], order64(X, k))
    bad = torch.tensor([0, 1, 1, 1, 0, 0], dtype=torch.bool, device="cuda")
    for t in (got[0], got[1], got[2], got[4][:, 0]):
        assert torch.equal(t.isnan(), bad)
    fine = ~bad
    check(X[fine], target[fine], 1.0, k, [t[fine] for t in got])


def test_targets_past_the_vocabulary_and_optional_outputs():
    X, target = logits(5, 700, "bf16")
    target[2], target[3] = 700, -(2 ** 40)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    lp = torch.empty(5, device="cuda")
    qg.qg_token_logprobs(X, target, lp, status=status)
    assert int(status) == 1 and float(lp[2]) == 0 and float(lp[3]) == 0
    want = score64(X, target.clamp(max=699), 1.0)[0]
    assert torch.allclose(lp[:2].double(), want[:2], atol=1e-4, rtol=0)
    status.zero_()
    target[2] = 1
    qg.qg_token_logprobs(X, target, lp, status=status)
    assert int(status) == 0
    lse = torch.empty(5, device="cuda")
    qg.qg_token_logprobs(X, None, None, lse=lse)
    assert torch.allclose(lse.double(), torch.logsumexp(X.double(), 1), atol=1e-4, rtol=0)
    qg.qg_token_logprobs(X[:0], target[:0], lp[:0])


@pytest.mark.parametrize("x", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,V,shift,pad,shift_out,ent", [(1, 1, 0, 0, 0, True), (5, 32003, 1, 0, 1, True), (5, 32003, 1, 0, 2, False), (333, 1000, 0, 24, 0, True),
                                                        (2, 100352, 0, 0, 0, False), (40, 77, 3, 1, 3, True)])
def test_gradient(x, T, V, shift, pad, shift_out, ent):
    inv_t = 0.75
    X, target = logits(T, V, x, seed=V, shift=shift, pad=pad)
    target[1::4] = -100
    target[2::9] = V  # past the end: no token
    g = torch.Generator(device="cuda").manual_seed(1)
    d, h = torch.randn(T, generator=g, device="cuda"), torch.randn(T, generator=g, device="cuda")
    d[3::7] = 0
    h[3::7] = 0
    given = (target >= 0) & (target < V)
    clean = torch.where(given, target, -1)
    lp, entropy, lse, logp = score64(X, clean, inv_t)
    lse32, ent32 = lse.float(), entropy.float()
    room = torch.full((shift_out + T * V + 8,), 9.0, dtype=DT[x], device="cuda")
    dX = room[shift_out:shift_out + T * V].view(T, V)
    qg.qg_token_logprobs_grad(X, target, lse32, d, dX, entropy=ent32 if ent else None, d_entropy=h if ent else None, inv_temperature=inv_t)
    p = logp.exp()
    dd = (d.double() * given)[:, None]
    hh = h.double()[:, None] if ent else torch.zeros_like(dd)
    want = inv_t * (dd * (torch.nn.functional.one_hot(clean.clamp(min=0), V) - p) - hh * p * (logp + entropy[:, None]))
    # p: roundings of z (2), of lse as given and of its product, the exponential; then one rounding to the type
    size = inv_t * p * (dd.abs() + hh.abs() * (logp.abs() + entropy[:, None].abs() + 1))
    off = size * (2.0 ** -20 + 2.0 ** -22 * (logp.abs() + lse.abs()[:, None])) + UNIT[DT[x]] * want.abs() * 1.01 + 2.0 ** -24 * dd.abs() + (2.0 ** -25 if x == "f16" else 2.0 ** -120)
    assert ((dX.double() - want).abs() <= off).all()
    assert (room[:shift_out] == 9).all() and (room[shift_out + T * V:] == 9).all()
    zero = (d * given == 0) & ((h == 0) if ent else torch.ones_like(given))
    assert not dX[zero].any()
    if shift == shift_out and pad == 0:  # into the logits themselves
        qg.qg_token_logprobs_grad(X, target, lse32, d, X, entropy=ent32 if ent else None, d_entropy=h if ent else None, inv_temperature=inv_t)
        assert torch.equal(X, dX)


def test_gradient_against_differences():
    """Of sum d logprob + h entropy as the forward pass computes it, along random directions."""
    T, V, inv_t = 12, 500, 1.3
    X, target = logits(T, V, "f32", seed=9, std=1.0)
    g = torch.Generator(device="cuda").manual_seed(2)
    d, h, along = (torch.randn(*s, generator=g, device="cuda") for s in ((T,), (T,), (T, V)))
    lp, entropy, lse, _, _ = call(X, target, inv_t)
    dX = torch.empty_like(X)
    qg.qg_token_logprobs_grad(X, target, lse, d, dX, entropy=entropy, d_entropy=h, inv_temperature=inv_t)
    step = 2.0 ** -7
    value = lambda s: sum(w.double() * v.double() for w, v in zip((d, h), call(X + s * along, target, inv_t)[:2]))
    slope = (value(step) - value(-step)) / (2 * step)
    want = (dX.double() * along.double()).sum(dim=1)
    # a third derivative of some tens times step^2 / 6, and forward roundings over the step
    assert ((slope - want).abs() <= 40 * step ** 2 / 6 * 8 + 2.0 ** -18 / step).all()
    assert ((slope - want).norm() <= 0.02 * want.norm())


def test_gradient_of_masked_infinite_and_nan_rows():
    X, target = logits(6, 3001, "bf16", seed=4)
    X[0] = -math.inf
    X[1, 100:] = -math.inf
    X[2, 5] = math.nan
    X[3, 5] = math.nan
    target[:] = 7
    target[3] = -1
    lp, entropy, lse, _, _ = call(X, target)
    d, h = torch.ones(6, device="cuda"), torch.full((6,), 0.5, device="cuda")
    h[3] = 0
    dX = torch.full_like(X, 5.0)
    qg.qg_token_logprobs_grad(X, target, lse, d, dX, entropy=entropy, d_entropy=h)
    assert not dX[0].any() and not dX[1, 100:].any() and dX[2].isnan().all() and not dX[3].any()
    assert torch.isfinite(dX[[1, 4, 5]]).all() and dX[1, :100].any()


def test_long_rows_far_apart():
    """Rows whose distance passes 2^31 values, and a row of over 2^24 of them."""
    flat = torch.zeros(2 ** 31 + 70000, dtype=torch.bfloat16, device="cuda")
    X = flat.as_strided((2, 60000), (2 ** 31 + 8, 1))
    v, target = logits(2, 60000, "bf16", seed=8)
    X.copy_(v)
    check(X, target, 1.0, 5, call(X, target, 1.0, 5))
    lp, entropy, lse, _, _ = call(X, target)
    dX = torch.empty(2, 60000, dtype=torch.bfloat16, device="cuda")
    qg.qg_token_logprobs_grad(X, target, lse, torch.ones(2, device="cuda"), dX)
    again = torch.empty_like(dX)
    qg.qg_token_logprobs_grad(v, target, lse, torch.ones(2, device="cuda"), again)
    assert torch.equal(dX, again)
    del flat, X
    X, target = logits(1, 2 ** 24 + 3, "f16", seed=2)
    check(X, target, 1.0, 64, call(X, target, 1.0, 64))


def test_repeated_captured_and_on_another_stream():
    X, target = logits(5, 40001, "bf16", seed=1)
    first = call(X, target, 1.0, 9)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(first, call(X, target, 1.0, 9)))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = call(X, target, 1.0, 9, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, got))
    out, dX, d = torch.empty(2, 5, device="cuda"), torch.empty_like(X), torch.ones(5, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qg.qg_token_logprobs(X, target, out[0], lse=out[1])
        qg.qg_token_logprobs_grad(X, target, out[1], d, dX)
    X.copy_(logits(5, 40001, "bf16", seed=2)[0])
    graph.replay()
    want, again = call(X, target), torch.empty_like(X)
    qg.qg_token_logprobs_grad(X, target, want[2], d, again)
    assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[2]) and torch.equal(dX, again)


@pytest.mark.parametrize("limit", [1, 4, 8])
def test_narrower_clusters(limit):
    X, target = logits(2, 100352, "f32", seed=3)
    before = qg.qg_test_cluster_limit(limit)
    try:
        check(X, target, 1.0, 20, call(X, target, 1.0, 20))
    finally:
        qg.qg_test_cluster_limit(before)


@pytest.mark.parametrize("limit", [1, 2, 4, 8])
@pytest.mark.parametrize("T,k", [(1, 20), (3, 64), (30, 5), (70, 0)])
def test_rows_shared_by_fewer_ctas(limit, T, k):
    """As many CTAs to a row as the device gives them."""
    X, target = logits(T, 60000, "bf16", seed=T)
    before = qg.qg_test_cluster_limit(limit)
    try:
        check(X, target, 0.9, k, call(X, target, 0.9, k))
    finally:
        qg.qg_test_cluster_limit(before)
