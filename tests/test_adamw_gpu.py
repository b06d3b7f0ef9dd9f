"""One AdamW step over lists of tensors against fp64: types, 8-bit states, clipping, odd sizes and addresses."""
import math

import pytest
import torch

import gemm_blockwise_dequant_gb300 as qg

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
UNIT = {t: torch.finfo(t).eps / 2 for t in DT.values()}
LR, BETAS, EPS = 2e-3, (0.9, 0.999), 1e-8
BLOCK = qg.QG_STATE_BLOCK


def shifted(t, shift):
    """The same values `shift` values after a 256-byte boundary."""
    room = torch.zeros(t.numel() + shift + 64, dtype=t.dtype, device="cuda")
    room[shift:shift + t.numel()] = t
    return room[shift:shift + t.numel()]


def codes(x, keep=False):
    """e4m3 codes and scales of random states, by blocks."""
    n = x.numel()
    b = torch.nn.functional.pad(x, (0, -n % BLOCK)).view(-1, BLOCK)
    scale = b.abs().amax(1) / 448
    c = (b / scale.clamp(min=1e-38)[:, None]).to(torch.float8_e4m3fn).view(-1)[:n].contiguous()
    return c, scale


def values(c, scale):
    return c.double() * scale.double().repeat_interleave(BLOCK)[:c.numel()]


class Case:
    def __init__(self, sizes, p="f32", g="f32", state="f32", master=False, shift=0, seed=0, gstd=1e-2):
        r = torch.Generator(device="cuda").manual_seed(seed)
        rnd = lambda n, std: torch.randn(n, generator=r, device="cuda") * std
        self.state, self.sizes = state, sizes
        w = [rnd(n, 0.1) for n in sizes]
        self.p = [shifted(t.to(DT[p]), shift) for t in w]
        self.master = [shifted(t, shift) for t in w] if master else None
        self.g = [shifted(rnd(n, gstd).to(DT[g]), shift) for n in sizes]
        m, v = [rnd(n, 1e-2) for n in sizes], [rnd(n, 1e-2).square() for n in sizes]
        if state == "f32":
            self.states = dict(exp_avg=[shifted(t, shift) for t in m], exp_avg_sq=[shifted(t, shift) for t in v])
        else:
            mc, uc = [codes(t) for t in m], [codes(t.sqrt()) for t in v]
            self.states = dict(exp_avg=[shifted(c, shift) for c, _ in mc], exp_avg_scale=[s for _, s in mc], exp_avg_rms=[shifted(c, shift) for c, _ in uc],
                               exp_avg_rms_scale=[s for _, s in uc])
        self.list = qg.QGAdamWList(self.p, self.g, master=self.master, weight_decay=0.1, **self.states)

    def moments(self, i):
        s = self.states
        if self.state == "f32":
            return s["exp_avg"][i].double(), s["exp_avg_sq"][i].double()
        return values(s["exp_avg"][i], s["exp_avg_scale"][i]), values(s["exp_avg_rms"][i], s["exp_avg_rms_scale"][i]) ** 2


def step64(c, step, max_norm=None, lr=LR, decay=0.1):
    """[(p', m', v', size of the update)] and the norm."""
    norm = math.sqrt(sum(float(g.double().square().sum()) for g in c.g))
    coef = 1.0 if max_norm is None else min(1.0, max_norm / (norm + 1e-6))
    out = []
    for i in range(len(c.sizes)):
        m, v = c.moments(i)
        g = c.g[i].double() * coef
        m, v = BETAS[0] * m + (1 - BETAS[0]) * g, BETAS[1] * v + (1 - BETAS[1]) * g * g
        p = (c.master if c.master else c.p)[i].double()
        move = lr * (m / (1 - BETAS[0] ** step)) / ((v / (1 - BETAS[1] ** step)).sqrt() + EPS)
        size = lr * (BETAS[0] * c.moments(i)[0].abs() + (1 - BETAS[0]) * g.abs()) / (1 - BETAS[0] ** step) / ((v / (1 - BETAS[1] ** step)).sqrt() + EPS)
        out.append((p * (1 - lr * decay) - move, m, v, size))
    return out, norm


def check(c, want):
    for i, (p, m, v, size) in enumerate(want):
        near = lambda got, x, off: bool(((got.double() - x).abs() <= off).all())
        # every product, sum, quotient and root 2^-24 of its value; sixteen of them
        exact = 2.0 ** -20 * size + 2.0 ** -22 * p.abs()
        assert near(c.p[i], p, exact + UNIT[c.p[i].dtype] * 1.01 * p.abs() + (2.0 ** -25 if c.p[i].dtype == torch.float16 else 0))
        if c.master:
            assert near(c.master[i], p, exact)
            assert torch.equal(c.p[i], c.master[i].to(c.p[i].dtype))
        got_m, got_v = c.moments(i)
        if c.state == "f32":
            assert near(got_m, m, 2.0 ** -21 * (m.abs() + 1e-3)) and near(got_v, v, 2.0 ** -21 * v)
        else:  # half a step of e4m3: 2^-4 of the value, or of its smallest normal value 2^-6 in units of the scale
            n = m.numel()
            for got, x in ((got_m, m), (got_v.sqrt(), v.sqrt())):
                top = torch.nn.functional.pad(x.abs(), (0, -n % BLOCK)).view(-1, BLOCK).amax(1).repeat_interleave(BLOCK)[:n]
                off = 2.0 ** -4 * 1.001 * x.abs() + 2.0 ** -10 * 1.001 * top / 448
                keep = (x.abs() < 2.0 ** -9 * top / 448) & (x > 0)  # kept above zero
                assert near(got[~keep], x[~keep], off[~keep])
                assert near(got[keep], x[keep], 2.0 ** -9 * 1.001 * top[keep] / 448)
            assert bool((got_v[v > 0] > 0).all())


SIZES = [1, 7, 8, 255, 256, 257, 2048, 2049, 0, 4096, 4097, 5000, 70001]


@pytest.mark.parametrize("state", ["f32", "e4m3"])
@pytest.mark.parametrize("p,g,master", [("f32", "f32", False), ("bf16", "bf16", False), ("f16", "f32", False), ("bf16", "bf16", True), ("f16", "f16", True), ("f32", "bf16", False)])
@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("max_norm", [None, 0.5])
def test_step(state, p, g, master, shift, max_norm):
    c = Case(SIZES, p, g, state, master, shift, seed=3)
    want, norm64 = step64(c, 5, max_norm)
    norm = torch.full((1,), -3.0, device="cuda")
    qg.qg_adamw_step(c.list, lr=LR, step=5, betas=BETAS, eps=EPS, max_norm=max_norm, norm=norm)
    check(c, want)
    # sums of eight squares in fp32, the rest in fp64
    assert float(norm) == -3.0 if max_norm is None else abs(float(norm) / norm64 - 1) <= 2.0 ** -21


@pytest.mark.parametrize("state", ["f32", "e4m3"])
def test_many_steps_from_zero_states(state):
    """Ten steps with states made by the list: as fp64 from what the step before left."""
    c = Case([3000, 17], "f32", "f32", "f32", seed=1)
    c.list = qg.QGAdamWList(c.p, c.g, weight_decay=[0.1, 0.1], state=state)
    c.state = state
    c.states = {k: getattr(c.list, k) for k in ("exp_avg", "exp_avg_sq", "exp_avg_scale", "exp_avg_rms", "exp_avg_rms_scale")}
    for step in range(1, 11):
        for g in c.g:
            g.mul_(-0.7)
        want, _ = step64(c, step)
        qg.qg_adamw_step(c.list, lr=LR, step=step, betas=BETAS, eps=EPS)
        check(c, want)


def test_many_and_large_tensors():
    c = Case([40 + 13 * i for i in range(700)] + [9_000_001], "bf16", "bf16", "e4m3", seed=2)
    want, norm64 = step64(c, 3, 1.0)
    norm = torch.empty(1, device="cuda")
    qg.qg_adamw_step(c.list, lr=LR, step=3, betas=BETAS, eps=EPS, max_norm=1.0, norm=norm)
    check(c, want)
    assert abs(float(norm) / norm64 - 1) <= 2.0 ** -21


def test_states_of_both_kinds_in_one_list():
    a, b = Case([5000], "bf16", "bf16", "f32", seed=4), Case([5000], "bf16", "f32", "e4m3", seed=5)
    none = [None]
    both = qg.QGAdamWList(a.p + b.p, a.g + b.g, weight_decay=0.1, exp_avg=a.states["exp_avg"] + b.states["exp_avg"], exp_avg_sq=a.states["exp_avg_sq"] + none,
                          exp_avg_scale=none + b.states["exp_avg_scale"], exp_avg_rms=none + b.states["exp_avg_rms"], exp_avg_rms_scale=none + b.states["exp_avg_rms_scale"])
    wa, wb = step64(a, 2)[0], step64(b, 2)[0]
    qg.qg_adamw_step(both, lr=LR, step=2, betas=BETAS, eps=EPS)
    check(a, wa)
    check(b, wb)


@pytest.mark.parametrize("gstd,dtype", [(1e-25, "f32"), (1e22, "f32"), (3e-7, "f16")])
def test_norm_of_small_and_large_gradients(gstd, dtype):
    c = Case([5000, 300], "f32", dtype, "f32", seed=6, gstd=gstd)
    norm = torch.empty(1, device="cuda")
    norm64 = step64(c, 1)[1]
    qg.qg_adamw_step(c.list, lr=LR, step=1, betas=BETAS, max_norm=1.0, norm=norm)
    assert abs(float(norm) / norm64 - 1) <= 2.0 ** -21


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("state", ["f32", "e4m3"])
def test_a_norm_that_is_not_finite_leaves_everything(bad, state):
    c = Case([3000, 500], "bf16", "bf16", state, master=True, seed=7)
    c.g[1][77] = bad
    tensors = c.p + c.master + [t for v in c.states.values() for t in v]
    before = [t.clone() for t in tensors]
    norm = torch.zeros(1, device="cuda")
    qg.qg_adamw_step(c.list, lr=LR, step=1, betas=BETAS, max_norm=1.0, norm=norm)
    assert not math.isfinite(float(norm))
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(before, tensors))


def test_a_nan_gradient_without_clipping_stays_in_its_block():
    c = Case([2000], "f32", "f32", "e4m3", seed=8)
    c.g[0][300] = math.nan
    want, _ = step64(c, 1)
    qg.qg_adamw_step(c.list, lr=LR, step=1, betas=BETAS, eps=EPS)
    assert torch.equal(c.p[0].isnan(), want[0][0].isnan()) and int(c.p[0].isnan().sum()) == 1
    m, v = c.moments(0)
    outside = torch.ones(2000, dtype=torch.bool, device="cuda")
    outside[256:512] = False
    assert torch.isfinite(m[outside]).all() and torch.isfinite(v[outside]).all() and m[300].isnan()


def test_zero_gradients_and_small_second_moments():
    """A root of the second moment far below its block's largest stays above zero, so no later step divides by eps alone."""
    p = torch.zeros(512, device="cuda")
    g = torch.full((512,), 1e-7, device="cuda")
    g[0] = g[256] = 1.0
    t = qg.QGAdamWList([p], [g], state="e4m3")
    qg.qg_adamw_step(t, lr=1.0, step=1, eps=1e-12)
    g.zero_()
    for step in range(2, 6):
        before = p.clone()
        qg.qg_adamw_step(t, lr=1.0, step=step, eps=1e-12)
        assert float((p - before).abs().max()) <= 2.0
    assert bool((t.exp_avg_rms[0].float() > 0).all())


def test_step_and_rate_from_device_memory_in_a_graph():
    a, b = Case([70001, 33], "bf16", "bf16", "e4m3", seed=9), Case([70001, 33], "bf16", "bf16", "e4m3", seed=9)
    lr, step = torch.full((1,), LR, device="cuda"), torch.zeros(1, dtype=torch.int64, device="cuda")
    norm = torch.empty(2, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step.add_(1)
        qg.qg_adamw_step(a.list, lr=lr, step=step, betas=BETAS, eps=EPS, max_norm=0.3, norm=norm[:1])
    step.zero_()
    for i in range(1, 4):
        lr.fill_(LR / i)
        graph.replay()
        qg.qg_adamw_step(b.list, lr=float(torch.tensor(LR / i, dtype=torch.float32)), step=i, betas=BETAS, eps=EPS, max_norm=0.3, norm=norm[1:])
        assert float(norm[0]) == float(norm[1])
        for x, y in zip(a.p + a.states["exp_avg"] + a.states["exp_avg_rms"], b.p + b.states["exp_avg"] + b.states["exp_avg_rms"]):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_on_another_stream_and_without_tensors():
    c = Case([5000], "f32", "f32", "f32", seed=3)
    want, _ = step64(c, 1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    qg.qg_adamw_step(c.list, lr=LR, step=1, betas=BETAS, eps=EPS, stream=side)
    side.synchronize()
    check(c, want)
    norm = torch.ones(1, device="cuda")
    qg.qg_adamw_step(qg.QGAdamWList([], []), lr=LR, step=1, max_norm=1.0, norm=norm)
    assert float(norm) == 0


@pytest.mark.parametrize("state", ["f32", "e4m3"])
@pytest.mark.parametrize("max_norm,norm_eps,zero", [(0.0, 0.0, True), (0.0, 1e-6, True), (1.0, 0.0, True), (0.0, 1e-6, False), (math.inf, 0.0, False)])
def test_clipping_of_nothing_to_nothing_and_by_any_bound(state, max_norm, norm_eps, zero):
    """Gradients of zero, and bounds of zero and infinity: the moments decay, and gradients enter by 0 or as they are."""
    c = Case([3000, 17], "f32", "f32", state, seed=10)
    if zero:
        for g in c.g:
            g.zero_()
    want, _ = step64(c, 3, None if max_norm > 0 or zero else 0.0)
    norm = torch.empty(1, device="cuda")
    qg.qg_adamw_step(c.list, lr=LR, step=3, betas=BETAS, eps=EPS, max_norm=max_norm, norm_eps=norm_eps, norm=norm)
    check(c, want)
    assert (float(norm) == 0) == zero
