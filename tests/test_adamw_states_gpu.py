"""8-bit states of the AdamW step, code for code and scale for scale, against the formula in fp32 operations of torch, each
rounded by itself: a code that goes to its neighbour is up to 7% of its value, and the largest of a block decides its scale.
What is not finite, and what is zero, beside that."""
import math

import pytest
import torch

import gemm_blockwise_dequant_gb300 as qg
from test_adamw_gpu import BETAS, BLOCK, EPS, LR, SIZES, Case

pytestmark = pytest.mark.gpu
NAMES = ("exp_avg", "exp_avg_scale", "exp_avg_rms", "exp_avg_rms_scale")


def blocks(x):
    return torch.nn.functional.pad(x, (0, -x.numel() % BLOCK)).view(-1, BLOCK)


def decoded(c, scale):
    return c.float() * scale.repeat_interleave(BLOCK)[:c.numel()]


def coded(x, keep):
    """(codes, scales) of x; keep: what is above zero stays above."""
    b = blocks(x)
    top = b.abs().amax(1, keepdim=True)
    big = top >= 1e-30
    c = b * torch.where(big, 448.0 / top, 0.0)
    if keep:
        c = torch.where((c > 0) & (c < 2.0 ** -9), 2.0 ** -9, c)
    return c.to(torch.float8_e4m3fn).view(-1)[:x.numel()], torch.where(big, top / 448, 0.0).view(-1)


def moments32(g, m, u):
    return BETAS[0] * m + (1 - BETAS[0]) * g, (BETAS[1] * u.square() + (1 - BETAS[1]) * g.square()).sqrt()


def same(got, want):
    return torch.equal(got.float(), want.float())  # a zero of either sign


def restated(c, max_norm=None, norm=None):
    """What the states of a Case become, from what they and its gradients are."""
    s = c.states
    coef = 1.0 if max_norm is None else (max_norm / (norm + 1e-6)).clamp(max=1.0)
    out = []
    for i, g in enumerate(c.g):
        m, u = moments32(g.float() * coef, decoded(s["exp_avg"][i], s["exp_avg_scale"][i]), decoded(s["exp_avg_rms"][i], s["exp_avg_rms_scale"][i]))
        out.append(coded(m, False) + coded(u, True))
    return out


@pytest.mark.parametrize("p,g,master", [("bf16", "bf16", False), ("f16", "f16", False), ("f32", "f32", False), ("bf16", "f32", True), ("f16", "bf16", False)])
@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("max_norm", [None, 0.5])
def test_ten_steps_each_from_what_the_one_before_left(p, g, master, shift, max_norm):
    """Every way through the kernel: whole vectors and odd addresses, chunks ahead and tails."""
    c = Case(SIZES + [600_011], p, g, "e4m3", master, shift, seed=11)
    norm = torch.empty(1, device="cuda")
    for step in range(1, 11):
        before = Case.__new__(Case)
        before.g, before.states = c.g, {k: [t.clone() for t in v] for k, v in c.states.items()}
        qg.qg_adamw_step(c.list, lr=LR, step=step, betas=BETAS, eps=EPS, max_norm=max_norm, norm=norm)
        for i, want in enumerate(restated(before, max_norm, norm)):
            for name, w in zip(NAMES, want):
                assert same(c.states[name][i], w), (step, i, name)
        for t in c.g:
            t.mul_(-0.7)


@pytest.mark.parametrize("heavy", [False, True])
def test_twelve_steps_apart_from_each_other(heavy):
    """Eight million values from states of zero, gradients anew each step: the states as kept by the kernel and by the formula are the same at the end."""
    n = 1 << 23
    r = torch.Generator(device="cuda").manual_seed(5)
    g, p = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    t = qg.QGAdamWList([p], [g], state="e4m3")
    mc, ms, uc, us = (getattr(t, k)[0].clone() for k in NAMES)
    for step in range(1, 13):
        g.normal_(generator=r).mul_(1e-3)
        if heavy:
            g.mul_(torch.randn(n, generator=r, device="cuda").exp())
        qg.qg_adamw_step(t, lr=LR, step=step, betas=BETAS, eps=EPS)
        m, u = moments32(g, decoded(mc, ms), decoded(uc, us))
        (mc, ms), (uc, us) = coded(m, False), coded(u, True)
    for name, want in zip(NAMES, (mc, ms, uc, us)):
        assert same(getattr(t, name)[0], want), name


def test_scales_are_a_448th_of_the_largest():
    """Every product, sum, root and quotient of a scale rounds once: seven of 2^-24."""
    c = Case([300_007], "bf16", "bf16", "e4m3", seed=12)
    m, v = c.moments(0)
    g = c.g[0].double()
    m, u = BETAS[0] * m + (1 - BETAS[0]) * g, (BETAS[1] * v + (1 - BETAS[1]) * g * g).sqrt()
    size = BETAS[0] * c.moments(0)[0].abs() + (1 - BETAS[0]) * g.abs()  # the terms of m' may cancel
    qg.qg_adamw_step(c.list, lr=LR, step=7, betas=BETAS, eps=EPS)
    for x, s, most in ((m, c.states["exp_avg_scale"][0], size), (u, c.states["exp_avg_rms_scale"][0], u)):
        assert ((s.double() - blocks(x).abs().amax(1) / 448).abs() <= 2.0 ** -21 * blocks(most).amax(1) / 448).all()


@pytest.mark.parametrize("state", ["f32", "e4m3"])
def test_gradients_that_are_not_finite_or_square_to_infinity(state):
    """Without clipping.  A second moment past fp32's range leaves the decay alone; what is NaN is so in its own value."""
    g = torch.randn(2000, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda")
    g[10], g[300], g[301], g[800], g[1500] = 1e20, math.nan, 0.0, math.inf, -3e38
    p = torch.linspace(1.0, 2.0, 2000, device="cuda")
    before = p.clone()
    t = qg.QGAdamWList([p], [g], weight_decay=0.1, state=state)
    qg.qg_adamw_step(t, lr=LR, step=1, betas=BETAS, eps=EPS)
    m = (1 - BETAS[0]) * g
    v = (1 - BETAS[1]) * g.square()
    want = before.double() * (1 - LR * 0.1) - LR * (m / (1 - BETAS[0])).double() / ((v / (1 - BETAS[1])).sqrt().double() + EPS)
    assert torch.equal(p.isnan(), want.isnan()) and p.isnan().nonzero().flatten().tolist() == [300, 800]
    fine = ~want.isnan()
    assert ((p.double() - want)[fine].abs() <= 2.0 ** -18 * LR + 2.0 ** -22 * want[fine].abs()).all()
    if state == "f32":
        assert torch.equal(t.exp_avg[0].isnan(), m.isnan()) and torch.equal(t.exp_avg_sq[0].isinf(), v.isinf())
    else:
        for name, scale, hit in (("exp_avg", "exp_avg_scale", {1, 3}), ("exp_avg_rms", "exp_avg_rms_scale", {0, 1, 3, 5})):
            x = decoded(getattr(t, name)[0], getattr(t, scale)[0])
            assert {i for i in range(8) if not torch.isfinite(x[256 * i:256 * i + 256]).all()} == hit


@pytest.mark.parametrize("state", ["f32", "e4m3"])
def test_second_moments_from_nothing_to_the_largest(state):
    """Blocks of one magnitude each, from squares that are no normal fp32 any more: an update is lr, or m' over eps where eps is above the root."""
    n = 256 * 60
    size = 2.0 ** torch.linspace(-70, 63, 60, device="cuda").round().repeat_interleave(256)
    g = size * torch.where(torch.rand(n, generator=torch.Generator(device="cuda").manual_seed(4), device="cuda") < 0.5, -1.0, 1.0)
    p = torch.zeros(n, device="cuda")
    t = qg.QGAdamWList([p], [g], state=state)
    qg.qg_adamw_step(t, lr=LR, step=1, betas=BETAS, eps=EPS)
    # (1 - beta2) g^2 below 2^-126 counts as 0
    root = torch.where((1 - BETAS[1]) * g.double().square() >= 2.0 ** -126, g.double().abs(), 0.0)
    want = -LR * g.double() / (root + EPS)
    assert ((p.double() - want).abs() <= 2.0 ** -20 * want.abs()).all()
