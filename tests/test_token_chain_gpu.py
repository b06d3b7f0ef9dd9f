"""The calls around tokens as programs use them, one behind another on a stream with nothing waited for on the host: a decode
step (router, experts, output projection, log probabilities) and a fine-tuning step (adapters over a frozen output
projection, log probabilities, their gradient, the adapters' gradients, AdamW).  Every stage is right for what the one
before wrote, and results are those of the calls one at a time and of a captured graph."""
import pytest
import torch

import gemm_blockwise_dequant_gb300 as qg
import test_adamw_gpu as adamw
import test_moe_tokens_gpu as moe
import test_token_logprobs_gpu as scores
from lora_util import DT, SUMS
from test_dgrad_gpu import run as dgrad, weight

pytestmark = pytest.mark.gpu


def captured(f):
    f()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f()
    return graph


@pytest.mark.parametrize("T,V,x", [(1, 4000, "f16"), (7, 1001, "bf16"), (40, 8008, "bf16")])
def test_a_decode_step(T, V, x):
    E, k, H, I, bs = 16, 4, 512, 384, 32
    w = moe.layer(E, H, I, 4, bs, zp=True, bias=True, seed=T)
    g = torch.Generator(device="cuda").manual_seed(V)
    head = torch.randint(0, 256, (V, H // 2), generator=g, device="cuda", dtype=torch.uint8)
    head_scales = (torch.rand(V, H // bs, generator=g, device="cuda") * 0.02).half()
    inputs = [(torch.randn(T, H, generator=g, device="cuda").to(DT[x]), torch.randn(T, E, generator=g, device="cuda"),
               torch.randint(-1, V, (T,), generator=g, device="cuda")) for _ in range(3)]
    X, router, target = (torch.empty_like(t) for t in inputs[0])
    ids, weights, y = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda"), torch.empty(T, H, dtype=DT[x], device="cuda")
    Z, stats = torch.empty(T, V, device="cuda"), torch.empty(3, T, device="cuda")
    top_ids, top = torch.empty(T, 5, dtype=torch.int64, device="cuda"), torch.empty(T, 5, device="cuda")
    room = torch.empty(qg.qmoe_tokens_workspace_bytes(T, k, H, I), dtype=torch.uint8, device="cuda")
    outs = [ids, weights, y, Z, stats, top_ids, top]

    def step(wait=False):
        for call in (lambda: qg.qmoe_route_topk(router, ids, weights),
                     lambda: qg.qmoe_tokens_fused(X, ids, weights, **w, bits=4, block_size=bs, y=y, workspace=room),
                     lambda: qg.qgemm_nbits(y, head, head_scales, None, Z, bits=4, block_size=bs),
                     lambda: qg.qg_token_logprobs(Z, target, stats[0], entropy=stats[1], lse=stats[2], top_ids=top_ids, top_logprobs=top, inv_temperature=1.25)):
            call()
            if wait:
                torch.cuda.synchronize()

    def steps(f):
        kept = []
        for i in range(6):
            for to, t in zip((X, router, target), inputs[i % 3]):
                to.copy_(t)
            f()
            kept.append([t.clone() for t in outs])
        torch.cuda.synchronize()
        return kept

    alone = steps(lambda: step(True))
    for f in (step, step, captured(step).replay):
        for a, b in zip(alone, steps(f)):
            assert all(torch.equal(u, v) for u, v in zip(a, b))
    for i in range(3):
        for to, t in zip((X, router, target), inputs[i]):
            to.copy_(t)
        ids, weights, y, Z, stats, top_ids, top = alone[i]
        assert torch.equal(ids.long(), router.double().sort(dim=1, descending=True, stable=True).indices[:, :k])
        moe.check(y, X, ids, weights, w, 4, bs)
        scores.check(Z, target, 1.25, 5, [stats[0], stats[1], stats[2], top_ids, top])


class Tuned:
    """Adapters of rank r over a frozen output projection of vocabulary V, trained on tokens' log probabilities and entropies."""

    def __init__(self, T, V, K, x, seed=0, r=16):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rnd = lambda *s, std=1.0: torch.randn(*s, generator=g, device="cuda") * std
        self.p, self.w64 = weight(V, K, "nf4", "none", 64, seed)
        self.p["absmax"].mul_(2.0 ** -4)  # exact in both
        self.w64 = self.w64 * 2.0 ** -4
        self.X, self.A, self.B = rnd(T, K).to(DT[x]), rnd(1, r, K, std=K ** -0.5).to(DT[x]), rnd(1, V, r, std=0.1).to(DT[x])
        self.scaling = torch.full((1,), 1.5, device="cuda")
        self.offsets, self.ids = torch.tensor([0, T], dtype=torch.int64, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
        self.target = torch.randint(0, V, (T,), generator=g, device="cuda")
        self.target[T // 3] = -100
        self.d_logprob, self.d_entropy = rnd(T, std=1.0 / T), rnd(T, std=0.1 / T)
        self.base, self.Z, self.dZ = torch.empty(T, V, device="cuda"), torch.empty(T, V, device="cuda", dtype=DT[x]), torch.empty(T, V, device="cuda", dtype=DT[x])
        self.U, self.stats, self.dX = torch.empty(T, r, device="cuda"), torch.empty(3, T, device="cuda"), torch.empty_like(self.X)
        self.dA, self.dB, self.norm = torch.empty_like(self.A), torch.empty_like(self.B), torch.empty(1, device="cuda")
        self.step_number = torch.zeros(1, dtype=torch.int64, device="cuda")
        self.master = [self.A.float().flatten(), self.B.float().flatten()]
        self.list = qg.QGAdamWList([self.A.view(-1), self.B.view(-1)], [self.dA.view(-1), self.dB.view(-1)], master=self.master, state="e4m3")

    def state(self):
        t = self.list
        return [self.Z, self.stats, self.dZ, self.dX, self.dA, self.dB, self.norm, self.A, self.B] + self.master + [
            s.view(torch.uint8) for s in t.exp_avg + t.exp_avg_rms + t.exp_avg_scale + t.exp_avg_rms_scale]

    def step(self, wait=False):
        s = self
        for call in (lambda: qg.qgemm_codebook4(s.X, s.p["W"], s.p["codebook"], s.p["absmax"], s.base, block_size=64),
                     lambda: qg.qg_lora_apply(s.X, s.offsets, s.ids, s.A, s.B, s.scaling, s.base, s.Z, V=s.U),
                     lambda: qg.qg_token_logprobs(s.Z, s.target, s.stats[0], entropy=s.stats[1], lse=s.stats[2]),
                     lambda: qg.qg_token_logprobs_grad(s.Z, s.target, s.stats[2], s.d_logprob, s.dZ, entropy=s.stats[1], d_entropy=s.d_entropy),
                     lambda: dgrad(qg, s.p, s.dZ, s.dX),
                     lambda: qg.qg_lora_grad(s.dZ, s.X, s.U, s.offsets, s.ids, s.A, s.B, s.scaling, s.dX, s.dX, s.dA, s.dB),
                     lambda: s.step_number.add_(1),
                     lambda: qg.qg_adamw_step(s.list, lr=adamw.LR, step=s.step_number, betas=adamw.BETAS, eps=adamw.EPS, max_norm=0.01, norm=s.norm)):
            call()
            if wait:
                torch.cuda.synchronize()


@pytest.mark.parametrize("T,V,x", [(5, 1000, "f32"), (70, 2504, "bf16"), (300, 4008, "bf16")])
def test_fine_tuning_steps(T, V, x):
    """Four steps: waited for, not waited for, and replayed."""
    cases = [Tuned(T, V, 256, x) for _ in range(3)]
    graph = captured(cases[2].step)  # has made one step already
    for i in range(4):
        cases[0].step(True)
        cases[1].step()
        if i:
            graph.replay()
        torch.cuda.synchronize()
        for c in cases[1:]:
            assert all(torch.equal(a, b) for a, b in zip(cases[0].state(), c.state()))
    assert int(cases[2].step_number) == 4 and not torch.equal(cases[0].A, Tuned(T, V, 256, x).A)


@pytest.mark.parametrize("T,V", [(6, 504), (40, 1000)])
def test_gradients_of_a_step(T, V):
    """Of the adapters and of the input, against differences of the loss in fp64 along random directions; then the step."""
    c = Tuned(T, V, 128, "f32", seed=3)
    x, A, B = c.X.double(), c.A[0].double(), c.B[0].double()

    def loss(x, A, B):
        logp = torch.log_softmax(x @ c.w64.t() + 1.5 * (x @ A.t()) @ B.t(), dim=1)
        lp = torch.where(c.target >= 0, logp.gather(1, c.target.clamp(min=0)[:, None])[:, 0], 0.0)
        return (c.d_logprob.double() * lp - c.d_entropy.double() * (logp.exp() * logp).sum(1)).sum()

    before = [t.clone() for t in c.master]
    c.step()
    g = torch.Generator(device="cuda").manual_seed(5)
    for i, (got, at) in enumerate(((c.dX, x), (c.dA[0], A), (c.dB[0], B))):
        for _ in range(4):
            d = torch.randn(at.shape, generator=g, device="cuda", dtype=torch.float64)
            h = 1e-5  # the difference is off by h^2 of the third derivative, and 2^-53 / h of the loss
            move = lambda s: [t + s * h * d if j == i else t for j, t in enumerate((x, A, B))]
            slope = (loss(*move(1)) - loss(*move(-1))) / (2 * h)
            # four products, each off by 2^-15 of its terms' magnitudes, which are up to 16 times a sum of 256 of them
            assert abs(float((got.double() * d).sum() - slope)) <= 4 * 16 * SUMS * float((got.double() * d).abs().sum())
    # the first step from states of zero: m / (1 - beta1) is g, v / (1 - beta2) is g^2
    grads = torch.cat([c.dA.flatten(), c.dB.flatten()]).double()
    clip = min(1.0, 0.01 / (float(grads.norm()) + 1e-6))
    for p, old, d in zip(c.master, before, (c.dA, c.dB)):
        d = d.flatten().double() * clip
        want = old.double() - adamw.LR * d / (d.abs() + adamw.EPS)
        # sixteen roundings of the step, four of the value; the second moment is a square (2^-20 more of the step)
        assert ((p.double() - want).abs() <= 2.0 ** -18 * adamw.LR + 2.0 ** -22 * want.abs()).all()
