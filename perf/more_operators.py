"""Operators around the quantized projections that decode and fine-tuning loops need next, as measured cases.

  score   log probabilities of given tokens from the logits of the last projection, with the entropy of each row and
          its k most probable alternatives
  loss    the gradient of the logits from those of the log probabilities and of the entropies
  adamw   one AdamW step over all the tensors that a program trains, with states in fp32 or in 8 bits and, where a
          case says so, the clipping of the gradients by their norm in the same call
  moe     a whole mixture-of-experts layer over a few tokens: the k experts of each token from its router logits, then
          both quantized projections of those experts with SwiGLU between them, weighted and added

``run`` computes them with elementary torch operations in fp32, rounded once at the end, or, where ``own`` is true,
with the calls that a user makes of this package.  ``exact`` computes them in fp64.
"""
import math

import torch

own = False

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}

# AdamW: the usual constants, and a state after a hundred steps
LR, BETA1, BETA2, EPS, DECAY, STEP = 1e-4, 0.9, 0.999, 1e-8, 0.01, 101
MAX_NORM, NORM_EPS = 1.0, 1e-6
BLOCK = 256       # values that share a scale in 8-bit states
E4M3_MAX = 448.0  # the largest value of the 8-bit type

# (N, K) of the projections of a transformer layer with hidden 5120 and intermediate 17920
LAYER = ((7680, 5120), (5120, 5120), (35840, 5120), (5120, 17920))


# ------------------------------------------------------------------------------------------------ the cases
def listed():
    return [
        # one decoded token behind an fp32 output projection, with the twenty alternatives that an API reports
        dict(name="score 1 token", op="score", rows=1, vocab=100352, x="f32", top=20, mask=0.0),
        # a decode step of 64 users under a grammar that rules nine tokens of ten out
        dict(name="score 64 masked", op="score", rows=64, vocab=100352, x="bf16", top=5, mask=0.9),
        # scoring whole prompts, no alternatives: the forward pass of a loss as well
        dict(name="score 4096", op="score", rows=4096, vocab=100352, x="bf16", top=0, mask=0.0),
        # a short fine-tuning sample, vocabulary of odd width
        dict(name="loss 333", op="loss", rows=333, vocab=32003, x="f16", entropy=False),
        # a large batch of a policy update, with an entropy bonus
        dict(name="loss 4096", op="loss", rows=4096, vocab=100352, x="bf16", entropy=True),
        # the adapters of one layer, everything in fp32
        dict(name="adamw layer", op="adamw", layers=1, rank=16, full=0, odd=0, p="f32", g="f32", state="f32", master=False, clip=False),
        # the adapters of a 40-layer model, 8-bit states, clipped
        dict(name="adamw adapters", op="adamw", layers=40, rank=16, full=0, odd=40, p="bf16", g="bf16", state="e4m3", master=False, clip=True),
        # adapters and six whole weight matrices trained beside them, fp32 states and master weights
        dict(name="adamw full", op="adamw", layers=40, rank=64, full=6, odd=0, p="bf16", g="bf16", state="f32", master=True, clip=True),
        # one token through a small layer of eight experts: latency
        dict(name="moe 1 token", op="moe", tokens=1, experts=8, k=2, hidden=1024, inter=768, bits=2, block=64, x="f16", zp=False, bias=False),
        # two tokens of a decode step through 128 experts
        dict(name="moe 2 tokens", op="moe", tokens=2, experts=128, k=8, hidden=2880, inter=2880, bits=4, block=32, x="f16", zp=False, bias=True),
        # sixteen drafted tokens being verified, zero points
        dict(name="moe 16 tokens", op="moe", tokens=16, experts=128, k=8, hidden=2048, inter=768, bits=4, block=64, x="bf16", zp=True, bias=False),
        # a decode step of 64 users: nearly every expert has rows
        dict(name="moe 64 tokens", op="moe", tokens=64, experts=128, k=8, hidden=2880, inter=2880, bits=4, block=32, x="bf16", zp=False, bias=True),
    ]


def _log(rng, lo, hi, step=1):
    return step * int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("score", "loss", "adamw", "moe"))
    x = rng.choice(("f32", "f16", "bf16"))
    if op in ("score", "loss"):
        vocab = _log(rng, 500, 12544, 8) if rng.random() < 0.6 else _log(rng, 1000, 100000)
        rows = _log(rng, 1, 4096 if x != "f32" else 2048)
        if op == "loss":
            return dict(op=op, rows=rows, vocab=vocab, x=x, entropy=rng.random() < 0.5)
        return dict(op=op, rows=rows, vocab=vocab, x=x, top=rng.choice((0, 1, 5, 8, 20, 32)), mask=rng.choice((0.0, 0.0, 0.5, 0.95)))
    if op == "adamw":
        p = x
        return dict(op=op, layers=_log(rng, 1, 40), rank=rng.choice((4, 8, 12, 16, 32, 64)), full=rng.choice((0, 0, 1, 2)),
                    odd=rng.choice((0, 1, 30)), p=p, g=rng.choice((p, "f32")), state=rng.choice(("f32", "e4m3")),
                    master=p != "f32" and rng.random() < 0.4, clip=rng.random() < 0.6)
    bits = rng.choice((2, 4, 4, 4, 8))
    block = rng.choice((32, 64, 128))
    experts = rng.choice((4, 8, 16, 32, 64, 100, 128))
    hidden, inter = _log(rng, 4, 40, 128), _log(rng, 3, 40, 128)
    while experts * hidden * inter > 128 * 2880 * 2880:
        experts = experts // 2
    return dict(op=op, tokens=_log(rng, 1, 64), experts=experts, k=min(experts, rng.choice((1, 2, 4, 6, 8))), hidden=hidden, inter=inter,
                bits=bits, block=block, x=rng.choice(("f16", "bf16")), zp=rng.random() < 0.4, bias=rng.random() < 0.5)


# ------------------------------------------------------------------------------------------------ the inputs
def _normal(g, shape, std, dtype=torch.float32):
    return torch.randn(shape, generator=g, device="cuda").mul_(std).to(dtype)


def _uniform(g, shape, lo, hi, dtype=torch.float32):
    return torch.rand(shape, generator=g, device="cuda").mul_(hi - lo).add_(lo).to(dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case=case)
    {"score": _logits, "loss": _logits, "adamw": _parameters, "moe": _layer}[case["op"]](s, case, g)
    return s


def _logits(s, case, g):
    """Logits of a model: most rows have a likely token, and it is the given one in half of them."""
    T, V, dt = case["rows"], case["vocab"], DT[case["x"]]
    x = _normal(g, (T, V), 2.0, dt)
    rows = torch.arange(T, device="cuda")
    target = torch.randint(0, V, (T,), generator=g, device="cuda")
    likely = torch.where(torch.rand(T, generator=g, device="cuda") < 0.5, target, torch.randint(0, V, (T,), generator=g, device="cuda"))
    x[rows, likely] += _uniform(g, (T,), 4.0, 16.0, dt)
    if case.get("mask"):
        out = torch.rand(V, generator=g, device="cuda") < case["mask"]
        out[likely] = False
        x[:, out] = -math.inf
    target[torch.rand(T, generator=g, device="cuda") < 0.06] = -100  # no token wanted there
    s["x"], s["target"], s["inv_temperature"] = x, target, 1.0 / 0.8
    if case["op"] == "loss":
        stats = [_score64(x[i:i + 256], target[i:i + 256], s["inv_temperature"]) for i in range(0, T, 256)]
        s["lse"], s["entropy"] = (torch.cat([t[n] for t in stats]).float() for n in (1, 2))
        s["d_logprob"] = _normal(g, (T,), 1.0 / T)
        s["d_entropy"] = _normal(g, (T,), 0.1 / T) if case["entropy"] else None
        s["dx"] = torch.empty_like(x)


def _tensor_sizes(case):
    """Of the adapters, the whole matrices and vectors of odd sizes, in values."""
    sizes = [m for _ in range(case["layers"]) for n, k in LAYER for m in (case["rank"] * k, n * case["rank"])]
    return sizes + [LAYER[i % 2][0] * LAYER[i % 2][1] for i in range(case["full"])] + [777 + 1003 * i for i in range(case["odd"])]


def _to_codes(x, keep):
    """8-bit values of x [n] and the scale of every BLOCK of them; keep: what is above zero stays above."""
    b = x.reshape(-1, BLOCK)
    top = b.abs().amax(dim=1, keepdim=True)
    big = top >= 1e-30
    c = b * torch.where(big, E4M3_MAX / top, 0.0)
    if keep:
        c = torch.where((c > 0) & (c < 2.0 ** -9), 2.0 ** -9, c)
    return c.to(torch.float8_e4m3fn).reshape(-1), torch.where(big, top / E4M3_MAX, 0.0).reshape(-1)


def _from_codes(c, scale, dtype):
    return (c.to(dtype).reshape(-1, BLOCK) * scale.to(dtype)[:, None]).reshape(-1)


def _parameters(s, case, g):
    """Flat buffers, as programs keep them; every tensor begins at a multiple of BLOCK and what lies between is zero."""
    sizes = _tensor_sizes(case)
    room = [-(-m // BLOCK) * BLOCK for m in sizes]
    n = sum(room)
    used = (torch.arange(n, device="cuda") - torch.repeat_interleave(torch.tensor([sum(room[:i]) for i in range(len(room))], device="cuda"),
            torch.tensor(room, device="cuda"), output_size=n)) < torch.repeat_interleave(torch.tensor(sizes, device="cuda"), torch.tensor(room, device="cuda"), output_size=n)
    w = _normal(g, (n,), 0.02) * used
    if case["master"]:
        s["master"] = w
    s["p"] = w.to(DT[case["p"]])
    s["g"] = (_normal(g, (n,), 1e-3) * used).to(DT[case["g"]])
    m, u = _normal(g, (n,), 3e-4) * used, _uniform(g, (n,), 3e-4, 1.5e-3) * used
    if case["state"] == "e4m3":
        (s["m"], s["m_scale"]), (s["u"], s["u_scale"]) = _to_codes(m, False), _to_codes(u, True)
    else:
        s["m"], s["v"] = m, u * u
    s["norm"] = torch.empty(1, device="cuda")
    if own:  # the list of a program's tensors, which it keeps from step to step
        import gemm_blockwise_dequant_gb300 as qg

        starts = [sum(room[:i]) for i in range(len(room))]
        part = lambda t: [t[a:a + m] for a, m in zip(starts, sizes)]
        blocks = lambda t: [t[a // BLOCK:(a + m + BLOCK - 1) // BLOCK] for a, m in zip(starts, sizes)]
        states = dict(exp_avg=part(s["m"]), exp_avg_sq=part(s["v"])) if case["state"] == "f32" else dict(
            exp_avg=part(s["m"]), exp_avg_scale=blocks(s["m_scale"]), exp_avg_rms=part(s["u"]), exp_avg_rms_scale=blocks(s["u_scale"]))
        s["list"] = qg.QGAdamWList(part(s["p"]), part(s["g"]), master=part(s["master"]) if case["master"] else None, weight_decay=DECAY, **states)


def _layer(s, case, g):
    T, E, H, I, bits, bs = (case[k] for k in ("tokens", "experts", "hidden", "inter", "bits", "block"))
    s["x"] = _normal(g, (T, H), 1.0, DT[case["x"]])
    s["router"] = _normal(g, (T, E), 1.5)
    top = 0.32 / (1 << bits)
    for name, n, k in (("fc1", 2 * I, H), ("fc2", H, I)):
        s[name + "_w"] = torch.randint(0, 256, (E, n, k * bits // 8), generator=g, device="cuda", dtype=torch.uint8)
        s[name + "_scales"] = _uniform(g, (E, n, k // bs), 0.25 * top, top, torch.float16)
        s[name + "_zp"] = torch.randint(0, 1 << bits, (E, n, k // bs), generator=g, device="cuda").to(torch.float16) if case["zp"] else None
        s[name + "_bias"] = _normal(g, (E, n), 0.01, torch.float16) if case["bias"] else None
    s["ids"] = torch.empty(T, case["k"], dtype=torch.int32, device="cuda")
    s["weights"] = torch.empty(T, case["k"], device="cuda")
    s["y"] = torch.empty_like(s["x"])


# ------------------------------------------------------------------------------------------------ one pass
def run(s):
    return (_OWN if own else _PLAIN)[s["case"]["op"]](s)


def _largest(x, k):
    """Indexes of the k largest of each row, the lower index first among equals."""
    bits = x.float().add(0.0).view(torch.int32).long()  # adding 0 makes one zero of two
    order = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits)
    key = (order << 32) + (0xFFFFFFFF - torch.arange(x.shape[1], device=x.device))
    return 0xFFFFFFFF - (key.topk(k, dim=1).values & 0xFFFFFFFF)


def _plain_score(s):
    z = s["x"].float() * s["inv_temperature"]
    top = z.amax(dim=1, keepdim=True)
    e = (z - top).exp()
    total = e.sum(dim=1)
    lse = top[:, 0] + total.log()
    part = torch.where(e > 0, e * (z - top), 0.0).sum(dim=1) / total
    given = s["target"] >= 0
    logprob = torch.where(given, z.gather(1, s["target"].clamp(min=0)[:, None])[:, 0] - lse, 0.0)
    out = {"logprob": logprob, "entropy": total.log() - part, "lse": lse}
    if s["case"]["top"]:
        out["top_ids"] = _largest(s["x"], s["case"]["top"])
        out["top_logprobs"] = z.gather(1, out["top_ids"]) - lse[:, None]
    return out


def _plain_loss(s):
    z = s["x"].float() * s["inv_temperature"]
    logp = z - s["lse"][:, None]
    given = s["target"] >= 0
    d = torch.where(given, s["d_logprob"], 0.0)
    factor = -d[:, None] if s["d_entropy"] is None else -(d[:, None] + s["d_entropy"][:, None] * (logp + s["entropy"][:, None]))
    dz = logp.exp() * factor
    dz.scatter_add_(1, s["target"].clamp(min=0)[:, None], d[:, None])
    return (dz * s["inv_temperature"]).to(s["x"].dtype)


def _plain_adamw(s):
    case = s["case"]
    g = s["g"].float()
    out = {}
    if case["clip"]:
        out["norm"] = g.square().sum().sqrt().reshape(1)
        g = g * (MAX_NORM / (out["norm"] + NORM_EPS)).clamp(max=1.0)
    eight = case["state"] == "e4m3"
    m = _from_codes(s["m"], s["m_scale"], torch.float32) if eight else s["m"]
    v = _from_codes(s["u"], s["u_scale"], torch.float32).square() if eight else s["v"]
    m = BETA1 * m + (1 - BETA1) * g
    v = BETA2 * v + (1 - BETA2) * g.square()
    u = v.sqrt()
    w = s["master"] if case["master"] else s["p"].float()
    w = w * (1 - LR * DECAY) - LR / (1 - BETA1 ** STEP) * m / (u / math.sqrt(1 - BETA2 ** STEP) + EPS)
    s["p"].copy_(w)
    if case["master"]:
        s["master"].copy_(w)
    if eight:
        for to, code in zip(("m", "m_scale", "u", "u_scale"), _to_codes(m, False) + _to_codes(u, True)):
            s[to].copy_(code)
    else:
        s["m"].copy_(m)
        s["v"].copy_(v)
    return out | _adamw_buffers(s)


def _adamw_buffers(s):
    return {k: s[k] for k in ("p", "master", "m", "v", "m_scale", "u", "u_scale") if k in s}


def _plain_weight(w, scales, zp, case, dtype=torch.float32):
    """[..., N, K] values of packed codes."""
    bits, bs = case["bits"], case["block"]
    shift = torch.arange(0, 8, bits, device="cuda", dtype=torch.uint8)
    q = ((w[..., None] >> shift) & ((1 << bits) - 1)).reshape(*scales.shape, bs).to(dtype)
    q = q - (zp.to(dtype)[..., None] if zp is not None else float(1 << (bits - 1)))
    return (q * scales.to(dtype)[..., None]).flatten(-2)


def _plain_moe(s):
    case = s["case"]
    T, E, k = case["tokens"], case["experts"], case["k"]
    ids = _largest(s["router"], k)
    chosen = s["router"].gather(1, ids)
    e = (chosen - chosen[:, :1]).exp()
    weights = e / e.sum(dim=1, keepdim=True)
    flat = ids.reshape(-1)
    x = s["x"].float()
    pick = (lambda t: None if t is None else t[flat]) if T * k < E else (lambda t: t)  # experts one by one for each pair, or all
    part = {n: pick(s[n]) for n in s if n.startswith("fc")}
    if T * k < E:
        rows = x.repeat_interleave(k, dim=0)[:, None]  # [pairs, 1, H]
    else:  # [E, T, H]: the rows of every expert in the order of the tokens
        place = (torch.nn.functional.one_hot(ids, E).sum(dim=1).cumsum(dim=0) - 1).gather(1, ids).reshape(-1)
        rows = torch.zeros(E, T, x.shape[1], device="cuda")
        rows[flat, place] = x.repeat_interleave(k, dim=0)
    product = lambda a, n: a @ _plain_weight(part[n + "_w"], part[n + "_scales"], part[n + "_zp"], case).transpose(1, 2) + (
        0.0 if part[n + "_bias"] is None else part[n + "_bias"].float()[:, None])
    gate, up = product(rows, "fc1").chunk(2, dim=2)
    o = product(gate / (1 + (-gate).exp()) * up, "fc2")
    o = o[:, 0] if T * k < E else o[flat, place]
    y = (o.reshape(T, k, -1) * weights[:, :, None]).sum(dim=1)
    return {"ids": ids.to(torch.int32), "weights": weights, "y": y.to(s["x"].dtype)}


def _own_score(s):
    import gemm_blockwise_dequant_gb300 as qg

    T, k = s["case"]["rows"], s["case"]["top"]
    stats = torch.empty(3, T, device="cuda")
    ids = torch.empty(T, k, dtype=torch.int64, device="cuda") if k else None
    top = torch.empty(T, k, device="cuda") if k else None
    qg.qg_token_logprobs(s["x"], s["target"], stats[0], entropy=stats[1], lse=stats[2], top_ids=ids, top_logprobs=top, inv_temperature=s["inv_temperature"])
    out = {"logprob": stats[0], "entropy": stats[1], "lse": stats[2]}
    return out | {"top_ids": ids, "top_logprobs": top} if k else out


def _own_loss(s):
    import gemm_blockwise_dequant_gb300 as qg

    qg.qg_token_logprobs_grad(s["x"], s["target"], s["lse"], s["d_logprob"], s["dx"], entropy=s["entropy"], d_entropy=s["d_entropy"],
                              inv_temperature=s["inv_temperature"])
    return s["dx"]


def _own_adamw(s):
    import gemm_blockwise_dequant_gb300 as qg

    clip = dict(max_norm=MAX_NORM, norm_eps=NORM_EPS, norm=s["norm"]) if s["case"]["clip"] else {}
    qg.qg_adamw_step(s["list"], lr=LR, step=STEP, betas=(BETA1, BETA2), eps=EPS, **clip)
    return ({"norm": s["norm"]} if clip else {}) | _adamw_buffers(s)


def _own_moe(s):
    import gemm_blockwise_dequant_gb300 as qg

    case = s["case"]
    qg.qmoe_route_topk(s["router"], s["ids"], s["weights"], renormalize=True)
    qg.qmoe_tokens_fused(s["x"], s["ids"], s["weights"], fc1_w=s["fc1_w"], fc1_scales=s["fc1_scales"], fc1_zp=s["fc1_zp"], fc1_bias=s["fc1_bias"],
                         fc2_w=s["fc2_w"], fc2_scales=s["fc2_scales"], fc2_zp=s["fc2_zp"], fc2_bias=s["fc2_bias"], bits=case["bits"],
                         block_size=case["block"], y=s["y"])
    return {"ids": s["ids"], "weights": s["weights"], "y": s["y"]}


_PLAIN = {"score": _plain_score, "loss": _plain_loss, "adamw": _plain_adamw, "moe": _plain_moe}
_OWN = {"score": _own_score, "loss": _own_loss, "adamw": _own_adamw, "moe": _own_moe}


# ------------------------------------------------------------------------------------------------ in 64 bits
def _score64(x, target, inv_temperature):
    z = x.double() * inv_temperature
    lse = torch.logsumexp(z, dim=1)
    logp = z - lse[:, None]
    p = logp.exp()
    entropy = -torch.where(p > 0, p * logp, 0.0).sum(dim=1)
    logprob = torch.where(target >= 0, logp.gather(1, target.clamp(min=0)[:, None])[:, 0], 0.0)
    return logprob, lse, entropy, logp


def exact(case, seed):
    s = prepare(case, seed)
    return {"score": _exact_score, "loss": _exact_loss, "adamw": _exact_adamw, "moe": _exact_moe}[case["op"]](s, case)


def _exact_score(s, case):
    got = []
    for i in range(0, case["rows"], 256):
        logprob, lse, entropy, logp = _score64(s["x"][i:i + 256], s["target"][i:i + 256], s["inv_temperature"])
        got.append((logprob, entropy, lse) + ((logp.sort(dim=1, descending=True).values[:, :case["top"]],) if case["top"] else ()))
    got = [torch.cat(t) for t in zip(*got)]
    out = {"logprob": got[0], "entropy": got[1], "lse": got[2]}
    return out | {"top_ids": None, "top_logprobs": got[3]} if case["top"] else out


def _exact_loss(s, case):
    t = s["inv_temperature"]
    out = torch.empty(s["x"].shape, dtype=torch.float64, device="cuda")
    for i in range(0, case["rows"], 256):
        rows = slice(i, i + 256)
        logp = s["x"][rows].double() * t - s["lse"][rows].double()[:, None]
        p = logp.exp()
        d = s["d_logprob"][rows].double() * (s["target"][rows] >= 0)
        onehot = torch.nn.functional.one_hot(s["target"][rows].clamp(min=0), case["vocab"])
        dz = d[:, None] * (onehot - p)
        if case["entropy"]:
            dz -= s["d_entropy"][rows].double()[:, None] * p * (logp + s["entropy"][rows].double()[:, None])
        out[rows] = t * dz
    return out


def _exact_adamw(s, case):
    g = s["g"].double()
    norm = g.norm()
    if case["clip"]:
        g = g * min(1.0, MAX_NORM / (float(norm) + NORM_EPS))
    if case["state"] == "e4m3":
        m, v = _from_codes(s["m"], s["m_scale"], torch.float64), _from_codes(s["u"], s["u_scale"], torch.float64) ** 2
    else:
        m, v = s["m"].double(), s["v"].double()
    m = m * BETA1 + g * (1 - BETA1)
    v = v * BETA2 + g * g * (1 - BETA2)
    w = (s["master"] if case["master"] else s["p"]).double()
    w = w - LR * DECAY * w - LR * (m / (1 - BETA1 ** STEP)) / ((v / (1 - BETA2 ** STEP)).sqrt() + EPS)
    out = {"p": w}
    if case["clip"]:
        out["norm"] = norm.reshape(1)
    if case["master"]:
        out["master"] = w
    if case["state"] == "e4m3":
        (out["m"], out["m_scale"]), (out["u"], out["u_scale"]) = _to_codes(m, False), _to_codes(v.sqrt(), True)
    else:
        out["m"], out["v"] = m, v
    return out


def _exact_moe(s, case):
    T, k = case["tokens"], case["k"]
    router = s["router"].double()
    top = router.sort(dim=1, descending=True, stable=True)
    ids, weights = top.indices[:, :k], top.values[:, :k].softmax(dim=1)
    y = torch.zeros(T, case["hidden"], dtype=torch.float64, device="cuda")
    for e in range(case["experts"]):
        t, j = (ids == e).nonzero(as_tuple=True)
        if t.numel():
            a = s["x"][t].double()
            for n in ("fc1", "fc2"):
                zp, bias = s[n + "_zp"], s[n + "_bias"]
                a = a @ _plain_weight(s[n + "_w"][e], s[n + "_scales"][e], None if zp is None else zp[e], case, torch.float64).t()
                a = a if bias is None else a + bias[e].double()
                a = torch.nn.functional.silu(a[:, :case["inter"]]) * a[:, case["inter"]:] if n == "fc1" else a
            y.index_add_(0, t, weights[t, j][:, None] * a)
    return {"ids": None, "weights": weights, "y": y}


# ------------------------------------------------------------------------------------------------ what a pass needs
def work(case):
    if case["op"] in ("score", "loss"):
        n, b = case["rows"] * case["vocab"], SIZE[case["x"]]
        if case["op"] == "score":
            return {"bytes": n * b + case["rows"] * (20 + 12 * case["top"]), "flops": 6 * n}
        return {"bytes": 2 * n * b + 24 * case["rows"], "flops": (6 if case["entropy"] else 4) * n}
    if case["op"] == "adamw":
        n = sum(_tensor_sizes(case))
        state = 4 * 4 if case["state"] == "f32" else 4 + 16 / BLOCK
        weights = SIZE[case["p"]] + 8 if case["master"] else 2 * SIZE[case["p"]]
        return {"bytes": int(n * (weights + SIZE[case["g"]] + state)), "flops": 14 * n}
    T, E, H, I, k = (case[n] for n in ("tokens", "experts", "hidden", "inter", "k"))
    used = E * (1 - (1 - k / E) ** T)  # experts that some token chose, as expected
    per = case["bits"] / 8 + (4 if case["zp"] else 2) / case["block"]
    weights = used * (3 * I * H * per + (2 * (2 * I + H) if case["bias"] else 0))
    return {"bytes": int(weights + 2 * SIZE[case["x"]] * T * H + 4 * T * (E + 2 * k)), "flops": 6 * T * k * H * I}
