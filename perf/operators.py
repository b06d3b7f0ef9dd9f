"""The fine-tuning and adapter-serving operators beside the quantized projections, as measured cases.

Four operators that a program needs around ``Y = A . dequant(W)^T`` when the quantized weight W [N, K] stays
frozen and low-rank adapters are served or trained beside it:

  apply   Y_out[t] = Y_in[t] + scaling[a] * (X[t] A[a]^T) B[a]^T for the rows t of every request, a the request's
          adapter (none for some): many requests with adapters of their own in one call
  grad    the backward pass of apply: G[t] = scaling[a] * dY[t] B[a], dX = dX_in + G A[a], dA[a] = G^T X and
          dB[a] = scaling[a] * dY^T V over the rows of adapter a, with V = X A[a]^T kept from the forward pass
  dgrad   dX = dY . dequant(W): the gradient of the activations through the frozen quantized weight
  clip    the norm over all the gradients of a step and their scaling to at most max_norm

``run`` computes them with elementary torch operations in fp32, rounded once at the end, or, where ``own`` is
true, with the calls that a user makes of this package.  ``exact`` computes them in fp64, request by request.
"""
import math
import random

import numpy as np
import torch

own = False

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
BLOCK = 64
MAX_NORM = 1.0
EPS = 1e-6

# The seven projections of a transformer layer with hidden 5120 and intermediate 17920, as (N, K): the adapters of
# a fine-tuning step are two tensors for each
LAYER = ((7680, 5120), (5120, 5120), (35840, 5120), (5120, 17920))


# ------------------------------------------------------------------------------------------------ the cases
def listed():
    return [
        # one token of one user in a decode step: nothing but latency; fp32 activations as in the 2-bit decode
        dict(name="apply 1 token", op="apply", rows=1, requests=1, adapters=4, rank=16, n=7680, k=5120, x="f32", w="f16"),
        # a decode step of 64 users with 32 adapters among them
        dict(name="apply 64 decode", op="apply", rows=64, requests=64, adapters=32, rank=16, n=14336, k=4096, x="bf16", w="bf16"),
        # the prompts of nine requests in one batch, on the widest contraction
        dict(name="apply 8192 prefill", op="apply", rows=8192, requests=9, adapters=6, rank=32, n=5120, k=17920, x="f16", w="f16"),
        # one short sample through a key/value projection, gradients kept in fp32
        dict(name="grad 333", op="grad", rows=333, requests=1, adapters=1, rank=8, n=1024, k=4096, x="bf16", w="bf16", g="f32"),
        # an ordinary fine-tuning batch of three packed samples, one adapter
        dict(name="grad 2048", op="grad", rows=2048, requests=3, adapters=1, rank=16, n=7680, k=5120, x="f16", w="f16", g="f16"),
        # a large batch that trains four adapters at once, high rank
        dict(name="grad 8192", op="grad", rows=8192, requests=11, adapters=4, rank=64, n=14336, k=4096, x="bf16", w="bf16", g="bf16"),
        # a short sample back through a codebook key/value projection
        dict(name="dgrad nf4 77", op="dgrad", rows=77, n=1024, k=4096, x="bf16", kind="nf4", zp="none"),
        # a batch back through the 2-bit down projection, all zero points 1.5
        dict(name="dgrad u2 2048", op="dgrad", rows=2048, n=5120, k=17920, x="f16", kind="u2", zp="uniform"),
        # the largest: a 4-bit gate/up projection with zero points
        dict(name="dgrad u4 4096", op="dgrad", rows=4096, n=35840, k=5120, x="bf16", kind="u4", zp="tensor"),
        # the adapters of one layer
        dict(name="clip layer", op="clip", layers=1, rank=16, full=0, x="f32"),
        # the adapters of a 40-layer model
        dict(name="clip adapters", op="clip", layers=40, rank=16, full=0, x="bf16"),
        # adapters and six whole weight matrices trained beside them
        dict(name="clip full", op="clip", layers=40, rank=64, full=6, x="bf16"),
    ]


def _log(rng, lo, hi, step=1):
    while True:
        v = step * int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
        if v != 3 << 10:
            return v


def draw(rng):
    op = rng.choice(("apply", "grad", "dgrad", "clip"))
    if op == "clip":
        x = rng.choice(("f32", "f16", "bf16"))
        return dict(op="clip", layers=_log(rng, 1, 40 if x != "f32" else 30), rank=rng.choice((4, 8, 12, 16, 32, 64)),
                    full=rng.choice((0, 0, 1) if x == "f32" else (0, 0, 0, 1, 3)), x=x)
    k = _log(rng, 8, 280, BLOCK)
    n = _log(rng, 4, 312, 64) if rng.random() < 0.75 else _log(rng, 256, 20000)  # most projections have round widths
    x = rng.choice(("f32", "f16", "bf16"))
    if op == "dgrad":
        rows = _log(rng, 1, 4096)
        while rows * n * k > 4096 * 35840 * 5120:
            rows = rows // 2 + 1
        return dict(op="dgrad", rows=rows, n=n, k=k, x=x, kind=rng.choice(("u2", "u4", "u8", "nf4")),
                    zp=rng.choice(("none", "uniform", "tensor")))
    rows = _log(rng, 1 if op == "apply" else 16, 8192)
    requests = min(rows, _log(rng, 1, 64))
    w = x if x != "f32" else rng.choice(("f32", "f16", "bf16"))
    case = dict(op=op, rows=rows, requests=requests, adapters=_log(rng, 1, 32 if op == "apply" else 8),
                rank=rng.choice((8, 16, 24, 32, 64)), n=n, k=k, x=x, w=w)
    if op == "grad":
        case["g"] = rng.choice((w, "f32"))
    while case["rows"] > 1 and case["rows"] * (n + k) * SIZE[x] > 8192 * (14336 + 4096) * 2:
        case["rows"] = case["rows"] // 2 + 1
        case["requests"] = min(case["requests"], case["rows"])
    return case


# ------------------------------------------------------------------------------------------------ the inputs
def _normal(g, shape, std, dtype):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _uniform(g, shape, lo, hi, dtype):
    return (torch.rand(shape, generator=g, device="cuda") * (hi - lo) + lo).to(dtype)


def _requests(case, seed):
    """Row offsets of the requests (ragged lengths that sum to the rows) and their adapters (every eighth has none)."""
    r = random.Random(seed)
    S, T = case["requests"], case["rows"]
    if S == T:
        lens = [1] * S  # a decode step
    else:
        w = [r.uniform(0.2, 1.0) for _ in range(S)]
        lens = [int(T * v / sum(w)) for v in w]
        lens[r.randrange(S)] += T - sum(lens)
    first = r.randrange(case["adapters"])
    ids = [-1 if i % 8 == 7 else (first + i) % case["adapters"] for i in range(S)]
    return [sum(lens[:i]) for i in range(S + 1)], ids


def _distinct(case):
    """How many adapters the requests use."""
    with_one = case["requests"] - case["requests"] // 8
    return min(case["adapters"], with_one)


def _tensors(case):
    """Sizes of the gradient tensors of a clip case."""
    sizes = []
    for _ in range(case["layers"]):
        for n, k in LAYER:
            sizes += [case["rank"] * k, n * case["rank"]]
    return sizes + [LAYER[i % 2][0] * LAYER[i % 2][1] for i in range(case["full"])]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case=case, op=case["op"])
    dt = DT[case["x"]]
    if case["op"] == "clip":
        sizes = _tensors(case)
        s["grads"] = [_normal(g, (m,), 1e-3, dt) for m in sizes]
        s["out"] = torch.empty(sum(sizes), dtype=dt, device="cuda")  # the optimizer's flat buffer
        s["outs"] = list(s["out"].split(sizes))
        s["norm"] = torch.empty(1, device="cuda")
        if own:  # the list of a program's gradient buffers, which it keeps from step to step
            import gemm_blockwise_dequant_gb300 as qg

            s["list"] = qg.QGGradList(s["grads"], s["outs"])
        return s
    N, K, T = case["n"], case["k"], case["rows"]
    if case["op"] == "dgrad":
        bits = int(case["kind"][1]) if case["kind"] != "nf4" else 4
        s["bits"] = bits
        s["dY"] = _normal(g, (T, N), 0.05, dt)
        s["dX"] = torch.empty(T, K, dtype=dt, device="cuda")
        s["W"] = torch.randint(0, 256, (N, K * bits // 8), generator=g, device="cuda", dtype=torch.uint8)
        if case["kind"] == "nf4":
            import statistics

            q = [statistics.NormalDist().inv_cdf(0.5 + 0.46875 * i / 8) for i in range(1, 9)]
            c = [-v / q[7] for v in q[1:]] + [0.0] + [v / q[7] for v in q]
            s["codebook"] = torch.tensor(sorted(c), dtype=torch.float32, device="cuda")
            s["absmax"] = _uniform(g, (N, K // BLOCK), 0.02, 0.1, torch.float32)
        else:
            top = 0.06 / (1 << (bits - 1))
            s["scales"] = _uniform(g, (N, K // BLOCK), 0.25 * top, top, torch.float16)
            if case["zp"] == "tensor":
                s["zp"] = torch.randint(0, 1 << bits, (N, K // BLOCK), generator=g, device="cuda").to(torch.float16)
            else:  # 1.5 for 2-bit codes, else the midpoint given or implied
                s["zp"] = 1.5 if bits == 2 and case["zp"] == "uniform" else float(1 << (bits - 1))
        return s
    offsets, ids = _requests(case, seed)
    na, r, wd = case["adapters"], case["rank"], DT[case["w"]]
    s["host"] = (offsets, ids)
    s["offsets"] = torch.tensor(offsets, dtype=torch.int64, device="cuda")
    s["ids"] = torch.tensor(ids, dtype=torch.int32, device="cuda")
    s["A"] = _uniform(g, (na, r, K), -K ** -0.5, K ** -0.5, wd)
    s["B"] = _normal(g, (na, N, r), 0.02, wd)
    s["scaling"] = _uniform(g, (na,), 0.5, 2.0, torch.float32)
    s["X"] = _normal(g, (T, K), 1.0, dt)
    if case["op"] == "apply":
        s["Yin"] = _normal(g, (T, N), 1.0, dt)
        s["Y"] = torch.empty(T, N, dtype=dt, device="cuda")
        return s
    s["dY"] = _normal(g, (T, N), 0.05, dt)
    s["V"] = torch.zeros(T, r, device="cuda")  # X A^T in fp32, kept from the forward pass
    for i, a in enumerate(ids):
        if a >= 0:
            s["V"][offsets[i]:offsets[i + 1]] = s["X"][offsets[i]:offsets[i + 1]].float() @ s["A"][a].float().t()
    s["dXin"] = _normal(g, (T, K), 0.05, dt)  # what dgrad left there
    s["dX"] = torch.empty(T, K, dtype=dt, device="cuda")
    gd = DT[case["g"]]
    s["dA"] = torch.empty(na, r, K, dtype=gd, device="cuda")
    s["dB"] = torch.empty(na, N, r, dtype=gd, device="cuda")
    return s


# ------------------------------------------------------------------------------------------------ one pass
def run(s):
    return (_run_own if own else _run_plain)[s["op"]](s)


def _rows_of(s, na, r, T):
    """[T, na * r] truth values: the columns of the row's own adapter; and the row's scaling [T, 1]."""
    lens = s["offsets"][1:] - s["offsets"][:-1]
    a = torch.repeat_interleave(s["ids"].long(), lens, output_size=T)
    mine = (a[:, None] == torch.arange(na, device=a.device)[None, :]).repeat_interleave(r, dim=1)
    return mine, s["scaling"][a.clamp(min=0)][:, None]


def _plain_apply(s):
    na, r, K = s["A"].shape
    N = s["B"].shape[1]
    mine, scale = _rows_of(s, na, r, s["X"].shape[0])
    v = s["X"].float() @ s["A"].float().reshape(na * r, K).t()
    v = torch.where(mine, v, 0.0) * scale
    y = s["Yin"].float() + v @ s["B"].float().transpose(1, 2).reshape(na * r, N)
    return y.to(s["Y"].dtype)


def _plain_grad(s):
    na, r, K = s["A"].shape
    N = s["B"].shape[1]
    T = s["X"].shape[0]
    mine, scale = _rows_of(s, na, r, T)
    dy = s["dY"].float()
    gv = torch.where(mine, dy @ s["B"].float().transpose(1, 2).reshape(na * r, N).t(), 0.0) * scale
    dx = s["dXin"].float() + gv @ s["A"].float().reshape(na * r, K)
    da = gv.t() @ s["X"].float()
    v = torch.where(mine, s["V"].repeat(1, na), 0.0) * scale
    db = (v.t() @ dy).reshape(na, r, N).transpose(1, 2).contiguous()
    return {"dX": dx.to(s["dX"].dtype), "dA": da.reshape(na, r, K).to(s["dA"].dtype), "dB": db.to(s["dB"].dtype)}


def _plain_weight(s):
    N = s["W"].shape[0]
    bits, K = s["bits"], s["case"]["k"]
    shift = torch.arange(0, 8, bits, device="cuda", dtype=torch.int32)
    q = ((s["W"].int()[:, :, None] >> shift) & ((1 << bits) - 1)).reshape(N, K // BLOCK, BLOCK)
    if "codebook" in s:
        return (s["codebook"][q] * s["absmax"][:, :, None]).reshape(N, K)
    zp = s["zp"].float()[:, :, None] if isinstance(s["zp"], torch.Tensor) else s["zp"]
    return ((q.float() - zp) * s["scales"].float()[:, :, None]).reshape(N, K)


def _plain_dgrad(s):
    return (s["dY"].float() @ _plain_weight(s)).to(s["dX"].dtype)


def _plain_clip(s):
    norm = torch.stack([t.float().square().sum() for t in s["grads"]]).sum().sqrt().reshape(1)
    coef = (MAX_NORM / (norm + EPS)).clamp(max=1.0)
    return {"norm": norm, "out": torch.cat([(t.float() * coef).to(t.dtype) for t in s["grads"]])}


def _own_apply(s):
    import gemm_blockwise_dequant_gb300 as qg

    qg.qg_lora_apply(s["X"], s["offsets"], s["ids"], s["A"], s["B"], s["scaling"], s["Yin"], s["Y"])
    return s["Y"]


def _own_grad(s):
    import gemm_blockwise_dequant_gb300 as qg

    qg.qg_lora_grad(s["dY"], s["X"], s["V"], s["offsets"], s["ids"], s["A"], s["B"], s["scaling"], s["dXin"], s["dX"],
                    s["dA"], s["dB"])
    return {"dX": s["dX"], "dA": s["dA"], "dB": s["dB"]}


def _own_dgrad(s):
    import gemm_blockwise_dequant_gb300 as qg

    if "codebook" in s:
        qg.qgemm_codebook4_dgrad(s["dY"], s["W"], s["codebook"], s["absmax"], s["dX"], block_size=BLOCK)
    elif isinstance(s["zp"], torch.Tensor):
        qg.qgemm_nbits_dgrad(s["dY"], s["W"], s["scales"], s["zp"], s["dX"], bits=s["bits"], block_size=BLOCK)
    elif s["case"]["zp"] == "uniform":
        qg.qgemm_nbits_uniform_zp_dgrad(s["dY"], s["W"], s["scales"], s["zp"], s["dX"], bits=s["bits"], block_size=BLOCK)
    else:
        qg.qgemm_nbits_dgrad(s["dY"], s["W"], s["scales"], None, s["dX"], bits=s["bits"], block_size=BLOCK)
    return s["dX"]


def _own_clip(s):
    import gemm_blockwise_dequant_gb300 as qg

    qg.qg_clip_grad_norm(s["list"], MAX_NORM, s["norm"], eps=EPS)
    return {"norm": s["norm"], "out": s["out"]}


_run_plain = {"apply": _plain_apply, "grad": _plain_grad, "dgrad": _plain_dgrad, "clip": _plain_clip}
_run_own = {"apply": _own_apply, "grad": _own_grad, "dgrad": _own_dgrad, "clip": _own_clip}


# ------------------------------------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "clip":
        total = sum(float((t.double() ** 2).sum()) for t in s["grads"])
        norm = math.sqrt(total)
        c = min(1.0, MAX_NORM / (norm + EPS))
        return {"norm": np.array([norm]), "out": torch.cat([t.double() * c for t in s["grads"]])}
    if case["op"] == "dgrad":
        N, K, bits = case["n"], case["k"], s["bits"]
        per = 8 // bits
        w = torch.empty(N, K // per, per, dtype=torch.float64, device="cuda")
        for j in range(per):
            code = (s["W"].int() // (1 << (j * bits))) % (1 << bits)
            w[:, :, j] = s["codebook"].double()[code.long()] if "codebook" in s else code.double()
        w = w.reshape(N, K)
        for b in range(K // BLOCK):
            cols = slice(b * BLOCK, (b + 1) * BLOCK)
            if "codebook" in s:
                w[:, cols] *= s["absmax"][:, b:b + 1].double()
            else:
                zp = s["zp"][:, b:b + 1].double() if isinstance(s["zp"], torch.Tensor) else s["zp"]
                w[:, cols] = (w[:, cols] - zp) * s["scales"][:, b:b + 1].double()
        return s["dY"].double() @ w
    offsets, ids = s["host"]
    if case["op"] == "apply":
        y = s["Yin"].double()
        for i, a in enumerate(ids):
            if a >= 0:
                t = slice(offsets[i], offsets[i + 1])
                v = s["X"][t].double() @ s["A"][a].double().t()
                y[t] += float(s["scaling"][a]) * (v @ s["B"][a].double().t())
        return y
    dx = s["dXin"].double()
    da = torch.zeros(s["dA"].shape, dtype=torch.float64, device="cuda")
    db = torch.zeros(s["dB"].shape, dtype=torch.float64, device="cuda")
    for i, a in enumerate(ids):
        if a >= 0:
            t = slice(offsets[i], offsets[i + 1])
            c, dy = float(s["scaling"][a]), s["dY"][t].double()
            gv = c * (dy @ s["B"][a].double())
            dx[t] += gv @ s["A"][a].double()
            da[a] += gv.t() @ s["X"][t].double()
            db[a] += c * (dy.t() @ s["V"][t].double())
    return {"dX": dx, "dA": da, "dB": db}


# ------------------------------------------------------------------------------------------------ what a pass needs
def work(case):
    b = SIZE[case["x"]]
    if case["op"] == "clip":
        m = sum(_tensors(case))
        return {"bytes": 2 * b * m + 4, "flops": 3 * m}
    T, N, K = case["rows"], case["n"], case["k"]
    if case["op"] == "dgrad":
        bits = int(case["kind"][1]) if case["kind"] != "nf4" else 4
        par = 4 if case["kind"] == "nf4" or case["zp"] == "tensor" else 2
        return {"bytes": b * T * (N + K) + N * K * bits // 8 + par * N * (K // BLOCK), "flops": 2 * T * N * K}
    r, used = case["rank"], _distinct(case)
    adapters = used * r * (N + K) * SIZE[case["w"]]
    if case["op"] == "apply":
        return {"bytes": b * T * (K + 2 * N) + adapters, "flops": 2 * T * r * (N + K)}
    grads = case["adapters"] * r * (N + K) * SIZE[case["g"]]
    return {"bytes": b * T * (N + 3 * K) + 4 * T * r + adapters + grads, "flops": 4 * T * r * (N + K)}
