"""Plain fp64 forms of the adapter operators, request by request, and inputs for their tests (test infrastructure)."""
from __future__ import annotations

import torch

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
# unit roundoffs: one rounding to the type is at most this much of the value
UNIT = {t: torch.finfo(t).eps / 2 for t in DT.values()}
# What the sums before that rounding may be off, as a share of the sum of the magnitudes of their terms: operands kept
# to 2^-17 (two bf16 terms) or better, twice, and at most 2^-24 for each of a few hundred additions
SUMS = 2.0 ** -15


def lora_case(lens, ids, *, na, r, N, K, x="bf16", w=None, seed=0, extra=0, pad=0, scaling=True):
    """Device tensors of one request list; `extra` rows belong to no request; `pad` values lie between rows."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    w = w or x
    T = sum(lens) + extra
    rnd = lambda *s, std=1.0: torch.randn(*s, generator=g, device="cuda") * std
    wide = lambda t, p: torch.nn.functional.pad(t, (0, p))[:, :t.shape[1]] if p else t
    c = dict(T=T, N=N, K=K, r=r, na=na, lens=lens, ids_host=ids, x=DT[x], w=DT[w])
    c["X"] = wide(rnd(T, K).to(DT[x]), pad)
    c["A"] = rnd(na, r, K, std=K ** -0.5).to(DT[w])
    c["B"] = rnd(na, N, r, std=0.1).to(DT[w])
    c["scaling"] = torch.rand(na, generator=g, device="cuda") + 0.5 if scaling else None
    off = [0]
    for n in lens:
        off.append(off[-1] + n)
    c["off_host"] = off
    c["offsets"] = torch.tensor(off, dtype=torch.int64, device="cuda")
    c["ids"] = torch.tensor(ids, dtype=torch.int32, device="cuda")
    c["dY"] = wide(rnd(T, N).to(DT[x]), pad)
    c["Yin"] = rnd(T, N)
    c["dXin"] = wide(rnd(T, K).to(DT[x]), pad)
    return c


def spans(c):
    for i, a in enumerate(c["ids_host"]):
        yield slice(c["off_host"][i], c["off_host"][i + 1]), (a if 0 <= a < c["na"] else -1)


def scale_of(c, a):
    return 1.0 if c["scaling"] is None else float(c["scaling"][a])


def apply64(c, Yin):
    """(Y, V, magnitude of Y's terms) in fp64; rows of no request are NaN in Y."""
    y = torch.full((c["T"], c["N"]), float("nan"), dtype=torch.float64, device="cuda")
    v = torch.zeros(c["T"], c["r"], dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(y)
    for t, a in spans(c):
        y[t] = 0 if Yin is None else Yin[t].double()
        if a >= 0:
            x, A, B, s = c["X"][t].double(), c["A"][a].double(), c["B"][a].double(), scale_of(c, a)
            v[t] = x @ A.t()
            y[t] += s * (v[t] @ B.t())
            mag[t] = s * ((x.abs() @ A.abs().t()) @ B.abs().t())
    return y, v, mag


def grad64(c, V, dXin):
    """dX, dA, dB and the magnitudes of their terms in fp64."""
    dx = torch.full((c["T"], c["K"]), float("nan"), dtype=torch.float64, device="cuda")
    mx = torch.zeros_like(dx)
    da = torch.zeros(c["na"], c["r"], c["K"], dtype=torch.float64, device="cuda")
    db = torch.zeros(c["na"], c["N"], c["r"], dtype=torch.float64, device="cuda")
    ma, mb = torch.zeros_like(da), torch.zeros_like(db)
    for t, a in spans(c):
        dx[t] = 0 if dXin is None else dXin[t].double()
        if a >= 0:
            s, dy, x, v = scale_of(c, a), c["dY"][t].double(), c["X"][t].double(), V[t].double()
            A, B = c["A"][a].double(), c["B"][a].double()
            g, mg = s * (dy @ B), s * (dy.abs() @ B.abs())
            dx[t] += g @ A
            mx[t] = mg @ A.abs()
            da[a] += g.t() @ x
            ma[a] += mg.t() @ x.abs()
            db[a] += s * (dy.t() @ v)
            mb[a] += s * (dy.abs().t() @ v.abs())
    return (dx, da, db), (mx, ma, mb)


def check(got, want, mag, sums=SUMS):
    """Every value within one rounding of its type plus `sums` of its terms' magnitude; whole norm a good deal closer."""
    u = UNIT[got.dtype]
    g, e = got.double(), (got.double() - want).abs()
    assert bool(torch.isfinite(g).all())
    tiny = 2.0 ** -25 if got.dtype == torch.float16 else 0.0  # half the spacing of fp16's subnormals
    room = u * want.abs() + sums * mag + tiny
    bad = e > room
    assert not bool(bad.any()), "%d of %d values off, worst %.3g of the room" % (
        int(bad.sum()), bad.numel(), float((e / room.clamp(min=1e-300)).max()))
    norm = float(want.norm())
    if norm:
        assert float(e.norm()) <= (u + 1e-5) * norm + (1e-5 * float(mag.norm()) if mag.numel() < 64 else 0.0) + tiny * mag.numel() ** 0.5
