"""What the calls around tokens (log probabilities and their gradient, AdamW, routing, experts) refuse on the host: every call
here returns before anything is enqueued, so no GPU is needed and no pointer is followed."""
import ctypes
import math

import pytest

from test_train_abi_cpu import P, qg  # noqa: F401  (qg: the fixture)


def scores(qg, **o):
    a = dict(X=P, xt=qg.QG_BF16, ldx=100, t=P, T=4, V=100, it=1.0, lp=P, en=P, lse=P, k=5, ids=P, top=P, st=P)
    a.update(o)
    return qg.lib().qg_token_logprobs(*[a[n] for n in ("X", "xt", "ldx", "t", "T", "V", "it", "lp", "en", "lse", "k", "ids", "top", "st")], None)


@pytest.mark.parametrize("o", [dict(xt=3), dict(xt=-1), dict(T=-1), dict(V=0), dict(V=-5), dict(ldx=99), dict(X=None), dict(X=P + 1), dict(t=P + 4),
                               dict(it=0.0), dict(it=-1.0), dict(it=math.inf), dict(it=math.nan), dict(k=-1), dict(k=101), dict(ids=None),
                               dict(top=None), dict(ids=P + 4), dict(top=P + 2), dict(lp=P + 2), dict(en=P + 1), dict(lse=P + 3), dict(st=P + 2)])
def test_scores_invalid(qg, o):
    assert scores(qg, **o) == qg.QG_ERR_INVALID_ARG


def test_scores_unsupported_and_empty(qg):
    for o in (dict(k=65), dict(T=(1 << 20) + 1), dict(V=(1 << 28) + 1, ldx=1 << 30)):
        assert scores(qg, **o) == qg.QG_ERR_UNSUPPORTED
    assert scores(qg, T=0, X=None, t=None, ids=None, top=None) == qg.QG_OK
    assert scores(qg, T=0, it=math.nan) == qg.QG_ERR_INVALID_ARG


def gradient(qg, **o):
    a = dict(X=P, xt=qg.QG_F16, ldx=100, t=P, lse=P, en=P, dl=P, de=P, it=1.0, dX=2 * P, lddx=100, T=4, V=100)
    a.update(o)
    return qg.lib().qg_token_logprobs_grad(*[a[n] for n in ("X", "xt", "ldx", "t", "lse", "en", "dl", "de", "it", "dX", "lddx", "T", "V")], None)


@pytest.mark.parametrize("o", [dict(xt=5), dict(T=-1), dict(V=0), dict(ldx=99), dict(lddx=99), dict(X=None), dict(dX=None), dict(dX=2 * P + 1), dict(lse=None),
                               dict(dl=None), dict(en=None), dict(dX=P, lddx=104), dict(de=P + 2), dict(t=P + 1), dict(it=math.inf)])
def test_gradient_invalid(qg, o):
    assert gradient(qg, **o) == qg.QG_ERR_INVALID_ARG


def test_gradient_unsupported_and_empty(qg):
    assert gradient(qg, V=(1 << 28) + 1, ldx=1 << 30, lddx=1 << 30) == qg.QG_ERR_UNSUPPORTED
    assert gradient(qg, T=0, X=None, t=None, lse=None, en=None, dl=None, de=None, dX=None) == qg.QG_OK


def route(qg, **o):
    a = dict(L=P, t=qg.QG_F32, ld=8, T=4, E=8, k=2, re=1, ids=P, w=P)
    a.update(o)
    return qg.lib().qmoe_route_topk(*[a[n] for n in ("L", "t", "ld", "T", "E", "k", "re", "ids", "w")], None)


def test_route(qg):
    for o in (dict(t=3), dict(T=-1), dict(E=0), dict(k=0), dict(k=9), dict(ld=7), dict(re=2), dict(L=None), dict(ids=None), dict(w=None), dict(L=P + 2),
              dict(ids=P + 2), dict(w=P + 1)):
        assert route(qg, **o) == qg.QG_ERR_INVALID_ARG, o
    for o in (dict(E=513, ld=513), dict(k=17, E=32, ld=32), dict(T=(1 << 20) + 1)):
        assert route(qg, **o) == qg.QG_ERR_UNSUPPORTED, o
    assert route(qg, T=0, L=None, ids=None, w=None) == qg.QG_OK


def experts(qg, **o):
    a = dict(x=P, xt=qg.QG_F16, ids=P, w=P, T=4, k=2, E=8, w1=P, s1=P, z1=P, b1=P, w2=P, s2=P, z2=P, b2=P, H=256, I=128, bits=4, bs=64, sw=0, y=P,
             yt=qg.QG_F16, st=P, ws=P, wsb=1 << 30)
    a.update(o)
    return qg.lib().qmoe_tokens_fused(*[a[n] for n in ("x", "xt", "ids", "w", "T", "k", "E", "w1", "s1", "z1", "b1", "w2", "s2", "z2", "b2", "H", "I", "bits",
                                                       "bs", "sw", "y", "yt", "st", "ws", "wsb")], None)


def test_experts(qg):
    for o in (dict(xt=4), dict(yt=-1), dict(T=-1), dict(k=0), dict(E=0), dict(H=0), dict(I=-64), dict(sw=2), dict(H=288), dict(I=96), dict(x=None), dict(ids=None),
              dict(w=None), dict(w1=None), dict(s1=None), dict(w2=None), dict(s2=None), dict(y=None), dict(x=P + 8), dict(w1=P + 8), dict(s2=P + 2), dict(z1=P + 2),
              dict(y=P + 2), dict(ids=P + 2), dict(w=P + 2), dict(b1=P + 1), dict(st=P + 2), dict(ws=P + 8)):
        assert experts(qg, **o) == qg.QG_ERR_INVALID_ARG, o
    for o in (dict(xt=qg.QG_F32), dict(bits=3), dict(bits=0), dict(bs=16), dict(bs=48), dict(k=17), dict(E=513), dict(T=513), dict(T=1025, k=1), dict(T=1 << 30, k=16)):
        assert experts(qg, **o) == qg.QG_ERR_UNSUPPORTED, o
    assert experts(qg, T=0, x=None, ids=None, w1=None, ws=None, wsb=0) == qg.QG_OK
    need = qg.qmoe_tokens_workspace_bytes(4, 2, 256, 128)
    assert need >= 8 * (256 + 128) * 4 and qg.qmoe_tokens_workspace_bytes(0, 2, 256, 128) == 0
    assert experts(qg, wsb=need - 1) == qg.QG_ERR_WORKSPACE_TOO_SMALL and experts(qg, ws=None) == qg.QG_ERR_WORKSPACE_TOO_SMALL


def entry(qg, **o):
    a = dict(param=P, grad=P, master=None, exp_avg=P, exp_avg_sq=P, exp_avg_scale=P, exp_avg_sq_scale=P, numel=1000, weight_decay=0.01,
             param_dtype=qg.QG_BF16, grad_dtype=qg.QG_F32, state=qg.QG_STATE_E4M3)
    a.update(o)
    return qg._AdamWTensor(**a)


def lay_out(qg, *entries):
    host, chunks = (qg._AdamWTensor * len(entries))(*entries), ctypes.c_int64(-1)
    return qg.lib().qg_adamw_list_init(host, len(entries), ctypes.byref(chunks)), chunks.value, [t.first_chunk for t in host]


@pytest.mark.parametrize("o", [dict(numel=-1), dict(param_dtype=3), dict(grad_dtype=-1), dict(state=2), dict(weight_decay=-0.1), dict(weight_decay=math.nan),
                               dict(weight_decay=math.inf), dict(param=None), dict(grad=None), dict(exp_avg=None), dict(exp_avg_sq=None),
                               dict(exp_avg_scale=None), dict(exp_avg_sq_scale=None), dict(exp_avg_scale=P + 2), dict(param=P + 1), dict(grad=P + 2),
                               dict(master=P + 2), dict(state=0, exp_avg=P + 1), dict(state=0, exp_avg_sq=P + 2)])
def test_list_invalid(qg, o):
    assert lay_out(qg, entry(qg), entry(qg, **o))[0] == qg.QG_ERR_INVALID_ARG


def test_list(qg):
    status, chunks, first = lay_out(qg, entry(qg, numel=0, param=None, grad=None, exp_avg=None, exp_avg_sq=None, exp_avg_scale=None, exp_avg_sq_scale=None),
                                    entry(qg, numel=1), entry(qg, numel=100001, state=qg.QG_STATE_F32, exp_avg_scale=None, exp_avg_sq_scale=None), entry(qg, exp_avg=P + 3))
    assert status == qg.QG_OK and first[:3] == [0, 0, 1] and 1 < first[3] < chunks == first[3] + 1
    assert lay_out(qg)[:2] == (qg.QG_OK, 0)
    assert lay_out(qg, entry(qg, numel=1 << 62))[0] == qg.QG_ERR_UNSUPPORTED
    chunks = ctypes.c_int64(0)
    assert qg.lib().qg_adamw_list_init(None, 1, ctypes.byref(chunks)) == qg.QG_ERR_INVALID_ARG
    assert qg.lib().qg_adamw_list_init(None, 0, None) == qg.QG_ERR_INVALID_ARG
    assert qg.lib().qg_adamw_list_init(None, -1, ctypes.byref(chunks)) == qg.QG_ERR_INVALID_ARG


def step(qg, **o):
    a = dict(t=P, n=2, c=7, lr=1e-3, lrd=None, b1=0.9, b2=0.999, eps=1e-8, step=1, sd=None, mx=1.0, ne=1e-6, nd=P, ws=P, wsb=1 << 20)
    a.update(o)
    return qg.lib().qg_adamw_step(*[a[n] for n in ("t", "n", "c", "lr", "lrd", "b1", "b2", "eps", "step", "sd", "mx", "ne", "nd", "ws", "wsb")], None)


def test_step(qg):
    for o in (dict(n=-1), dict(c=-1), dict(c=1 << 31), dict(n=0), dict(t=None), dict(t=P + 4), dict(lr=-1.0), dict(lr=math.nan), dict(lr=math.inf), dict(lrd=P + 2),
              dict(b1=1.0), dict(b1=-0.1), dict(b2=1.0), dict(b2=math.nan), dict(eps=-1.0), dict(eps=math.inf), dict(step=0), dict(sd=P + 4), dict(mx=math.nan),
              dict(ne=-1.0), dict(ne=math.nan), dict(nd=P + 2), dict(ws=P + 8)):
        assert step(qg, **o) == qg.QG_ERR_INVALID_ARG, o
    need = qg.qg_adamw_step_workspace_bytes(7)
    assert need > 0 and step(qg, wsb=need - 1) == qg.QG_ERR_WORKSPACE_TOO_SMALL and step(qg, ws=None) == qg.QG_ERR_WORKSPACE_TOO_SMALL
    assert step(qg, n=0, c=0, t=None, mx=-1.0, ws=None, wsb=0) == qg.QG_OK


def test_operands_of_the_python_calls(qg):
    """Types, shapes and order of every operand, and that each is on a GPU."""
    import torch

    T, V, k = 4, 50, 3
    f, i64, i32 = dict(dtype=torch.float32), dict(dtype=torch.int64), dict(dtype=torch.int32)
    good = dict(X=torch.zeros(T, V, dtype=torch.bfloat16), targets=torch.zeros(T, **i64), logprob=torch.zeros(T), entropy=torch.zeros(T), lse=torch.zeros(T),
                top_ids=torch.zeros(T, k, **i64), top_logprobs=torch.zeros(T, k), status=torch.zeros(1, **i32))
    for o in (dict(), dict(X=good["X"][0]), dict(X=torch.zeros(T, 2 * V, dtype=torch.bfloat16)[:, ::2]), dict(targets=good["targets"].int()), dict(targets=good["targets"][:2]),
              dict(logprob=good["logprob"].half()), dict(entropy=torch.zeros(2 * T)[::2]), dict(lse=torch.zeros(T + 1)), dict(top_ids=None),
              dict(top_ids=good["top_ids"].int()), dict(top_logprobs=torch.zeros(T, k + 1)), dict(status=torch.zeros(1))):
        a = dict(good, **o)
        with pytest.raises(ValueError):
            qg.qg_token_logprobs(a.pop("X"), a.pop("targets"), a.pop("logprob"), **a)
    grad = dict(X=good["X"], targets=good["targets"], lse=torch.zeros(T), d_logprob=torch.zeros(T), dX=torch.zeros(T, V, dtype=torch.bfloat16))
    for o in (dict(), dict(dX=torch.zeros(T, V)), dict(dX=grad["dX"][:2]), dict(d_logprob=torch.zeros(T, **i64)), dict(lse=torch.zeros(T, 1))):
        with pytest.raises(ValueError):
            qg.qg_token_logprobs_grad(*dict(grad, **o).values())
    for o in ((), (torch.zeros(T), None, None), (None, torch.zeros(T, k, **i64), None), (None, None, torch.zeros(T, 2)), (None, torch.zeros(2, k, **i32), torch.zeros(2, k))):
        a = [n if n is not None else d for n, d in zip(o + (None,) * (3 - len(o)), (torch.zeros(T, 8), torch.zeros(T, k, **i32), torch.zeros(T, k)))]
        with pytest.raises(ValueError):
            qg.qmoe_route_topk(*a)
    E, H, I = 8, 256, 128
    half, u8 = dict(dtype=torch.float16), dict(dtype=torch.uint8)
    moe = dict(x=torch.zeros(T, H, **half), expert_ids=torch.zeros(T, k, **i32), expert_weights=torch.zeros(T, k), fc1_w=torch.zeros(E, 2 * I, H // 2, **u8),
               fc1_scales=torch.zeros(E, 2 * I, H // 64, **half), fc1_zp=None, fc1_bias=torch.zeros(E, 2 * I, **half), fc2_w=torch.zeros(E, H, I // 2, **u8),
               fc2_scales=torch.zeros(E, H, I // 64, **half), fc2_zp=None, fc2_bias=torch.zeros(E, H, **half), bits=4, block_size=64, y=torch.zeros(T, H, **half))
    for o in (dict(), dict(x=moe["x"][0]), dict(y=torch.zeros(T, H + 1)), dict(x=torch.zeros(H, T, **half).t()), dict(expert_ids=torch.zeros(T, k, **i64)),
              dict(expert_weights=torch.zeros(T, k + 1)), dict(fc1_w=moe["fc1_w"].int()), dict(fc1_w=moe["fc1_w"][:, 1:]), dict(fc1_scales=moe["fc1_scales"].float()),
              dict(fc2_scales=moe["fc2_scales"][..., :1]), dict(fc1_zp=moe["fc1_scales"][:-1]), dict(fc2_bias=torch.zeros(H, **half)), dict(bits=3), dict(bits=0),
              dict(block_size=0), dict(fc2_w=moe["fc2_w"][:4], fc2_scales=moe["fc2_scales"][:4], fc2_bias=moe["fc2_bias"][:4]), dict(status=torch.zeros(1))):
        with pytest.raises(ValueError):
            qg.qmoe_tokens_fused(**dict(moe, **o))
    p = torch.zeros(1000)
    for a, o in (([p], dict()), ([p, p], dict()), ([p], dict(state="f16")), ([p], dict(exp_avg_sq=[p])), ([p], dict(weight_decay=[0.1, 0.2])), ([p], dict(master=[p, p]))):
        with pytest.raises(ValueError):
            qg.QGAdamWList(a, [p], **o)
    with pytest.raises(ValueError):
        qg.qg_adamw_step([p], lr=1e-3, step=1)
