"""What the adapter, activation-gradient and clipping entry points refuse, on the host: every call here returns before
anything is enqueued, so no GPU is needed and the pointers are never followed."""
import ctypes

import pytest

P = 1 << 20  # an aligned address that is never read


@pytest.fixture(scope="module")
def qg():
    from gemm_blockwise_dequant_gb300 import build

    build.build()
    import gemm_blockwise_dequant_gb300 as qg

    qg.lib()
    return qg


def apply(qg, **o):
    a = dict(X=P, xt=qg.QG_BF16, ldx=64, off=P, ids=P, S=2, A=P, B=P, wt=qg.QG_BF16, sc=P, na=2, r=8, Yin=P, yit=qg.QG_BF16, ldyi=32,
             Y=P, yt=qg.QG_BF16, ldy=32, V=P, T=4, N=32, K=64, st=P, ws=P, wsb=1 << 30)
    a.update(o)
    return qg.lib().qg_lora_apply(*[a[k] for k in ("X", "xt", "ldx", "off", "ids", "S", "A", "B", "wt", "sc", "na", "r", "Yin", "yit", "ldyi", "Y",
                                                   "yt", "ldy", "V", "T", "N", "K", "st", "ws", "wsb")], None)


def grad(qg, **o):
    a = dict(dY=P, xt=qg.QG_F16, lddy=32, X=P, ldx=64, V=P, off=P, ids=P, S=2, A=P, B=P, wt=qg.QG_F16, sc=P, na=2, r=8, dXi=P, dX=P, lddx=64,
             dA=P, dB=P, gt=qg.QG_F16, acc=0, T=4, N=32, K=64, st=P, ws=P, wsb=1 << 30)
    a.update(o)
    return qg.lib().qg_lora_grad(*[a[k] for k in ("dY", "xt", "lddy", "X", "ldx", "V", "off", "ids", "S", "A", "B", "wt", "sc", "na", "r", "dXi",
                                                  "dX", "lddx", "dA", "dB", "gt", "acc", "T", "N", "K", "st", "ws", "wsb")], None)


@pytest.mark.parametrize("o", [dict(xt=7), dict(wt=-1), dict(yt=3), dict(yit=9), dict(T=-1), dict(N=-1), dict(K=0), dict(S=-1), dict(na=-1),
                               dict(r=0), dict(off=None), dict(off=P + 4), dict(ids=None), dict(sc=P + 2), dict(st=P + 1), dict(ldx=56),
                               dict(ldy=31), dict(ldyi=31), dict(X=None), dict(X=P + 2), dict(ldx=68), dict(Y=None), dict(A=None), dict(B=P + 8),
                               dict(Y=P + 1), dict(Yin=P + 1), dict(V=P + 4), dict(Yin=P, Y=P, ldy=40)])
def test_apply_invalid(qg, o):
    assert apply(qg, **o) == qg.QG_ERR_INVALID_ARG


@pytest.mark.parametrize("o", [dict(wt=1), dict(r=4), dict(r=12), dict(r=136), dict(K=60, ldx=64), dict(yit=1), dict(T=1 << 21), dict(na=1 << 17)])
def test_apply_unsupported(qg, o):
    assert apply(qg, **o) == qg.QG_ERR_UNSUPPORTED


@pytest.mark.parametrize("o", [dict(xt=7), dict(gt=5), dict(acc=2), dict(lddy=31), dict(ldx=63), dict(lddx=63), dict(dX=None), dict(dA=None), dict(dB=P + 4),
                               dict(dY=None), dict(dY=P + 1), dict(V=None), dict(V=P + 8), dict(ldx=68), dict(lddx=68), dict(dX=P + 2), dict(dXi=P + 8),
                               dict(ws=P + 8)])
def test_grad_invalid(qg, o):
    assert grad(qg, **o) == qg.QG_ERR_INVALID_ARG


def test_grad_unsupported_and_workspace(qg):
    assert grad(qg, gt=qg.QG_BF16) == qg.QG_ERR_UNSUPPORTED
    assert grad(qg, wt=qg.QG_BF16, gt=qg.QG_BF16) == qg.QG_ERR_UNSUPPORTED
    need = qg.qg_lora_grad_workspace_bytes(4, 2, 2, 8, 32, 64)
    assert need >= 4 * 8 * 4 and grad(qg, wsb=need - 1) == qg.QG_ERR_WORKSPACE_TOO_SMALL and grad(qg, ws=None) == qg.QG_ERR_WORKSPACE_TOO_SMALL
    need = qg.qg_lora_apply_workspace_bytes(8192, 1, 32, 8192, 8192)
    assert need >= 8192 * 32 * 4
    assert apply(qg, T=8192, N=8192, K=8192, r=32, ldx=8192, ldy=8192, ldyi=8192, wsb=need - 1) == qg.QG_ERR_WORKSPACE_TOO_SMALL


def test_nothing_to_do(qg):
    for o in (dict(T=0), dict(N=0, ldy=0, ldyi=0), dict(S=0)):
        assert apply(qg, **o) == qg.QG_OK
    assert grad(qg, T=0, acc=1) == qg.QG_OK


def dgrad(qg, **o):
    a = dict(dY=P, yt=qg.QG_BF16, W=P, s=P, z=None, dX=P, xt=qg.QG_BF16, M=4, N=32, K=64, bits=4, bs=32, ws=P, wsb=1 << 30)
    a.update(o)
    return qg.lib().qgemm_nbits_dgrad(*[a[k] for k in ("dY", "yt", "W", "s", "z", "dX", "xt", "M", "N", "K", "bits", "bs", "ws", "wsb")], None)


def test_dgrad(qg):
    for o in (dict(yt=4), dict(xt=-1), dict(M=-1), dict(N=-3), dict(K=-32), dict(K=48), dict(dX=None), dict(dX=P + 4), dict(dY=None), dict(dY=P + 2),
              dict(W=P + 8), dict(s=None), dict(z=P + 2)):
        assert dgrad(qg, **o) == qg.QG_ERR_INVALID_ARG, o
    for o in (dict(bits=5), dict(bits=0), dict(bs=16), dict(M=1 << 21), dict(K=1 << 25)):
        assert dgrad(qg, **o) == qg.QG_ERR_UNSUPPORTED, o
    assert dgrad(qg, M=0) == qg.QG_OK and dgrad(qg, K=0) == qg.QG_OK
    assert qg.lib().qgemm_codebook4_dgrad(P, 2, P, None, P, P, 2, 4, 32, 64, 32, P, 1 << 30, None) == qg.QG_ERR_INVALID_ARG


def test_grad_list_and_clip(qg):
    T = qg._GradTensor
    n = ctypes.c_int64(-1)
    init = lambda *ts: qg.lib().qg_grad_list_init((T * max(1, len(ts)))(*ts), len(ts), ctypes.byref(n))
    assert init() == qg.QG_OK and n.value == 0
    big = (1 << 14) // 2
    ts = (T * 4)(T(P, None, big + 1, 0, qg.QG_BF16, 0), T(None, None, 0, 0, qg.QG_F32, 0), T(P + 2, P + 4, big, 0, qg.QG_F16, 0), T(P, P, 5, 0, qg.QG_F32, 0))
    assert qg.lib().qg_grad_list_init(ts, 4, ctypes.byref(n)) == qg.QG_OK
    # 16 KB a chunk, counted from the 16-byte boundary before a tensor
    assert [t.first_chunk for t in ts] == [0, 2, 2, 4] and n.value == 5 and ts[0].out == P
    for bad in (T(None, P, 4, 0, 0, 0), T(P, P, -1, 0, 0, 0), T(P, P, 4, 0, 5, 0), T(P + 2, P, 4, 0, 0, 0), T(P, P + 1, 4, 0, 1, 0)):
        assert init(bad) == qg.QG_ERR_INVALID_ARG
    need = qg.qg_clip_grad_norm_workspace_bytes(5)
    clip = lambda *a: qg.lib().qg_clip_grad_norm(*a, None)
    assert clip(P, 4, 5, -1.0, 0.0, P, P, need) == qg.QG_ERR_INVALID_ARG
    assert clip(P, 4, 5, float("nan"), 0.0, P, P, need) == qg.QG_ERR_INVALID_ARG
    assert clip(P, 4, 5, 1.0, float("nan"), P, P, need) == qg.QG_ERR_INVALID_ARG
    assert clip(None, 4, 5, 1.0, 0.0, P, P, need) == qg.QG_ERR_INVALID_ARG
    assert clip(P, 4, 5, 1.0, 0.0, None, P, need) == qg.QG_ERR_INVALID_ARG
    assert clip(P, 0, 5, 1.0, 0.0, P, P, need) == qg.QG_ERR_INVALID_ARG
    assert clip(P, 4, 5, 1.0, 0.0, P, None, need) == qg.QG_ERR_WORKSPACE_TOO_SMALL
    assert clip(P, 4, 5, 1.0, 0.0, P, P, need - 1) == qg.QG_ERR_WORKSPACE_TOO_SMALL
