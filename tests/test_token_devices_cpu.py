"""The calls around tokens refuse operands that are on different GPUs, or on another one than the current: with tensors that only say so, since
every call here returns before anything is enqueued."""
import pytest
import torch

from test_train_abi_cpu import qg  # noqa: F401  (the fixture)


class On(torch.Tensor):
    """A tensor that says it is on GPU `at`."""

    at = 0
    is_cuda = True

    def get_device(self):
        return self.at


def on(at, t):
    t = t.as_subclass(On)
    t.at = at
    return t


def operands(qg):
    T, V, k, E, H, I = 4, 50, 3, 8, 256, 128
    f, i64, i32, half, u8 = torch.float32, torch.int64, torch.int32, torch.float16, torch.uint8
    z = torch.zeros
    yield lambda a: qg.qg_token_logprobs(a.pop("X"), a.pop("targets"), a.pop("logprob"), **a), dict(
        X=z(T, V), targets=z(T, dtype=i64), logprob=z(T), entropy=z(T), lse=z(T), top_ids=z(T, k, dtype=i64), top_logprobs=z(T, k), status=z(1, dtype=i32))
    yield lambda a: qg.qg_token_logprobs_grad(a.pop("X"), a.pop("targets"), a.pop("lse"), a.pop("d"), a.pop("dX"), **a), dict(
        X=z(T, V), targets=z(T, dtype=i64), lse=z(T), d=z(T), dX=z(T, V), entropy=z(T), d_entropy=z(T))
    yield lambda a: qg.qmoe_route_topk(*a.values()), dict(logits=z(T, E), ids=z(T, k, dtype=i32), weights=z(T, k))
    yield lambda a: qg.qmoe_tokens_fused(**a, bits=4, block_size=64), dict(
        x=z(T, H, dtype=half), expert_ids=z(T, k, dtype=i32), expert_weights=z(T, k), y=z(T, H), status=z(1, dtype=i32), workspace=z(1 << 20, dtype=u8),
        fc1_w=z(E, 2 * I, H // 2, dtype=u8), fc1_scales=z(E, 2 * I, H // 64, dtype=half), fc1_zp=z(E, 2 * I, H // 64, dtype=half), fc1_bias=z(E, 2 * I, dtype=half),
        fc2_w=z(E, H, I // 2, dtype=u8), fc2_scales=z(E, H, I // 64, dtype=half), fc2_zp=z(E, H, I // 64, dtype=half), fc2_bias=z(E, H, dtype=half))
    t = qg.QGAdamWList.__new__(qg.QGAdamWList)
    t.count, t.chunks = 1, 1

    def step(a):
        t.table, t.workspace = a["table"], a["table"]
        qg.qg_adamw_step(t, lr=a["lr"], step=a["step"], max_norm=1.0, norm=a["norm"], workspace=a["workspace"])

    yield step, dict(table=z(4096, dtype=u8), lr=z(1), step=z(1, dtype=i64), norm=z(1), workspace=z(4096, dtype=u8))


@pytest.mark.parametrize("call", range(5))
def test_one_device_and_the_current_one(qg, monkeypatch, call):
    f, given = list(operands(qg))[call]
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: pytest.fail("went on to the launch"), raising=False)
    for name in given:
        with pytest.raises(ValueError, match="one GPU"):
            f({n: on(1 if n == name else 0, t) for n, t in given.items()})
        with pytest.raises(ValueError, match="a GPU"):
            f({n: on(-1 if n == name else 0, t) for n, t in given.items()})
    with pytest.raises(ValueError, match="current"):
        f({n: on(1, t) for n, t in given.items()})
