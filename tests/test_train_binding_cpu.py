"""What the fine-tuning entry points and their Python calls check on the host, beyond tests/test_train_abi_cpu.py: nothing here
needs a GPU, and no pointer is followed."""
import math

import pytest

from test_train_abi_cpu import P, qg  # noqa: F401  (qg: the fixture)


@pytest.mark.parametrize("zp", [math.nan, math.inf, -math.inf, 65505.0, -1e6])
@pytest.mark.parametrize("sizes", [(4, 32, 64), (0, 32, 64), (4, 0, 64)])
def test_uniform_zero_points_as_in_the_forward_pass(qg, zp, sizes):
    """A zero point that fp16 does not hold is refused by both passes, whatever the sizes."""
    M, N, K = sizes
    ws = (P, 1 << 30, None)
    assert qg.lib().qgemm_nbits_uniform_zp(P, qg.QG_F16, P, P, zp, P, qg.QG_F16, M, N, K, 4, 32, *ws) == qg.QG_ERR_INVALID_ARG
    assert qg.lib().qgemm_nbits_uniform_zp_dgrad(P, qg.QG_F16, P, P, zp, P, qg.QG_F16, M, N, K, 4, 32, *ws) == qg.QG_ERR_INVALID_ARG


def test_uniform_zero_points_at_the_ends(qg):
    for zp in (65504.0, -65504.0, 7.5):
        assert qg.lib().qgemm_nbits_uniform_zp_dgrad(P, qg.QG_F16, P, P, zp, P, qg.QG_F16, 0, 32, 64, 4, 32, None, 0, None) == qg.QG_OK


def test_activation_gradient_operands(qg):
    """Types, shapes and order of every operand: the library takes addresses, so nothing else would notice."""
    import torch

    M, N, K, bs = 4, 32, 128, 64
    half, single = dict(dtype=torch.float16), dict(dtype=torch.float32)
    good = dict(dY=torch.zeros(M, N), W=torch.zeros(N, K // 2, dtype=torch.uint8), scales=torch.zeros(N, K // bs, **half),
                zp=torch.zeros(N, K // bs, **half), absmax=torch.zeros(N, K // bs, **single), codebook=torch.zeros(16, **single), dX=torch.zeros(M, K))
    strided = lambda t: torch.zeros(t.shape[0], 2 * t.shape[1], dtype=t.dtype)[:, ::2]

    def nbits(**o):
        g = dict(good, **o)
        qg.qgemm_nbits_dgrad(g["dY"], g["W"], g["scales"], g["zp"], g["dX"], bits=4, block_size=bs)

    def uniform(**o):
        g = dict(good, **o)
        qg.qgemm_nbits_uniform_zp_dgrad(g["dY"], g["W"], g["scales"], 8.0, g["dX"], bits=4, block_size=bs)

    def codebook(**o):
        g = dict(good, **o)
        qg.qgemm_codebook4_dgrad(g["dY"], g["W"], g["codebook"], g["absmax"], g["dX"], block_size=bs)

    common = [dict(W=good["W"].int()), dict(W=strided(good["W"])), dict(W=good["W"][:-1]), dict(dY=strided(good["dY"])), dict(dX=strided(good["dX"]))]
    for o in common + [dict(scales=good["scales"].float()), dict(scales=strided(good["scales"])), dict(scales=good["scales"].flatten()[:N]),
                       dict(scales=good["scales"].bfloat16())]:
        for f in (nbits, uniform):
            with pytest.raises(ValueError):
                f(**o)
    for o in (dict(zp=good["zp"].float()), dict(zp=good["zp"].to(torch.uint8)), dict(zp=good["zp"][:, :1]), dict(zp=good["zp"][:-1]), dict(zp=strided(good["zp"]))):
        with pytest.raises(ValueError):
            nbits(**o)
    for o in common + [dict(absmax=good["absmax"].half()), dict(absmax=strided(good["absmax"])), dict(codebook=torch.zeros(15)),
                       dict(codebook=torch.zeros(16, **half)), dict(codebook=torch.zeros(32)[::2])]:
        with pytest.raises(ValueError):
            codebook(**o)


def test_clipping_operands(qg):
    """The norm is written as one float32 value, and the list's addresses are followed on the device."""
    import torch

    empty = qg.QGGradList.__new__(qg.QGGradList)  # refused before anything of it is used
    for norm in (torch.zeros(1, dtype=torch.float16), torch.zeros(1, dtype=torch.float64), torch.zeros(0), torch.zeros(2), torch.zeros(1)):
        with pytest.raises(ValueError, match="norm"):
            qg.qg_clip_grad_norm(empty, 1.0, norm)
    with pytest.raises(ValueError, match="GPU"):
        qg.QGGradList([torch.zeros(4)])


@pytest.mark.parametrize("status", ["uint8", "int64", "none"])
def test_adapter_status(qg, status):
    """The status is written as an int32."""
    import torch

    status = torch.zeros(0, dtype=torch.int32) if status == "none" else torch.zeros(1, dtype=getattr(torch, status))
    X, Y, A, B, V = torch.zeros(4, 64), torch.zeros(4, 32), torch.zeros(1, 8, 64), torch.zeros(1, 32, 8), torch.zeros(4, 8)
    off, ids = torch.tensor([0, 4]), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="status"):
        qg.qg_lora_apply(X, off, ids, A, B, None, None, Y, status=status)
    with pytest.raises(ValueError, match="status"):
        qg.qg_lora_grad(Y, X, V, off, ids, A, B, None, None, None, torch.zeros_like(A), torch.zeros_like(B), status=status)


class FakeTorch:
    """Stands in for torch where a call looks for scratch memory: records the stream that each piece is made on."""

    uint8 = "uint8"

    class Piece:
        def __init__(self, nbytes, stream):
            self.nbytes, self.stream = nbytes, stream

        def data_ptr(self):
            return P

        def record_stream(self, stream):
            pass

    class Stream:
        cuda_stream = 7

    def __init__(self):
        fake = self
        self.now, self.made = "current", []

        class Within:
            def __init__(self, stream):
                self.stream = stream

            def __enter__(self):
                self.before, fake.now = fake.now, self.stream

            def __exit__(self, *e):
                fake.now = self.before

        self.cuda = type("cuda", (), dict(stream=Within))
        self._C = type("_C", (), dict(_cuda_getCurrentRawStream=staticmethod(lambda device: 3)))

    def empty(self, nbytes, dtype, device):
        self.made.append(self.Piece(nbytes, self.now))
        return self.made[-1]


class FakeTensor:
    device = "cuda:0"

    def get_device(self):
        return 0


def test_scratch_memory_belongs_to_the_stream_of_the_call(qg, monkeypatch):
    """Memory of another stream's pool may still be in use there by an earlier call, and goes back there too early."""
    fake, s = FakeTorch(), FakeTorch.Stream()
    monkeypatch.setattr(qg, "_TORCH", fake)
    raw, at, size, piece = qg._stream_and_workspace(64, None, FakeTensor(), s)
    assert (raw, at, size, piece.stream, fake.now) == (7, P, 64, s, "current")
    raw, at, size, piece = qg._stream_and_workspace(64, None, FakeTensor(), None)
    assert (raw, at, size, piece.stream) == (3, P, 64, "current")
    assert qg._stream_and_workspace(0, None, FakeTensor(), s)[1:] == (None, 0, None) and len(fake.made) == 2


def test_scratch_memory_of_the_other_calls(qg, monkeypatch):
    fake, s = FakeTorch(), FakeTorch.Stream()
    monkeypatch.setattr(qg, "_TORCH", fake)
    for stream in (s, None):
        piece, size = qg._workspace(lambda: 128, None, "cuda:0", stream)
        assert size == 128 and piece.stream == (stream or "current") and fake.now == "current"
    assert qg._workspace(lambda: 0, None, "cuda:0", s) == (None, 0) and len(fake.made) == 2
