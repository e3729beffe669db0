"""Which stream's memory a result is taken from, with torch's stream calls replaced (no GPU needed)."""

import contextlib

import pytest
import torch

from compressed_index_matmul_b200 import layer


class FakeStream:
    def __init__(self, raw):
        self.cuda_stream = raw


@pytest.fixture
def streams(monkeypatch):
    """Current stream 7, default stream 0; what is entered around the allocation is recorded.  As torch's
    own constructor, an external stream of handle 0 is one from the pool."""
    entered = []

    @contextlib.contextmanager
    def enter(s):
        entered.append(s.cuda_stream)
        yield

    monkeypatch.setattr(torch.cuda, "stream", enter)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda raw, device=None: FakeStream(raw or 1234))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: FakeStream(0))
    monkeypatch.setattr(torch.cuda, "Stream", FakeStream)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 7, raising=False)
    return entered


@pytest.mark.parametrize("stream,want", [
    (None, []), (7, []), (FakeStream(7), []),  # the current stream's memory as it is
    (0, [0]), (FakeStream(0), [0]),            # the default stream, not one from the pool
    (9, [9]), (FakeStream(9), [9]),
])
def test_results_come_from_the_streams_memory(streams, stream, want):
    t = layer._new((2, 3), torch.float16, torch.device("cpu"), stream)
    assert t.shape == (2, 3) and t.dtype is torch.float16
    assert streams == want


@pytest.mark.parametrize("call", ["forward", "forward_rotated"])
def test_plain_forwards_take_their_streams_memory_too(streams, monkeypatch, call):
    L = layer.VQLinear.__new__(layer.VQLinear)
    L.N, L.K, L.act_dtype, L.device, L.handle = 16, 64, layer.B.VQ_F16, torch.device("cpu"), None
    L.planes = L.codebooks = None
    L.t = {"scales": None}
    given = []
    for name in ("vq_linear_forward", "vq_linear_forward_rotated"):
        monkeypatch.setattr(layer.B, name, lambda *a: given.append(a[-1]))
    x = torch.zeros((2, 64), dtype=torch.float16)
    args = (x,) if call == "forward" else (x, torch.ones(64, dtype=torch.int8))
    for stream, want in ((None, []), (0, [0]), (9, [9])):
        streams.clear()
        y = getattr(L, call)(*args, stream=stream)
        assert y.shape == (2, 16) and y.dtype is torch.float16
        assert streams == want and given[-1] is stream
    streams.clear()
    assert getattr(L, call)(*args, y=y, stream=9) is y and streams == []
