"""A workspace that a binding allocates for itself belongs to the stream that uses it (CPU only)."""
import contextlib

import pytest
import torch

import paged_kv_cache_372_b200 as pa


class FakeStream:
    def __init__(self, handle, device=None):
        self.cuda_stream, self.device = handle, device


@pytest.fixture
def streams(monkeypatch):
    """torch's streams replaced by handles; the list holds the ones current now."""
    current = [0]

    @contextlib.contextmanager
    def use(stream):
        current.append(stream.cuda_stream)
        yield
        current.pop()

    monkeypatch.setattr(torch.cuda, "Stream", FakeStream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", FakeStream)
    monkeypatch.setattr(torch.cuda, "stream", use)
    return current


@pytest.mark.parametrize("stream,handle", [(None, 0), (FakeStream(77), 77), (88, 88)])
def test_scratch_is_allocated_with_its_stream_current(streams, stream, handle):
    assert pa._scratch(lambda *a: (a, streams[-1]), stream, 0, 1, 2) == ((1, 2), handle)
    assert streams == [0]


class FakeCuda(torch.Tensor):
    """A CPU tensor that says it is on CUDA device 0."""
    is_cuda = property(lambda self: True)
    device = property(lambda self: torch.device("cuda", 0))

    def get_device(self):
        return 0


def fake(*shape, dtype=torch.float16):
    return torch.zeros(shape, dtype=dtype).as_subclass(FakeCuda)


class Allocated(Exception):
    pass


@pytest.mark.parametrize("stream,handle", [(None, 0), (FakeStream(77), 77), (88, 88)])
def test_prefill_paged_allocates_on_its_stream(streams, monkeypatch, stream, handle):
    def alloc(*a, **kw):
        raise Allocated(streams[-1])

    monkeypatch.setattr(pa, "alloc_prefill_workspace", alloc)
    q, pool = fake(4, 2, 64), fake(3, 2, 16, 64)
    tab, ctx, cu = (fake(*s, dtype=torch.int32) for s in ((2, 4), (2,), (3,)))
    with pytest.raises(Allocated) as e:
        pa.pa_prefill_paged(q, q, pool, pool, tab, ctx, cu, 0.1, 64, stream=stream)
    assert e.value.args[0] == handle


S, P8 = "e4m3", torch.uint8
DECODES = {
    "pa_decode": lambda q, kv, kp, k8, c, **kw: pa.pa_decode(q, q, kp, kp, *c, **kw),
    "pa_decode_append": lambda q, kv, kp, k8, c, **kw: pa.pa_decode_append(q, q, kv, kv, kp, kp, *c, **kw),
    "pa_decode_shared": lambda q, kv, kp, k8, c, **kw: pa.pa_decode_shared(q, q, kp, kp, *c, **kw),
    "pa_decode_fp8": lambda q, kv, kp, k8, c, **kw: pa.pa_decode_fp8(q, q, k8, k8, *c, 1.0, 1.0, **kw),
    "pa_decode_quant": lambda q, kv, kp, k8, c, **kw: pa.pa_decode_quant(q, q, k8, k8, *c, S, None, None, **kw),
    "pa_decode_quant_blocks":
        lambda q, kv, kp, k8, c, **kw: pa.pa_decode_quant_blocks(q, q, k8, k8, *c, S, None, None, **kw),
    "pa_decode_shared_quant":
        lambda q, kv, kp, k8, c, **kw: pa.pa_decode_shared_quant(q, q, k8, k8, *c, S, None, None, **kw),
    "pa_decode_shared_quant_blocks":
        lambda q, kv, kp, k8, c, **kw: pa.pa_decode_shared_quant_blocks(q, q, k8, k8, *c, S, None, None, **kw),
}


@pytest.mark.parametrize("name", DECODES)
@pytest.mark.parametrize("stream,handle", [(None, 0), (FakeStream(77), 77), (88, 88)])
def test_decode_allocates_on_its_stream(streams, monkeypatch, name, stream, handle):
    def alloc(*a, **kw):
        raise Allocated(streams[-1])

    monkeypatch.setattr(pa, "alloc_workspace", alloc)
    q, kv, kp, k8 = fake(2, 2, 64), fake(2, 2, 64), fake(3, 2, 16, 64), fake(3, 2, 16, 64, dtype=P8)
    tab, ctx = fake(2, 4, dtype=torch.int32), fake(2, dtype=torch.int32)
    with pytest.raises(Allocated) as e:
        DECODES[name](q, kv, kp, k8, (tab, ctx, 0.1, 64), stream=stream)
    assert e.value.args[0] == handle
