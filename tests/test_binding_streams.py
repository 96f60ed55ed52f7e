"""What the tensor wrappers allocate belongs to the stream of the call, on the CPU: the
library and torch's CUDA side are replaced by recorders."""
import contextlib
import types

import pytest
import torch

from decode_attention_09_b200 import binding


class Stream:
    cuda_stream = 0x77


@pytest.fixture
def allocated(monkeypatch):
    """The stream that was current at each allocation, in order."""
    current, got = [None], []

    @contextlib.contextmanager
    def on(stream):
        current.append(stream)
        yield
        current.pop()

    def recording(fn):
        def call(*a, **kw):
            got.append(current[-1])
            return fn(*a, **kw)
        return call

    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "device", lambda d: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: Stream())
    monkeypatch.setattr(torch, "empty", recording(torch.empty))
    monkeypatch.setattr(torch, "empty_like", recording(torch.empty_like))
    monkeypatch.setattr(torch.Tensor, "new_empty", recording(torch.Tensor.new_empty))
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: None)
    monkeypatch.setattr(binding, "_on", lambda *a: None)
    monkeypatch.setattr(binding, "_call", lambda *a: None)
    calls = types.SimpleNamespace(**{
        "gdattn_" + n: lambda *a: 0
        for n in ("decode", "decode_append", "decode_fp8", "decode_multi", "combine",
                  "workspace_init", "decode_sink", "decode_prefix", "slot_map")}, **{
        "gdattn_" + n: lambda *a: 512
        for n in ("workspace_size", "multi_workspace_size", "sink_workspace_size",
                  "prefix_workspace_size")})
    monkeypatch.setattr(binding, "lib", lambda: calls)
    return got


B, H, HKV, D, C = 2, 16, 8, 256, 8
CALLS = {}


def call(fn):
    CALLS[fn.__name__] = fn
    return fn


def desc(**kw):
    return binding.make_desc(H, HKV, D, kw.get("window", 4), 0.0, 1.0, False, C)


def z(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


def caches():
    return z(B, C, HKV, D), z(B, C, HKV, D)


@call
def decode(stream):
    binding.decode(z(B, H, D), *caches(), z(B, dtype=torch.int32), desc(), 8, stream=stream)


@call
def decode_append(stream):
    binding.decode_append(z(B, H, D), z(B, HKV, D), z(B, HKV, D), *caches(),
                          z(B, dtype=torch.int32), desc(), 8, stream=stream)


@call
def decode_fp8(stream):
    codes = z(B, C, HKV, D, dtype=torch.uint8)
    scale = z(B, HKV, C, dtype=torch.float32)
    binding.decode_fp8(z(B, H, D), codes, codes, scale, scale, z(B, dtype=torch.int32), desc(), 8,
                       stream=stream)


@call
def decode_multi(stream):
    binding.decode_multi(z(3, B, H, D), *caches(), z(B, dtype=torch.int32), desc(), 8,
                         stream=stream)


@call
def combine(stream):
    binding.combine(z(B, H, 2, D, dtype=torch.float32), z(B, H, 2, dtype=torch.float32),
                    stream=stream)


@call
def decode_sink(stream):
    binding.decode_sink(z(3, B, H, D), *caches(), z(B, dtype=torch.int32), desc(), 8, 2,
                        stream=stream)


@call
def decode_prefix(stream):
    binding.decode_prefix(z(3, B, H, D), z(5, HKV, D), z(5, HKV, D), z(1, dtype=torch.int32),
                          *caches(), z(B, dtype=torch.int32), desc(), 8, stream=stream)


@call
def slot_map(stream):
    binding.slot_map(z(B, dtype=torch.int32), z(B, dtype=torch.int32), 4, C, stream=stream)


@pytest.mark.parametrize("name", list(CALLS))
def test_a_call_allocates_on_its_stream(name, allocated):
    stream = Stream()
    CALLS[name](stream)
    assert allocated and all(s is stream for s in allocated)
    allocated.clear()
    CALLS[name](None)  # the current stream's memory, without a detour
    assert allocated and all(s is None for s in allocated)


@pytest.mark.parametrize("alloc", [
    lambda s: binding.alloc_workspace(B, 8, desc(), "cpu", s),
    lambda s: binding.alloc_sink_workspace(B, 1, 8, desc(), 2, "cpu", s),
    lambda s: binding.alloc_prefix_workspace(B, 1, 8, 5, desc(), "cpu", s)])
def test_a_workspace_is_allocated_where_it_is_cleared(alloc, allocated):
    stream = Stream()
    alloc(stream)
    assert len(allocated) == 1 and allocated[0] is stream
