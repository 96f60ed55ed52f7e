"""Wrappers that allocate outputs and workspace themselves, called for a stream that is not
the current one: nothing on the current stream gets that memory while it is in use."""
import pytest
import torch

import serving_ref as ref
from decode_attention_09_b200 import binding
from gpu_helpers import require_gpu
from test_gpu_serving import GLOBAL, SLIDING, Call

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def sink():
    c = ref.make_case(1, T=1, lens=[900, 70, 300], window=500, sinks=4, **SLIDING)
    call = Call(c)
    q, k, v, lens = call.args
    return lambda **kw: binding.decode_sink(q, k, v, lens, call.desc, call.max_seqlen, c.sinks,
                                            **kw)


def prefix():
    c = ref.make_case(2, T=2, lens=[9, 300], prefix=333, **GLOBAL)
    call = Call(c)
    q, k, v, lens = call.args
    return lambda **kw: binding.decode_prefix(q, *call.prefix, k, v, lens, call.desc,
                                              call.max_seqlen, **kw)


def ring(T=1):
    g = torch.Generator(device="cuda").manual_seed(0)
    d = binding.make_desc(16, 8, 256, 500, 0.0, 1 / 16, False, 512)
    q = torch.randn((T, 3, 16, 256), generator=g, device="cuda").to(torch.bfloat16)
    kv = torch.randn((2, 3, 512, 8, 256), generator=g, device="cuda").to(torch.bfloat16)
    return d, q, kv, torch.tensor([900, 70, 300], dtype=torch.int32, device="cuda")


def decode():
    d, q, kv, lens = ring()
    return lambda **kw: binding.decode(q[0], kv[0], kv[1], lens, d, 900, **kw)


def verify():
    d, q, kv, lens = ring(4)
    return lambda **kw: binding.decode_multi(q, kv[0], kv[1], lens, d, 900, **kw)


def slots():
    lens = torch.arange(1, 200, dtype=torch.int32, device="cuda")
    return lambda **kw: binding.slot_map(lens, lens, 20000, 100, 4, **kw)


@pytest.mark.parametrize("as_handle", [False, True])
@pytest.mark.parametrize("make", [sink, prefix, decode, verify, slots])
def test_a_call_on_another_stream(make, as_handle):
    call = make()
    want = [t.clone() for t in call()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(5):
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)  # the call below starts some 10 ms from now
        got = call(stream=side.cuda_stream if as_handle else side)
        # What the current stream allocates meanwhile, of all sizes up to the workspace's.
        mine = [torch.full((1 << n,), 7, dtype=torch.uint8, device="cuda")
                for n in range(8, 26) for _ in range(3)]
        side.synchronize()
        assert all((t == 7).all() for t in mine)
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        del mine, got


def test_the_default_stream_by_its_handle():
    call = sink()
    want = call()
    for handle in (0, torch.cuda.default_stream().cuda_stream):
        got = call(stream=handle)
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
