"""Continuous-batching calls that the header allows and ordinary use rarely makes."""
import pytest
import torch

import serving_ref as ref
from decode_attention_09_b200 import binding
from gpu_helpers import GUARD_BYTE, GUARD_BYTES, require_gpu
from test_gpu_serving import GLOBAL, SLIDING, Call

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


# ------------------------------------------------------------- the same bits
CAPPED = {  # tiles that end inside a box of rows, in slots that no token attends
    "decode": dict(T=1, lens=[70, 3, 130], window=100, sinks=4, **SLIDING),
    "verify": dict(T=4, lens=[900, 333, 5], window=500, sinks=4, **SLIDING),
    "chunk": dict(T=70, lens=[200, 75], window=100, sinks=4, capacity=190, **SLIDING),
    "wide": dict(T=2, lens=[300, 20], window=100, sinks=4, hq=16, hkv=1, dim=512, shared=True),
    "wide_separate": dict(T=5, lens=[300, 20], window=100, sinks=4, hq=16, hkv=2, dim=512),
    "prefix": dict(T=1, lens=[5, 90], prefix=101, prefix_rows=257, **GLOBAL),
    "prefix_window": dict(T=2, lens=[40, 3], prefix=75, prefix_rows=100, window=50, **SLIDING),
}


@pytest.mark.parametrize("softcap", [0.0, 50.0])
@pytest.mark.parametrize("name", list(CAPPED))
def test_slots_that_nobody_attends_have_no_say(name, softcap):
    """Whatever stands in them, the result is the same, bit for bit."""
    want = None
    for fill in (0.0, 3e4, -3e4, float("nan")):
        c = ref.make_case(len(name), softcap=softcap, **CAPPED[name])
        for t in (c.k, c.v, c.pk, c.pv):
            if t is not None:
                t.masked_fill_(t.isnan(), fill)
        got = [t.clone() for t in Call(c).run()]
        if want is None:
            ref.check(*got, ref.reference(c, "cuda"))
            want = got
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), fill


@pytest.mark.parametrize("softcap", [0.0, 50.0])
@pytest.mark.parametrize("name", list(CAPPED))
def test_what_ran_before_has_no_say(name, softcap):
    """Nor has what other calls left on the chip: rows of other sizes between the calls."""
    call = Call(ref.make_case(len(name), softcap=softcap, **CAPPED[name]))
    wide = call.desc.head_dim == 512
    others = []
    for size in (0.01, 300.0):
        c = ref.make_case(1, T=1, lens=[2000] * (8 if wide else 2), window=1900, sinks=4,
                          hq=16, hkv=1 if wide else 8, dim=512 if wide else 256, shared=wide)
        for t in (c.k, c.v):
            if t is not None:
                t *= size
        others.append(Call(c))
    want = None
    for i in range(12):
        others[i % 2].enqueue()
        got = [t.clone() for t in call.run()]
        want = want or got
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), i


# ---------------------------------------------------------------- alignment
class AtHalf:
    """A device tensor that starts at an odd multiple of 16 bytes, between guard bytes."""

    def __init__(self, like):
        n = like.numel() * like.element_size()
        self.lo, self.hi = GUARD_BYTES + 16, GUARD_BYTES + 16 + n
        self.raw = torch.full((self.hi + GUARD_BYTES,), GUARD_BYTE, dtype=torch.uint8,
                              device="cuda")
        self.t = self.raw[self.lo:self.hi].view(like.dtype).view(like.shape)
        assert self.t.data_ptr() % 32 == 16

    def check(self, what):
        assert (self.raw[:self.lo] == GUARD_BYTE).all(), f"{what}: written in front"
        assert (self.raw[self.hi:] == GUARD_BYTE).all(), f"{what}: written behind"


HALF = {  # what a block writes, by its rows and how its unit is cut
    "whole_units": dict(T=1, lens=[300, 70], window=200, sinks=4, **SLIDING),
    "whole_blocks": dict(T=130, lens=[300], window=100, sinks=4, **SLIDING),
    "few_rows": dict(T=1, lens=[900, 70], window=700, sinks=4, **SLIDING),
    "some_rows": dict(T=4, lens=[900, 333], window=500, sinks=4, softcap=50.0, **SLIDING),
    "full_blocks": dict(T=70, lens=[900], window=700, sinks=4, **SLIDING),
    "wide_few_rows": dict(T=1, lens=[900], window=700, sinks=4, hq=4, hkv=1, dim=512),
    "wide_some_rows": dict(T=1, lens=[900, 20, 0], window=700, sinks=4, hq=16, hkv=1, dim=512,
                           shared=True),
    "wide_full_blocks": dict(T=20, lens=[900], window=700, sinks=4, hq=16, hkv=1, dim=512,
                             shared=True, softcap=30.0),
    "prefix": dict(T=1, lens=[40, 3], prefix=100, window=0, **SLIDING),
    "wide_prefix": dict(T=2, lens=[40, 3, 300], prefix=333, **GLOBAL),
}


@pytest.mark.parametrize("split", [1, 0])
@pytest.mark.parametrize("name", list(HALF))
def test_outputs_and_workspace_on_a_16_byte_boundary(name, split):
    """16 bytes are all that a pointer has to be aligned to: the result is the same, bit
    for bit, as on wider boundaries."""
    c = ref.make_case(seed=len(name), **HALF[name])
    call = Call(c, split)
    want = [t.clone() for t in call.run()]
    ref.check(*want, ref.reference(c, "cuda"))
    for moved in (("out",), ("ws",), ("out", "ws")):
        call = Call(c, split)
        for n in moved:
            setattr(call, n, AtHalf(getattr(call, n).t))
        binding.workspace_init(call.ws.t)
        call.out.t.fill_(float("nan"))
        got = call.run()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), moved


# ------------------------------------------------------------ the ends of 32 bits
@pytest.mark.parametrize("dim,hkv,shared", [(256, 8, False), (512, 1, True)])
@pytest.mark.parametrize("sinks", [0, 3])
@pytest.mark.parametrize("split", [0, 5])
def test_the_widest_window(dim, hkv, shared, sinks, split):
    """A window of 2^31 - 1 (everything is visible), also over sequences shorter than
    the step, whose tokens in front of position 0 get 0."""
    kw = dict(hq=16, hkv=hkv, dim=dim, window=2 ** 31 - 1, sinks=sinks, shared=shared)
    for T, lens, status in ((9, [4, 30, 0, 8], binding.GDATTN_ERR_DEVICE_SEQLEN),
                            (70, [3, 200], binding.GDATTN_ERR_DEVICE_SEQLEN),
                            (1, [1, 300, 64], binding.GDATTN_OK),
                            (66, [66, 130], binding.GDATTN_OK)):
        c = ref.make_case(T, T, lens, **kw)
        out, lse = Call(c, split).run(status)
        ref.check(out, lse, ref.reference(c, "cuda"))


# ------------------------------------------------------------------ fp8 codes
@pytest.mark.parametrize("dim", [256, 512])
def test_fp8_codes_byte_by_byte(dim):
    """Codes as bytes: a zero has its sign, whichever way the scale makes the kernel
    divide, and so has what rounds to zero; a row of zeros has codes and scale 0."""
    g = torch.Generator().manual_seed(dim)
    x = torch.randn((60, 1, dim), generator=g).to(torch.bfloat16)
    x[:, :, ::7], x[:, :, 1::7] = -0.0, 0.0
    x[:, :, 2::7] *= 2.0 ** -14  # below half of e4m3's smallest number
    x *= torch.exp2(torch.arange(-120.0, 120.0, 4.0))[:, None, None].to(torch.bfloat16)
    x[5], x[6] = 0.0, -0.0
    n = x.shape[0]
    desc = binding.make_desc(1, 1, dim, 0, 0.0, 1.0, True, n)
    codes = torch.full((1, n, 1, dim), 0x55, dtype=torch.uint8, device="cuda")
    scale = torch.full((1, 1, n), -1.0, device="cuda")
    at = torch.arange(n, dtype=torch.int32, device="cuda")
    binding.cache_write_fp8(x.cuda(), None, torch.zeros_like(at), at, desc, codes, None, scale)
    s = x.float().abs().amax(-1) / 448
    want = (x.float() / s[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
    want[s[:, 0] == 0] = 0
    assert (want == 0x80).sum() > 60 * dim // 7 - 200  # the signs are there to be lost
    assert torch.equal(scale.cpu().view(-1), s.view(-1))
    assert torch.equal(codes.cpu().view(n, 1, dim), want)
