"""Continuous-batching operators on the GPU against their float64 definitions."""
import pytest
import torch

import serving_ref as ref
from decode_attention_09_b200 import binding
from gpu_helpers import Guarded, require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def desc_of(c, split=0, flags=0):
    hkv, dim = c.k.shape[2], c.k.shape[3]
    return binding.make_desc(c.q.shape[2], hkv, dim, c.window, c.softcap, c.scale, c.v is None,
                             c.capacity, 0, split, flags)


def dev(t):
    return None if t is None else t.cuda()


class Call:
    """One attention call with guard bytes around everything it writes."""

    def __init__(self, c, split=0, max_seqlen=None, flags=0):
        self.c, self.desc = c, desc_of(c, split, flags)
        T, B, Hq, D = c.q.shape
        self.max_seqlen = max_seqlen or max(T, int(c.lens.max()))
        self.args = [dev(t) for t in (c.q, c.k, c.v, c.lens)]
        self.prefix = None
        if c.pk is not None:
            self.prefix = [dev(c.pk), dev(c.pv),
                           torch.tensor([c.plen], dtype=torch.int32, device="cuda")]
            n = binding.prefix_workspace_size(B, T, self.max_seqlen, c.pk.shape[0], self.desc)
        else:
            n = binding.sink_workspace_size(B, T, self.max_seqlen, self.desc, c.sinks)
        assert n > 0
        self.ws = Guarded((n,), torch.uint8)
        binding.workspace_init(self.ws.t)
        self.out = Guarded((T, B, Hq, D), torch.bfloat16, fill=float("nan"))
        self.lse = Guarded((T, B, Hq), torch.float32, fill=float("nan"))

    def enqueue(self, stream=None):
        q, k, v, lens = self.args
        kw = dict(out=self.out.t, lse=self.lse.t, workspace=self.ws.t, stream=stream)
        if self.prefix:
            pk, pv, plen = self.prefix
            binding.decode_prefix(q, pk, pv, plen, k, v, lens, self.desc, self.max_seqlen, **kw)
        else:
            binding.decode_sink(q, k, v, lens, self.desc, self.max_seqlen, self.c.sinks, **kw)

    def run(self, status=binding.GDATTN_OK):
        self.enqueue()
        st = binding.check_device_status(self.ws.t)
        assert st == status, binding.status_string(st)
        for g, n in ((self.out, "out"), (self.lse, "lse"), (self.ws, "workspace")):
            g.check(n)
        return self.out.t, self.lse.t


def run_and_check(c, split=0, status=binding.GDATTN_OK, max_seqlen=None):
    out, lse = Call(c, split, max_seqlen).run(status)
    ref.check(out, lse, ref.reference(c, "cuda"))


SLIDING = dict(hq=16, hkv=8, dim=256)
SINKS = {
    "one_token": dict(T=1, lens=[1], window=512, sinks=4, **SLIDING),
    "below_the_pins": dict(T=1, lens=[2, 3, 4, 5], window=512, sinks=4, **SLIDING),
    "window_of_one": dict(T=1, lens=[1, 2, 9, 40], window=1, sinks=3, **SLIDING),
    "window_edges": dict(T=1, lens=[63, 64, 65, 67, 68, 69, 128, 131, 132, 133], window=64,
                         sinks=4, **SLIDING),
    "wrapped": dict(T=1, lens=[1500, 700, 900], window=300, sinks=5, capacity=311, **SLIDING),
    "no_pins": dict(T=1, lens=[100, 700], window=130, sinks=0, **SLIDING),
    "many_pins": dict(T=1, lens=[50, 69, 70, 71, 500], window=40, sinks=70, **SLIDING),
    "pins_of_a_tile": dict(T=1, lens=[64, 300], window=64, sinks=64, **SLIDING),
    "padding_entries": dict(T=1, lens=[0, 80, 0, 1, 0], window=64, sinks=4, **SLIDING),
    "softcap": dict(T=1, lens=[400, 77], window=200, sinks=4, softcap=50.0, heavy=4.0, **SLIDING),
    "verify4": dict(T=4, lens=[4, 5, 70, 1000, 0], window=96, sinks=6, softcap=30.0, **SLIDING),
    "verify8_wrapped": dict(T=8, lens=[900, 333], window=128, sinks=4, capacity=150, **SLIDING),
    "chunk65": dict(T=65, lens=[65, 200, 500], window=100, sinks=4, **SLIDING),
    "chunk200_pins_in_window": dict(T=200, lens=[200, 230], window=64, sinks=33, **SLIDING),
    "chunk130_wrapped": dict(T=130, lens=[700], window=77, sinks=9, capacity=260, **SLIDING),
    "group1": dict(T=3, lens=[100, 9], window=60, sinks=4, hq=8, hkv=8, dim=256),
    "group4": dict(T=2, lens=[150, 64], window=60, sinks=4, hq=8, hkv=2, dim=256),
    "group3": dict(T=50, lens=[150, 60], window=60, sinks=4, hq=9, hkv=3, dim=256),
    "group16_shared": dict(T=9, lens=[150, 40], window=70, sinks=4, hq=16, hkv=1, dim=256,
                           shared=True),
    "group128": dict(T=2, lens=[90], window=70, sinks=4, hq=128, hkv=1, dim=256),
    "wide_shared": dict(T=1, lens=[300, 20, 0], window=100, sinks=4, hq=16, hkv=1, dim=512,
                        shared=True),
    "wide_shared_chunk": dict(T=40, lens=[300, 41], window=100, sinks=4, hq=16, hkv=1, dim=512,
                              shared=True, softcap=50.0),
    "wide_separate": dict(T=5, lens=[300, 20], window=100, sinks=4, hq=16, hkv=2, dim=512),
    "wide_group2": dict(T=70, lens=[200, 71], window=90, sinks=10, hq=4, hkv=2, dim=512),
}


@pytest.mark.parametrize("split", [0, 1, 7, 148])
@pytest.mark.parametrize("name", list(SINKS))
def test_sinks(name, split):
    run_and_check(ref.make_case(seed=len(name), **SINKS[name]), split)


GLOBAL = dict(hq=16, hkv=1, dim=512, shared=True, window=0)
PREFIX = {
    "one_row": dict(T=1, lens=[1], prefix=1, **GLOBAL),
    "no_prefix": dict(T=1, lens=[1, 70, 130], prefix=0, **GLOBAL),
    "tile_edges": dict(T=1, lens=[63, 64, 65], prefix=64, **GLOBAL),
    "odd": dict(T=1, lens=[1, 2, 200, 7], prefix=333, **GLOBAL),
    "rows_behind": dict(T=1, lens=[5, 90], prefix=100, prefix_rows=257, **GLOBAL),
    "padding_entries": dict(T=1, lens=[0, 40, 0], prefix=130, **GLOBAL),
    "batch70": dict(T=1, lens=[1 + i % 9 for i in range(70)], prefix=200, softcap=50.0, **GLOBAL),
    "verify3": dict(T=3, lens=[3, 50, 4], prefix=150, **GLOBAL),
    "chunk30": dict(T=30, lens=[30, 95], prefix=150, **GLOBAL),
    "group8": dict(T=1, lens=[9, 30], prefix=200, hq=8, hkv=1, dim=512, shared=True, window=0),
    "wide_separate": dict(T=2, lens=[9, 300], prefix=200, hq=16, hkv=2, dim=512, window=0),
    "sliding_window": dict(T=1, lens=[1, 50, 128, 200], prefix=300, window=128, softcap=50.0,
                           **SLIDING),
    "window_past_prefix": dict(T=1, lens=[300, 400], prefix=300, window=128, **SLIDING),
    "window_over_all": dict(T=1, lens=[10, 40], prefix=100, window=1000, **SLIDING),
    "window_chunk": dict(T=70, lens=[70, 90, 71], prefix=100, window=60, **SLIDING),
    "window_verify_wrapped": dict(T=4, lens=[500, 20, 4], prefix=90, window=64, capacity=67,
                                  **SLIDING),
    "batch65_sliding": dict(T=1, lens=[1 + 3 * i for i in range(65)], prefix=77, window=0,
                            **SLIDING),
    "group4": dict(T=2, lens=[40, 3], prefix=100, hq=8, hkv=2, dim=256, window=0),
    "group3": dict(T=1, lens=[40, 3, 8], prefix=100, hq=9, hkv=3, dim=256, window=50),
    "group16_shared": dict(T=1, lens=[40, 3], prefix=100, hq=16, hkv=1, dim=256, shared=True,
                           window=0),
}


@pytest.mark.parametrize("split", [0, 1, 7, 74])
@pytest.mark.parametrize("name", list(PREFIX))
def test_prefix(name, split):
    run_and_check(ref.make_case(seed=len(name), **PREFIX[name]), split)


# -------------------------------------------------------- slot maps and writes
def i32(x):
    return torch.tensor(x, dtype=torch.int32)


SLOT_MAPS = {
    "one": ([1], [1], 1, 8, 0),
    "none_new": ([5, 9], [0, 0], 3, 16, 4),
    "no_rows": ([5, 9], [2, 1], 0, 16, 4),
    "decode": ([1, 2, 700, 31, 0], [1, 1, 1, 1, 0], 6, 28, 4),
    "mixed": ([40, 0, 7, 300, 1, 2000], [40, 0, 1, 200, 0, 2000], 2300, 130, 4),
    "prompt_longer_than_ring": ([5000], [5000], 5000, 100, 10),
    "rows_cut": ([50, 60], [50, 60], 70, 200, 0),
    "new_above_length": ([3, 10, 5], [5, -2, 5], 12, 20, 2),
    "ring_of_one": ([9, 4], [9, 4], 13, 4, 3),
    "many_empty": ([7] * 3000, [1 if i % 7 == 0 else 0 for i in range(3000)], 500, 64, 4),
    "many_ones": ([7] * 3000, [1] * 3000, 3000, 64, 4),
}


@pytest.mark.parametrize("name", list(SLOT_MAPS))
def test_slot_map(name):
    lens, new, n_rows, capacity, sinks = SLOT_MAPS[name]
    B = len(lens)
    want = ref.slot_map(lens, new, n_rows, capacity, sinks)
    bufs = [Guarded((n,), torch.int32, fill=77) for n in (B + 1, n_rows, n_rows, n_rows)]
    got = binding.slot_map(dev(i32(lens)), dev(i32(new)), n_rows, capacity, sinks,
                           out=binding.RowMap(*(b.t for b in bufs)))
    torch.cuda.synchronize()
    for g, b, w, field in zip(got, bufs, want, binding.RowMap._fields):
        b.check(field)
        assert torch.equal(g.cpu(), w), field


def write_inputs(B, new, capacity, sinks, H, D, shared, seed=0, extra_rows=3):
    g = torch.Generator().manual_seed(seed)
    lens = [n + 17 * (b % 3) for b, n in enumerate(new)]
    n_rows = sum(new) + extra_rows
    fused = torch.randn((n_rows, 2 + (1 if shared else 2) * H, D), generator=g)
    fused = (fused * torch.exp2(torch.randint(-20, 21, (n_rows, 1, 1), generator=g).float()))
    fused = fused.to(torch.bfloat16)
    rows = [fused[:, 2:2 + H]] + ([] if shared else [fused[:, 2 + H:]])
    _, seq, _, slot = ref.slot_map(lens, new, n_rows, capacity, sinks)
    return rows, seq, slot


WRITES = [  # B, new, capacity, sinks, Hkv, D, K = V
    (1, [1], 8, 0, 8, 256, False), (3, [1, 0, 70], 40, 4, 8, 256, False),
    (2, [300, 9], 64, 4, 1, 512, True), (2, [33, 2], 64, 0, 2, 512, False),
    (1, [5], 9, 3, 1, 256, True), (4, [100, 1, 1, 31], 128, 4, 3, 256, False),
]


@pytest.mark.parametrize("case", WRITES)
def test_cache_write(case):
    B, new, C, S, H, D, shared = case
    rows, seq, slot = write_inputs(B, new, C, S, H, D, shared)
    desc = binding.make_desc(2 * H, H, D, 0, 0.0, 1.0, shared, C)
    caches = [Guarded((B, C, H, D), torch.bfloat16, fill=3.0) for _ in rows]
    fused = dev(rows[0]._base)
    args = [fused[:, 2 + i * H:2 + (i + 1) * H] for i in range(len(rows))]
    binding.cache_write(args[0], None if shared else args[1], dev(seq), dev(slot), desc,
                        caches[0].t, None if shared else caches[1].t)
    torch.cuda.synchronize()
    keep = slot >= 0
    for cache, r in zip(caches, rows):
        cache.check("cache")
        want = torch.full((B, C, H, D), 3.0, dtype=torch.bfloat16)
        want[seq[keep].long(), slot[keep].long()] = r[keep]
        assert torch.equal(cache.t.cpu(), want)


@pytest.mark.parametrize("case", WRITES)
def test_cache_write_fp8(case):
    B, new, C, S, H, D, shared = case
    rows, seq, slot = write_inputs(B, new, C, S, H, D, shared, seed=1)
    rows[0][0] = 0.0  # a row of zeros
    rows[0][-4 if len(seq) > 4 else 0, 0, 3] = -0.0
    desc = binding.make_desc(2 * H, H, D, 0, 0.0, 1.0, shared, C)
    codes = [Guarded((B, C, H, D), torch.uint8, fill=0x31) for _ in rows]
    scales = [Guarded((B, H, C), torch.float32, fill=9.0) for _ in rows]
    fused = dev(rows[0]._base)
    args = [fused[:, 2 + i * H:2 + (i + 1) * H] for i in range(len(rows))]
    binding.cache_write_fp8(args[0], None if shared else args[1], dev(seq), dev(slot), desc,
                            codes[0].t, None if shared else codes[1].t, scales[0].t,
                            None if shared else scales[1].t)
    torch.cuda.synchronize()
    keep = slot >= 0
    at = seq[keep].long(), slot[keep].long()
    untouched = torch.ones((B, C), dtype=torch.bool)
    untouched[at] = False
    for code, scale, r in zip(codes, scales, rows):
        code.check("codes")
        scale.check("scales")
        value, s = ref.e4m3_rows(r[keep])
        got = code.t.cpu().view(torch.float8_e4m3fn)
        assert torch.equal(got[at].double(), value)
        assert torch.equal(scale.t.cpu()[at[0], :, at[1]].double(), s)
        assert (code.t.cpu()[untouched] == 0x31).all()
        assert (scale.t.cpu().permute(0, 2, 1)[untouched] == 9.0).all()


def test_rows_out_of_range_are_skipped():
    """Sequences and slots that are not there write nothing."""
    H, D, B, C = 2, 256, 2, 4
    desc = binding.make_desc(4, H, D, 0, 0.0, 1.0, True, C)
    rows = torch.randn((6, H, D), device="cuda").to(torch.bfloat16)
    cache = Guarded((B, C, H, D), torch.bfloat16, fill=1.0)
    seq, slot = i32([0, 2, -1, 1, 1, 0]), i32([0, 0, 1, 4, -1, 1 << 30])
    binding.cache_write(rows, None, dev(seq), dev(slot), desc, cache.t)
    torch.cuda.synchronize()
    cache.check("cache")
    want = torch.ones((B, C, H, D), dtype=torch.bfloat16)
    want[0, 0] = rows[0].cpu()
    assert torch.equal(cache.t.cpu(), want)


def test_fp8_codes_of_every_pair_of_mantissas():
    """The kernel's division against the definition for every mantissa of a row's
    largest magnitude, every mantissa of a value and the exponents down to zero codes,
    at scales of ordinary size and at the ends of fp32's range."""
    H, D = 1, 256
    m = torch.arange(128, dtype=torch.float64)
    big = 1 + m / 128                       # every bf16 mantissa
    rows = []
    for shift in (0, -100, 120):            # exponent of the row
        for e in range(0, 20):              # the values' exponents below it
            x = torch.cat([big[:, None], -(big[None, :] * 2.0 ** -e).expand(128, -1)], 1)
            x[:, 1:] = torch.where(x[:, 1:].abs() > big[:, None], -0.5 * big[:, None], x[:, 1:])
            rows.append(torch.cat([x, x[:, 1:].abs(), x[:, :0]], 1)[:, :256] * 2.0 ** shift)
    rows = torch.cat(rows).to(torch.bfloat16)
    rows = torch.cat([rows, torch.zeros(rows.shape[0], D - rows.shape[1], dtype=torch.bfloat16)], 1)
    n = rows.shape[0]
    desc = binding.make_desc(1, H, D, 0, 0.0, 1.0, True, n)
    codes = torch.zeros((1, n, H, D), dtype=torch.uint8, device="cuda")
    scale = torch.zeros((1, H, n), device="cuda")
    at = torch.arange(n, dtype=torch.int32, device="cuda")
    binding.cache_write_fp8(rows.cuda().view(n, H, D), None, torch.zeros_like(at), at, desc, codes,
                            None, scale)
    value, s = ref.e4m3_rows(rows)
    assert torch.equal(scale.cpu().view(-1).double(), s)
    assert torch.equal(codes.cpu().view(n, D).view(torch.float8_e4m3fn).double(), value)
