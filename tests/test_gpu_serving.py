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
    "growing_scores": dict(T=3, lens=[900, 400], window=700, sinks=4, growth=15.0, **SLIDING),
    "growing_scores_chunk": dict(T=100, lens=[400], window=300, sinks=4, growth=20.0, **SLIDING),
    "large_scores": dict(T=1, lens=[300, 70], window=200, sinks=4, q_scale=64.0, **SLIDING),
    "capped_large_scores": dict(T=1, lens=[300, 70], window=200, sinks=4, q_scale=64.0,
                                softcap=20.0, **SLIDING),
    "scale_zero": dict(T=2, lens=[150, 64], window=100, sinks=4, scale=0.0, **SLIDING),
    "scale_negative": dict(T=2, lens=[150, 64], window=100, sinks=4, scale=-0.05, **SLIDING),
    "scale_negative_capped": dict(T=2, lens=[150, 64], window=100, sinks=4, scale=-0.05,
                                  softcap=5.0, **SLIDING),
    "many_sequences": dict(T=1, lens=[(7 * i) % 90 for i in range(333)], window=40, sinks=3, hq=2,
                           hkv=1, dim=256),
    "group100": dict(T=3, lens=[90, 3], window=70, sinks=4, hq=100, hkv=1, dim=256),
    "wide_growing": dict(T=20, lens=[400], window=300, sinks=4, growth=20.0, hq=16, hkv=1,
                         dim=512, shared=True),
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
    "scale_negative": dict(T=1, lens=[40, 3, 8], prefix=100, scale=-0.1, **GLOBAL),
    "growing": dict(T=2, lens=[300, 40], prefix=400, growth=20.0, **GLOBAL),
    "group128": dict(T=1, lens=[40, 3], prefix=100, hq=128, hkv=1, dim=512, window=0),
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


# --------------------------------------------------- errors seen by the device
@pytest.mark.parametrize("dim,hkv,shared", [(256, 8, False), (512, 1, True)])
@pytest.mark.parametrize("split", [0, 5])
def test_sequences_shorter_than_the_step(dim, hkv, shared, split):
    """0 < L < T is reported; the tokens that have a position are right, the others 0."""
    c = ref.make_case(1, 9, [4, 30, 0, 8], 16, hkv, dim, window=20, sinks=3, shared=shared)
    run_and_check(c, split, status=binding.GDATTN_ERR_DEVICE_SEQLEN)


def test_negative_and_too_long_lengths_are_reported():
    c = ref.make_case(2, 1, [40, 40, 40], 16, 8, 256, window=20, sinks=3, capacity=23)
    good = Call(c, max_seqlen=1000).run()[0].clone()
    call = Call(c, max_seqlen=1000)
    call.args[3] = torch.tensor([40, -7, 40], dtype=torch.int32, device="cuda")
    out, lse = call.run(binding.GDATTN_ERR_DEVICE_SEQLEN)
    assert torch.equal(out[:, [0, 2]], good[:, [0, 2]])
    assert (out[:, 1] == 0).all() and (lse[:, 1] == -float("inf")).all()
    # Longer than the ring can serve: never outside the cache, the others untouched.
    c = ref.make_case(3, 1, [40, 64], 16, 1, 512, window=0, prefix=30, shared=True)
    good = Call(c).run()[0].clone()
    call = Call(c)
    call.args[3] = torch.tensor([40, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    out, _ = call.run(binding.GDATTN_ERR_DEVICE_SEQLEN)
    assert torch.equal(out[:, 0], good[:, 0])


@pytest.mark.parametrize("plen", [-5, 65])
def test_prefix_length_out_of_range_is_clamped(plen):
    c = ref.make_case(4, 1, [9, 70], 16, 1, 512, window=0, prefix=64 if plen > 0 else 0,
                      prefix_rows=64, shared=True)
    call = Call(c)
    call.prefix[2].fill_(plen)
    out, lse = call.run(binding.GDATTN_ERR_DEVICE_SEQLEN)
    ref.check(out, lse, ref.reference(c, "cuda"))


@pytest.mark.parametrize("kind", ["sink", "prefix", "wide"])
def test_a_wait_that_runs_out_is_reported(kind):
    """Every CTA leaves its first K tile unloaded: the call ends, says so, and a
    re-initialised workspace then gives the right result."""
    args = dict(sink=dict(T=1, lens=[500, 90], window=300, sinks=4, **SLIDING),
                prefix=dict(T=1, lens=[9, 30], prefix=200, **GLOBAL),
                wide=dict(T=2, lens=[300, 20], window=100, sinks=4, hq=16, hkv=2, dim=512))[kind]
    c = ref.make_case(5, **args)
    call = Call(c, flags=binding.GDATTN_FLAG_TEST_WITHHOLD_KV)
    call.run(binding.GDATTN_ERR_DEVICE_TIMEOUT)
    call.desc.flags = 0
    binding.workspace_init(call.ws.t)
    out, lse = call.run()
    ref.check(out, lse, ref.reference(c, "cuda"))


# ----------------------------------------------- streams, graphs, workspaces
def test_captured_call_follows_lengths_and_prefix():
    """One graph, replayed with other lengths, another prefix length and other rows."""
    for kind in ("sink", "prefix"):
        base = dict(T=2, window=100, sinks=4, **SLIDING) if kind == "sink" else dict(T=1, **GLOBAL)
        more = {} if kind == "sink" else dict(prefix_rows=200)
        cases = []
        for k, lens in enumerate(([150, 30, 0], [2, 99, 260], [101, 102, 3])):
            cap = 105 if kind == "sink" else 260
            px = {} if kind == "sink" else dict(prefix=(200, 77, 0)[k])
            cases.append(ref.make_case(k, lens=lens, capacity=cap, **base, **more, **px))
        call = Call(cases[0], max_seqlen=1000)
        call.run()
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            call.enqueue()
        for c in cases + cases[::-1]:
            for t, new in zip(call.args, (c.q, c.k, c.v, c.lens)):
                if t is not None:
                    t.copy_(new)
            if call.prefix:
                call.prefix[0].copy_(c.pk)
                call.prefix[2].fill_(c.plen)
            graph.replay()
            graph.replay()
            torch.cuda.synchronize()
            assert binding.check_device_status(call.ws.t) == binding.GDATTN_OK
            ref.check(call.out.t, call.lse.t, ref.reference(c, "cuda"), kind)


def test_calls_on_two_streams_with_their_own_workspaces():
    cases = [ref.make_case(k, T=1, lens=[900 + k, 70], window=500, sinks=4, **SLIDING)
             for k in range(2)]
    calls = [Call(c) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(20):
        for call, s in zip(calls, streams):
            call.enqueue(stream=s)
    torch.cuda.synchronize()
    for call, c in zip(calls, cases):
        assert binding.check_device_status(call.ws.t) == binding.GDATTN_OK
        ref.check(call.out.t, call.lse.t, ref.reference(c, "cuda"))


def test_one_workspace_serves_different_calls_in_turn():
    """Sinks, prefix and the decode kernels that were there, back to back on one
    workspace, each call's result as alone and bit for bit the same every time."""
    cases = [ref.make_case(1, T=1, lens=[900, 70, 300], window=500, sinks=4, **SLIDING),
             ref.make_case(2, T=1, lens=[9, 300], prefix=333, **GLOBAL),
             ref.make_case(3, T=70, lens=[90, 71], window=60, sinks=4, **SLIDING),
             ref.make_case(4, T=1, lens=[700, 2], window=0, prefix=100, **SLIDING)]
    calls = [Call(c) for c in cases]
    d = binding.make_desc(16, 8, 256, 500, 0.0, 1 / 16, False, 512)
    q = torch.randn((3, 16, 256), device="cuda").to(torch.bfloat16)
    kv = torch.randn((2, 3, 512, 8, 256), device="cuda").to(torch.bfloat16)
    lens = torch.tensor([900, 70, 300], dtype=torch.int32, device="cuda")
    n = max([binding.workspace_size(3, 900, d)] + [call.ws.t.numel() for call in calls])
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    binding.workspace_init(ws)
    want = [tuple(t.clone() for t in call.run()) for call in calls]
    old = binding.decode(q, kv[0], kv[1], lens, d, 900)
    for call in calls:
        call.ws.t = ws
    for _ in range(5):
        for call in calls:
            call.out.t.fill_(float("nan"))
            call.enqueue()
            got = binding.decode(q, kv[0], kv[1], lens, d, 900, workspace=ws)
            assert torch.equal(got[0], old[0]) and torch.equal(got[1], old[1])
        for call, w in zip(calls, want):
            assert torch.equal(call.out.t, w[0]) and torch.equal(call.lse.t, w[1])
    assert binding.check_device_status(ws) == binding.GDATTN_OK


def test_strided_caches_and_offsets_past_32_bits():
    """Sequences far apart in one buffer: more than 2^31 elements in front of the last."""
    c = ref.make_case(6, T=2, lens=[150, 90], window=100, sinks=4, **SLIDING)
    rows = c.k[0].numel()
    stride = 2 ** 31 // rows * rows + 8 * rows
    call = Call(c)
    big = []
    for t in (c.k, c.v):
        flat = torch.empty(stride + rows, dtype=torch.bfloat16, device="cuda")
        for b in range(2):
            flat[b * stride:b * stride + rows].copy_(t[b].reshape(-1))
        big.append(flat.as_strided(c.k.shape, (stride, *c.k[0].stride())))
    call.args[1:3] = big
    call.desc.cache_batch_stride = stride
    out, lse = call.run()
    ref.check(out, lse, ref.reference(c, "cuda"))
    # and writes there
    new = torch.randn((2, 8, 256), device="cuda").to(torch.bfloat16)
    at = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    slot = torch.tensor([5, 101], dtype=torch.int32, device="cuda")
    binding.cache_write(new, new, at, slot, call.desc, big[0], big[1])
    for t in big:
        assert torch.equal(t[0, 5], new[0]) and torch.equal(t[1, 101], new[1])
        assert torch.equal(t[1, 80], dev(c.k[1, 80]) if t is big[0] else dev(c.v[1, 80]))


def test_a_long_ring_of_many_tiles():
    """A context far longer than its ring, and a ring of many tiles and pieces."""
    run_and_check(ref.make_case(7, T=1, lens=[100000], window=5000, sinks=4, hq=2, hkv=1,
                                dim=256))


# -------------------------------------------------------------- as one server
def test_serving_steps_end_to_end():
    """Prompts written by a slot map and attended in one chunk, then decode steps of the
    batch with one token each, sliding layer with pins: every step's output against the
    definition over all rows so far.  A second layer keeps an fp8 copy of its rows."""
    g = torch.Generator().manual_seed(0)
    hq, hkv, dim, window, sinks = 16, 8, 256, 48, 4
    capacity = sinks + window + 40 - 1
    B, prompt = 3, [40, 17, 33]
    desc = binding.make_desc(hq, hkv, dim, window, 30.0, 1 / 16, False, capacity)
    k = torch.full((B, capacity, hkv, dim), ref.NAN, dtype=torch.bfloat16, device="cuda")
    v = k.clone()
    codes = torch.zeros((2, B, capacity, hkv, dim), dtype=torch.uint8, device="cuda")
    scale = torch.zeros((2, B, hkv, capacity), device="cuda")
    rows = [[torch.zeros((0, hkv, dim), dtype=torch.bfloat16) for _ in range(B)] for _ in range(2)]

    def write(new):
        n = sum(new)
        fused = torch.randn((n, hq + 2 * hkv, dim), generator=g).to(torch.bfloat16)
        at = 0
        for b, m in enumerate(new):
            for i in range(2):
                part = fused[at:at + m, hq + i * hkv:hq + (i + 1) * hkv]
                rows[i][b] = torch.cat([rows[i][b], part])
            at += m
        lens = torch.tensor([len(r) for r in rows[0]], dtype=torch.int32, device="cuda")
        m = binding.slot_map(lens, torch.tensor(new, dtype=torch.int32, device="cuda"), n + 2,
                             capacity, sinks)
        f = torch.cat([fused, fused[:2]]).cuda()  # two rows behind the step's last
        kr, vr = f[:, hq:hq + hkv], f[:, hq + hkv:]
        binding.cache_write(kr, vr, m.seq, m.slot, desc, k, v)
        binding.cache_write_fp8(kr, vr, m.seq, m.slot, desc, codes[0], codes[1], scale[0],
                                scale[1])
        return lens

    def attend(T, lens):
        q = torch.randn((T, B, hq, dim), generator=g).to(torch.bfloat16)
        out, lse = binding.decode_sink(q.cuda(), k, v, lens, desc, 1000, sinks)
        c = ref.Case(q, rows[0], rows[1], k.cpu(), v.cpu(), lens.cpu(), window, sinks, capacity,
                     30.0, 1 / 16)
        ref.check(out, lse, ref.reference(c, "cuda"), f"T = {T}")

    lens = write(prompt)
    attend(17, lens)
    for step in range(60):
        lens = write([1, 1 if step % 3 else 0, 1])
        attend(1, lens)
    # the fp8 copy holds the same rows, rounded
    slot = ref.slot_of(torch.arange(len(rows[0][0])), sinks, capacity)
    last = len(rows[0][0]) - 1
    value, s = ref.e4m3_rows(rows[1][0][last])
    got = codes[1, 0, slot[last]].cpu().view(torch.float8_e4m3fn).double()
    assert torch.equal(got, value)
    assert torch.equal(scale[1, 0, :, slot[last]].cpu().double(), s)


def test_fp8_rows_written_here_are_what_the_fp8_decode_reads():
    """A ring filled by gdattn_cache_write_fp8 and read by gdattn_decode_fp8."""
    import oracle
    orc = oracle.get()
    g = torch.Generator().manual_seed(3)
    hq, hkv, dim, window = 16, 8, 256, 64
    lens = [100, 64, 7]
    B = len(lens)
    desc = binding.make_desc(hq, hkv, dim, window, 0.0, 1 / 16, False, window)
    codes = torch.zeros((2, B, window, hkv, dim), dtype=torch.uint8, device="cuda")
    scale = torch.zeros((2, B, hkv, window), device="cuda")
    lens_t = torch.tensor(lens, dtype=torch.int32, device="cuda")
    m = binding.slot_map(lens_t, lens_t, sum(lens), window)
    kv = [torch.randn((sum(lens), hkv, dim), generator=g).to(torch.bfloat16).cuda()
          for _ in range(2)]
    binding.cache_write_fp8(kv[0], kv[1], m.seq, m.slot, desc, codes[0], codes[1], scale[0],
                            scale[1])
    q = torch.randn((B, hq, dim), generator=g).to(torch.bfloat16)
    out, lse = binding.decode_fp8(q.cuda(), codes[0], codes[1], scale[0], scale[1], lens_t, desc,
                                  max(lens))
    o_ref, l_ref = orc.decode_fp8(q, codes[0].cpu(), codes[1].cpu(), scale[0].cpu(),
                                  scale[1].cpu(), lens_t.cpu(), window, 0.0, 1 / 16)
    # the entry point's own gates
    assert (out.cpu().double() - torch.as_tensor(o_ref)).abs().max() <= 8e-3
    assert (lse.cpu().double() - torch.as_tensor(l_ref)).abs().max() <= 1e-3


# ------------------------------------------- what one call leaves for the next
def test_pieces_of_a_pair_are_joined_from_this_call():
    """head_dim 512, few rows: each CTA of a pair joins its half of the dims from pieces
    and sums of this call, not of the one before on the same workspace."""
    args = dict(T=1, window=2500, sinks=4, hq=16, hkv=1, dim=512, shared=True)
    calls = [Call(ref.make_case(k, lens=lens, capacity=2504, q_scale=4.0 + 8 * k, **args),
                  max_seqlen=4000) for k, lens in enumerate(([3000, 2600], [900, 2700]))]
    want = [tuple(t.clone() for t in call.run()) for call in calls]
    for call, w in zip(calls, want):
        ref.check(*w, ref.reference(call.c, "cuda"))
        call.ws.t = calls[0].ws.t
    got = []
    for _ in range(100):
        for call in calls:
            call.enqueue()
            got.append((call.out.t.clone(), call.lse.t.clone()))
    for i, (out, lse) in enumerate(got):
        assert torch.equal(out, want[i % 2][0]) and torch.equal(lse, want[i % 2][1]), i


def test_a_prefix_that_the_call_in_front_appends_to():
    """Sequence 0's cache serves as the others' prefix right behind its own append."""
    g = torch.Generator(device="cuda").manual_seed(0)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)

    hq, dim, P, B = 16, 512, 4000, 3
    desc = binding.make_desc(hq, 1, dim, 0, 0.0, dim ** -0.5, True, P)
    cache, own = normal(1, P, 1, dim), normal(B, P, 1, dim)
    plen = torch.tensor([P], dtype=torch.int32, device="cuda")
    lens = torch.tensor([5, 1, 70], dtype=torch.int32, device="cuda")
    q0, q = normal(1, hq, dim), normal(1, B, hq, dim)
    ws = [torch.empty(n, dtype=torch.uint8, device="cuda")
          for n in (binding.workspace_size(1, P, desc),
                    binding.prefix_workspace_size(B, 1, 100, P, desc))]
    for w in ws:
        binding.workspace_init(w)

    def behind():
        return binding.decode_prefix(q, cache[0], None, plen, own, None, lens, desc, 100,
                                     workspace=ws[1])[0]

    for _ in range(20):
        new = normal(1, 1, dim) * 8
        binding.decode_append(q0, new, None, cache, None, plen, desc, P, workspace=ws[0])
        got = behind()
        torch.cuda.synchronize()
        assert torch.equal(cache[0, P - 1], new[0])
        assert torch.equal(got, behind())


def test_new_rows_far_above_a_length():
    """Positions below -2^31 read as that; no row has a slot."""
    m = binding.slot_map(dev(i32([-5, 9])), dev(i32([2 ** 31 - 1, 2])), 4, 8, 2)
    assert m.pos.tolist() == [-2 ** 31] * 4 and m.slot.tolist() == [-1] * 4
    assert m.seq.tolist() == [0] * 4 and m.start.tolist() == [0, 2 ** 31 - 1, 2 ** 31 - 1]


def test_a_step_without_rows():
    desc = binding.make_desc(16, 8, 256, 0, 0.0, 1.0, False, 8)
    kv = torch.ones((2, 1, 8, 8, 256), device="cuda").to(torch.bfloat16)
    rows = torch.zeros((0, 32, 256), dtype=torch.bfloat16, device="cuda")
    at = torch.zeros(0, dtype=torch.int32, device="cuda")
    binding.cache_write(rows[:, 16:24], rows[:, 24:], at, at, desc, kv[0], kv[1])
    assert (kv == 1).all()
