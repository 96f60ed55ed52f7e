"""Continuous-batching operators without a GPU: what the host checks refuse, and the
float64 definitions the GPU tests use, pinned against independent forms."""
import ctypes
import math

import pytest
import torch

import serving_ref as ref
from decode_attention_09_b200 import binding
from decode_attention_09_b200 import build as libbuild

A = 0x100000  # a 16-byte-aligned fake device address (never dereferenced)
INVALID = binding.GDATTN_ERR_INVALID_ARG
UNSUPPORTED = binding.GDATTN_ERR_UNSUPPORTED
MISALIGNED = binding.GDATTN_ERR_MISALIGNED
WORKSPACE = binding.GDATTN_ERR_WORKSPACE


@pytest.fixture(scope="module", autouse=True)
def lib():
    libbuild.build()
    return binding.lib()


def sliding(**kw):
    d = dict(n_q_heads=16, n_kv_heads=8, head_dim=256, window=1024, softcap=0.0, scale=1 / 16,
             kv_shared=False, cache_capacity=1028)
    d.update(kw)
    return binding.make_desc(**d)


def shared(**kw):
    d = dict(n_q_heads=16, n_kv_heads=1, head_dim=512, window=0, kv_shared=True,
             cache_capacity=4096)
    d.update(kw)
    return sliding(**d)


def sink(desc=None, q=A, k=A, v=A, lens=A, batch=1, T=1, max_seqlen=8192, n_sink=4, out=A, lse=A,
         ws=A, ws_bytes=1 << 12):
    return binding.decode_sink_raw(q, k, v, lens, batch, T, max_seqlen, desc or sliding(), n_sink,
                                   out, lse, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,expect", [
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID),
    (dict(lens=None), INVALID), (dict(out=None), INVALID), (dict(batch=0), INVALID),
    (dict(T=0), INVALID), (dict(T=(1 << 20) + 1, max_seqlen=1 << 21), INVALID),
    (dict(T=5, max_seqlen=4), INVALID), (dict(max_seqlen=0), INVALID),
    (dict(n_sink=-1), INVALID), (dict(n_sink=1028), INVALID),
    (dict(n_sink=5), INVALID),               # C < n_sink + window
    (dict(T=2), INVALID),                    # C < n_sink + window + T - 1
    (dict(q=A + 8), MISALIGNED), (dict(k=A + 2), MISALIGNED), (dict(v=A + 8), MISALIGNED),
    (dict(out=A + 4), MISALIGNED), (dict(lens=A + 1), MISALIGNED), (dict(lse=A + 2), MISALIGNED),
    (dict(ws=None), WORKSPACE), (dict(ws=A + 8), MISALIGNED),
])
def test_sink_refusals(kw, expect):
    assert sink(**kw) == expect


@pytest.mark.parametrize("desc_kw,expect", [
    (dict(window=0), INVALID),               # every token is visible: gdattn_decode's case
    (dict(n_q_heads=12), INVALID), (dict(softcap=-1.0), INVALID), (dict(flags=4), INVALID),
    (dict(cache_batch_stride=8), INVALID),
    (dict(head_dim=128), UNSUPPORTED), (dict(n_q_heads=129 * 8), UNSUPPORTED),
])
def test_sink_refuses_descriptors(desc_kw, expect):
    assert sink(sliding(**desc_kw)) == expect


def test_a_cache_that_never_wraps_needs_no_ring():
    assert sink(sliding(cache_capacity=8192), T=8192, ws=None) == WORKSPACE
    assert sink(sliding(cache_capacity=8191), T=8192, ws=None) == INVALID


def prefix(desc=None, q=A, pk=A, pv=None, plen=A, rows=64, k=A, v=None, lens=A, batch=1, T=1,
           max_seqlen=100, out=A, lse=A, ws=A, ws_bytes=1 << 12):
    return binding.decode_prefix_raw(q, pk, pv, plen, rows, k, v, lens, batch, T, max_seqlen,
                                     desc or shared(), out, lse, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,expect", [
    (dict(q=None), INVALID), (dict(pk=None), INVALID), (dict(pv=A), INVALID),
    (dict(plen=None), INVALID), (dict(rows=0), INVALID), (dict(k=None), INVALID),
    (dict(v=A), INVALID), (dict(lens=None), INVALID), (dict(out=None), INVALID),
    (dict(batch=0), INVALID), (dict(T=0), INVALID), (dict(T=101), INVALID),
    (dict(max_seqlen=-1), INVALID),
    (dict(pk=A + 8), MISALIGNED), (dict(plen=A + 2), MISALIGNED), (dict(q=A + 8), MISALIGNED),
    (dict(ws=None), WORKSPACE), (dict(ws=A + 8), MISALIGNED),
    (dict(desc=shared(kv_shared=False), v=A), INVALID),          # no v_prefix
    (dict(desc=shared(kv_shared=False), v=A, pv=A + 2), MISALIGNED),
    (dict(desc=shared(head_dim=64)), UNSUPPORTED),
    (dict(desc=shared(n_q_heads=130)), UNSUPPORTED),
    (dict(desc=shared(window=64, cache_capacity=64), T=2), INVALID),
])
def test_prefix_refusals(kw, expect):
    assert prefix(**kw) == expect


def test_more_work_than_32_bits_count_is_refused():
    """2^20 tokens of one sequence, each over up to 2^20 positions."""
    d = shared(cache_capacity=1 << 20)
    assert prefix(d, T=1 << 20, max_seqlen=1 << 20) == UNSUPPORTED
    many = shared(n_q_heads=128, cache_capacity=64)  # batch * T * Hq above 2^31 - 1
    assert prefix(many, batch=1 << 20, T=17) == UNSUPPORTED


def test_workspace_queries_refuse():
    assert binding.sink_workspace_size(0, 1, 8, sliding(), 4) == 0
    assert binding.sink_workspace_size(1, 1, 8192, sliding(window=0), 4) == 0
    assert binding.sink_workspace_size(1, 1, 8192, sliding(), 1028) == 0
    assert binding.prefix_workspace_size(1, 1, 8, 0, shared()) == 0
    assert binding.prefix_workspace_size(1, 9, 8, 64, shared()) == 0
    assert binding.prefix_workspace_size(1, 1, 8, 64, shared(head_dim=64)) == 0


def slots(lens=A, new=A, batch=2, rows=4, C=8, S=2, start=A, seq=A, pos=A, slot=A):
    return binding.lib().gdattn_slot_map(lens, new, batch, rows, C, S, start, seq, pos, slot, None)


@pytest.mark.parametrize("kw,expect", [
    (dict(lens=None), INVALID), (dict(new=None), INVALID), (dict(start=None), INVALID),
    (dict(seq=None), INVALID), (dict(pos=None), INVALID), (dict(slot=None), INVALID),
    (dict(batch=0), INVALID), (dict(rows=-1), INVALID), (dict(C=0), INVALID),
    (dict(S=8), INVALID), (dict(S=-1), INVALID),
    (dict(lens=A + 2), MISALIGNED), (dict(slot=A + 1), MISALIGNED),
])
def test_slot_map_refusals(kw, expect):
    assert slots(**kw) == expect


def write(desc=None, k=A, v=A, stride=8 * 256, seq=A, slot=A, n=4, batch=2, kc=A, vc=A):
    return binding.cache_write_raw(k, v, stride, seq, slot, n, batch, desc or sliding(), kc, vc,
                                   None)


def write_fp8(desc=None, k=A, v=A, stride=8 * 256, seq=A, slot=A, n=4, batch=2, kc=A, vc=A, ks=A,
              vs=A):
    return binding.cache_write_fp8_raw(k, v, stride, seq, slot, n, batch, desc or sliding(), kc,
                                       vc, ks, vs, None)


@pytest.mark.parametrize("call", [write, write_fp8])
@pytest.mark.parametrize("kw,expect", [
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(seq=None), INVALID),
    (dict(slot=None), INVALID), (dict(kc=None), INVALID), (dict(vc=None), INVALID),
    (dict(n=-1), INVALID), (dict(batch=0), INVALID), (dict(stride=8 * 256 - 8), INVALID),
    (dict(stride=8 * 256 + 4), INVALID), (dict(desc=sliding(head_dim=64)), UNSUPPORTED),
    (dict(k=A + 8), MISALIGNED), (dict(vc=A + 8), MISALIGNED), (dict(seq=A + 2), MISALIGNED),
])
def test_write_refusals(call, kw, expect):
    assert call(**kw) == expect


def test_write_fp8_refuses_scales():
    assert write_fp8(ks=None) == INVALID
    assert write_fp8(vs=None) == INVALID
    assert write_fp8(ks=A + 2) == MISALIGNED
    assert write_fp8(sliding(cache_batch_stride=1028 * 8 * 256 + 8)) == MISALIGNED


def test_no_rows_is_no_launch():
    assert write(n=0) == binding.GDATTN_OK
    assert write_fp8(n=0) == binding.GDATTN_OK


@pytest.mark.parametrize("call", [write, write_fp8])
def test_no_rows_need_no_pointers(call):
    """What a tensor without elements points at is null."""
    none = dict(k=None, v=None, seq=None, slot=None)
    assert call(n=0, **none) == binding.GDATTN_OK
    assert call(n=0, kc=None, **none) == INVALID
    assert call(n=0, vc=None, **none) == INVALID
    assert call(n=1, k=A, v=None) == INVALID


# ------------------------------------------------- the binding's tensor checks
@pytest.fixture
def any_device(monkeypatch):
    """CPU tensors stand in for device ones: only the checks run."""
    monkeypatch.setattr(binding, "_on", lambda *a: None)


def test_row_tensors(any_device):
    d = sliding()
    fused = torch.zeros((5, 32, 256), dtype=torch.bfloat16)
    k, v = fused[:, 16:24], fused[:, 24:]
    cache = torch.zeros((2, 1028, 8, 256), dtype=torch.bfloat16)
    at = torch.zeros(5, dtype=torch.int32)
    assert binding._check_write(k, v, at, at, d, cache, cache, binding._BF16) == (5, 2, 32 * 256)
    assert binding._check_write(k[:1], v[:1], at[:1], at[:1], d, cache, cache,
                                binding._BF16) == (1, 2, 8 * 256)
    for bad, message in [
            (dict(k=k.float()), "k_rows: dtype"), (dict(k=k[:4]), "k_rows: shape"),
            (dict(k=fused[:, 15:23, :128]), "k_rows: shape"),
            (dict(k=k.transpose(1, 2).contiguous().transpose(1, 2)), "next to one another"),
            (dict(v=v.contiguous()), "v_rows: must have the row stride"),
            (dict(at=at.long()), "row_seq: dtype"),
            (dict(cache=cache[:, :1000].contiguous()), "k: storage holds"),
            (dict(cache=cache.float()), "k: dtype")]:
        a = dict(k=k, v=v, at=at, cache=cache)
        a.update(bad)
        with pytest.raises(ValueError, match=message):
            binding._check_write(a["k"], a["v"], a["at"], a["at"], d, a["cache"], a["cache"],
                                 binding._BF16)


def test_query_tensors(any_device):
    d = sliding()
    q = torch.zeros((2, 1, 16, 256), dtype=torch.bfloat16)
    cache = torch.zeros((1, 1028, 8, 256), dtype=torch.bfloat16)
    lens = torch.ones(1, dtype=torch.int32)
    lse = torch.zeros((2, 1, 16))
    binding._check_tokens(q, cache, cache, lens, q, lse, d)
    with pytest.raises(ValueError, match="q: heads and head_dim"):
        binding._check_tokens(q[:, :, :8].contiguous(), cache, cache, lens, q, lse, d)
    with pytest.raises(ValueError, match="out: .* the call reaches"):
        binding._check_tokens(q, cache, cache, lens, q[:1], lse, d)
    with pytest.raises(ValueError, match="workspace: dtype"):
        binding._check_workspace(lse, q, q.get_device())


# ------------------------------------------------------------ definitions
def test_definition_is_plain_attention_over_the_listed_keys():
    """One token over a window with pins, and one behind a prefix, against
    scaled_dot_product_attention in float64 over the gathered keys."""
    c = ref.make_case(3, 2, [30], 4, 2, 256, window=7, sinks=3)
    r = ref.reference(c)
    for t, p in enumerate((28, 29)):
        keys = [0, 1, 2] + list(range(p - 6, p + 1))
        k = c.k_rows[0][keys].double().repeat_interleave(2, 1).transpose(0, 1)
        v = c.v_rows[0][keys].double().repeat_interleave(2, 1).transpose(0, 1)
        q = c.q[t, 0].double()[:, None]
        o = torch.nn.functional.scaled_dot_product_attention(q, k, v, scale=c.scale)
        assert torch.allclose(r.out[t, 0], o[:, 0], rtol=0, atol=1e-12)
        lse = torch.logsumexp((q @ k.transpose(1, 2)).squeeze(1) * c.scale, -1)
        assert torch.allclose(r.lse[t, 0], lse, rtol=0, atol=1e-12)
    c = ref.make_case(4, 1, [5], 2, 2, 256, window=8, prefix=9)
    keys = torch.cat([c.pk[6:], c.k_rows[0]]).double().transpose(0, 1)  # 14 positions, last 8
    vals = torch.cat([c.pv[6:], c.v_rows[0]]).double().transpose(0, 1)
    o = torch.nn.functional.scaled_dot_product_attention(c.q[0, 0].double()[:, None], keys, vals,
                                                         scale=c.scale)
    assert torch.allclose(ref.reference(c).out[0, 0], o[:, 0], rtol=0, atol=1e-12)


def test_definition_caches_hold_what_the_rows_say():
    """Filling a ring with pins token by token leaves what make_case lays out."""
    c = ref.make_case(5, 1, [40], 2, 2, 256, window=9, sinks=4, capacity=13)
    cache = torch.full_like(c.k[0], ref.NAN)
    for L in range(1, 41):
        _, _, _, slot = ref.slot_map([L], [1], 1, 13, 4)
        cache[slot[0]] = c.k_rows[0][L - 1]
    assert torch.equal(cache, c.k[0])
    at_once = torch.full_like(c.k[0], ref.NAN)
    _, _, pos, slot = ref.slot_map([40], [40], 40, 13, 4)
    keep = slot >= 0
    at_once[slot[keep].long()] = c.k_rows[0][pos[keep].long()]
    assert torch.equal(at_once, cache)
    assert keep.sum() == 13


def test_definition_of_e4m3_is_torchs():
    g = torch.Generator().manual_seed(0)
    x = torch.randn((64, 256), generator=g).to(torch.bfloat16)
    value, scale = ref.e4m3_rows(x)
    y = x.float() / scale.float()[:, None]
    assert torch.equal(value, y.to(torch.float8_e4m3fn).double())
    assert math.isclose(float(scale[0]), float(x[0].double().abs().max()) / 448, rel_tol=1e-6)
