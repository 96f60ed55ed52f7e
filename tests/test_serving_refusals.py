"""Arguments of the continuous-batching wrappers that the C ABI cannot see, or would see
cut down to 32 bits, on the CPU."""
import pytest
import torch

from decode_attention_09_b200 import binding

H, HKV, D, C, B = 16, 8, 256, 8, 2


@pytest.fixture(autouse=True)
def checks_only(monkeypatch):
    """CPU tensors stand in for device ones, and no call may get past the checks."""
    monkeypatch.setattr(binding, "_on", lambda *a: None)

    def call(fn, what, *a):
        raise AssertionError(f"{what} was called")

    monkeypatch.setattr(binding, "_call", call)


def z(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


def desc():
    return binding.make_desc(H, HKV, D, 4, 0.0, 1.0, False, C)


ws = z(512, dtype=torch.uint8)
lens = z(B, dtype=torch.int32)


def prefix(k_prefix, max_seqlen=8):
    binding.decode_prefix(z(1, B, H, D), k_prefix, k_prefix, z(1, dtype=torch.int32),
                          z(B, C, HKV, D), z(B, C, HKV, D), lens, desc(), max_seqlen,
                          workspace=ws)


@pytest.mark.parametrize("shape", [(1, 5, HKV, D), (5, HKV * D), (5, D, HKV), (HKV, 5, D),
                                   (5 * HKV, 1, D)])
def test_a_prefix_of_another_shape(shape):
    """Read as rows, it would be a shorter prefix or other heads."""
    with pytest.raises(ValueError, match="k_prefix: shape"):
        prefix(z(*shape))


@pytest.mark.parametrize("wide", [2 ** 31, 2 ** 32 + 8, 2 ** 40])
def test_counts_beyond_32_bits(wide):
    with pytest.raises(ValueError, match="at most"):
        prefix(z(5, HKV, D), wide)
    for max_seqlen, n_sink in ((wide, 2), (8, wide)):
        with pytest.raises(ValueError, match="at most"):
            binding.decode_sink(z(1, B, H, D), z(B, C, HKV, D), z(B, C, HKV, D), lens, desc(),
                                max_seqlen, n_sink, workspace=ws)
    for n_rows, capacity, n_sink in ((wide, 8, 0), (4, wide, 0), (4, 8, wide)):
        with pytest.raises(ValueError, match="at most"):
            binding.slot_map(lens, lens, n_rows, capacity, n_sink)


def test_more_rows_than_32_bits_count():
    many = torch.zeros(1, dtype=torch.int32).expand(2 ** 31)
    rows = z(1, HKV, D).expand(2 ** 31, HKV, D)
    cache = z(B, C, HKV, D)
    for dtypes in (binding._BF16, binding._CODES):
        with pytest.raises(ValueError, match="at most"):
            binding._check_write(rows, rows, many, many, desc(), cache, cache, dtypes)


# --------------------------------------------------------- caches that are views
def by_sink(k, v, d):
    binding._check_tokens(z(1, B, H, D), k, v, lens, None, None, d)


def by_write(k, v, d):
    binding._check_write(z(3, HKV, D), z(3, HKV, D), z(3, dtype=torch.int32),
                         z(3, dtype=torch.int32), d, k, v, binding._BF16)


@pytest.mark.parametrize("check", [by_sink, by_write])
def test_views_of_caches_go_by_the_descriptor(check):
    dense = z(B, C, HKV, D)
    larger = z(B, C + 3, HKV, D)
    part = larger[:, :C]
    stride = (C + 3) * HKV * D
    d = binding.make_desc(H, HKV, D, 4, 0.0, 1.0, False, C, stride)
    check(dense, dense, desc())
    check(part, part, d)
    check(larger[1:, :C], larger[1:, :C], d) if check is by_write else None
    for bad, dd in ((part, desc()),                                # the stride not given
                    (z(B, HKV, C, D).transpose(1, 2), desc()),     # heads before slots
                    (z(B, C, D, HKV).transpose(2, 3), desc()),
                    (larger[:, ::2][:, :4].expand(B, 4, HKV, D), d)):
        for k, v in ((bad, bad), (dense if dd is not d else part, bad)):
            with pytest.raises(ValueError, match="strides|storage holds"):
                check(k, v, dd)
