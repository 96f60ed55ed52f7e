"""ctypes binding of libgdattn's C ABI (include/gdattn.h).

Argument marshalling only: every step of decode attention runs in the CUDA
kernels of libgdattn.so.  The tensor wrappers check what the C ABI cannot see
(dtype, contiguity, that each tensor reaches as far as the call reads or
writes, and its device) and raise ValueError before anything is enqueued; the
``*_raw`` functions pass addresses through unchecked.  Torch supplies device memory and streams.  There is no
fallback: if the library has not been built, loading it raises.
"""
from __future__ import annotations

import ctypes
import os
from typing import NamedTuple, Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libgdattn.so")

GDATTN_OK = 0
GDATTN_ERR_INVALID_ARG = 1
GDATTN_ERR_UNSUPPORTED = 2
GDATTN_ERR_MISALIGNED = 3
GDATTN_ERR_WORKSPACE = 4
GDATTN_ERR_CUDA = 5
GDATTN_ERR_DEVICE_TIMEOUT = 6
GDATTN_ERR_DEVICE_SEQLEN = 7


class LayerDesc(ctypes.Structure):
    """Mirror of gdattn_layer_desc."""

    _fields_ = [
        ("n_q_heads", ctypes.c_int32),
        ("n_kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("window", ctypes.c_int32),
        ("softcap", ctypes.c_float),
        ("scale", ctypes.c_float),
        ("kv_shared", ctypes.c_int32),
        ("cache_capacity", ctypes.c_int32),
        ("cache_batch_stride", ctypes.c_int64),
        ("split_ctas", ctypes.c_int32),
        ("flags", ctypes.c_int32),
    ]


class GdattnError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} ({status})")


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded libgdattn.so.  Raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"libgdattn.so not found at {LIB_PATH}; build it with "
                "`python decode_attention_09_b200/build.py` (nvcc, sm_100a)")
        L = ctypes.CDLL(LIB_PATH)
        vp, sz, i32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int32
        descp = ctypes.POINTER(LayerDesc)
        L.gdattn_version.restype = i32
        L.gdattn_status_string.argtypes = [ctypes.c_int]
        L.gdattn_status_string.restype = ctypes.c_char_p
        L.gdattn_workspace_size.argtypes = [i32, i32, descp]
        L.gdattn_workspace_size.restype = sz
        L.gdattn_plan_splits.argtypes = [i32, i32, descp]
        L.gdattn_plan_splits.restype = i32
        L.gdattn_plan_launches.argtypes = [i32, i32, descp]
        L.gdattn_plan_launches.restype = i32
        L.gdattn_workspace_init.argtypes = [vp, sz, vp]
        L.gdattn_workspace_init.restype = ctypes.c_int
        L.gdattn_decode.argtypes = [vp, vp, vp, vp, i32, i32, descp, vp, vp, vp, sz, vp]
        L.gdattn_decode.restype = ctypes.c_int
        if hasattr(L, "gdattn_decode_append"):  # libraries built before it was added lack it
            L.gdattn_decode_append.argtypes = [vp, vp, vp, vp, vp, vp, i32, i32, descp, vp, vp,
                                               vp, sz, vp]
            L.gdattn_decode_append.restype = ctypes.c_int
        if hasattr(L, "gdattn_decode_multi"):
            L.gdattn_multi_workspace_size.argtypes = [i32, i32, i32, descp]
            L.gdattn_multi_workspace_size.restype = sz
            L.gdattn_decode_multi.argtypes = [vp, vp, vp, vp, i32, i32, i32, descp, vp, vp, vp,
                                              sz, vp]
            L.gdattn_decode_multi.restype = ctypes.c_int
        if hasattr(L, "gdattn_decode_fp8"):
            L.gdattn_decode_fp8.argtypes = [vp, vp, vp, vp, vp, vp, i32, i32, descp, vp, vp, vp,
                                            sz, vp]
            L.gdattn_decode_fp8.restype = ctypes.c_int
        L.gdattn_decode_noalloc.argtypes = [vp, vp, vp, vp, i32, i32, descp, vp, vp, vp]
        L.gdattn_decode_noalloc.restype = ctypes.c_int
        L.gdattn_combine.argtypes = [vp, vp, i32, i32, i32, i32, vp, vp, vp]
        L.gdattn_combine.restype = ctypes.c_int
        if hasattr(L, "gdattn_decode_sink"):
            L.gdattn_sink_workspace_size.argtypes = [i32, i32, i32, descp, i32]
            L.gdattn_sink_workspace_size.restype = sz
            L.gdattn_decode_sink.argtypes = [vp, vp, vp, vp, i32, i32, i32, descp, i32, vp, vp,
                                             vp, sz, vp]
            L.gdattn_decode_sink.restype = ctypes.c_int
            L.gdattn_prefix_workspace_size.argtypes = [i32, i32, i32, i32, descp]
            L.gdattn_prefix_workspace_size.restype = sz
            L.gdattn_decode_prefix.argtypes = [vp, vp, vp, vp, i32, vp, vp, vp, i32, i32, i32,
                                               descp, vp, vp, vp, sz, vp]
            L.gdattn_decode_prefix.restype = ctypes.c_int
            L.gdattn_slot_map.argtypes = [vp, vp, i32, i32, i32, i32, vp, vp, vp, vp, vp]
            L.gdattn_slot_map.restype = ctypes.c_int
            i64 = ctypes.c_int64
            L.gdattn_cache_write.argtypes = [vp, vp, i64, vp, vp, i32, i32, descp, vp, vp, vp]
            L.gdattn_cache_write.restype = ctypes.c_int
            L.gdattn_cache_write_fp8.argtypes = [vp, vp, i64, vp, vp, i32, i32, descp, vp, vp,
                                                 vp, vp, vp]
            L.gdattn_cache_write_fp8.restype = ctypes.c_int
        L.gdattn_check_device_status.argtypes = [vp, vp]
        L.gdattn_check_device_status.restype = ctypes.c_int
        L.gdattn_read_probe.argtypes = [vp, sz, i32, vp, vp]
        L.gdattn_read_probe.restype = ctypes.c_int
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().gdattn_status_string(int(status)).decode()


def version() -> int:
    return int(lib().gdattn_version())


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream_handle(stream) -> Optional[int]:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _empty(shape, dtype, device, stream) -> torch.Tensor:
    """A tensor for a call on ``stream`` (None: the current one).  The caching allocator
    hands memory out again in the order of the stream it was allocated on, so what a
    wrapper allocates belongs to the stream its kernels run on."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if not hasattr(stream, "cuda_stream"):
        handle = int(stream)  # 0 and 1 are the legacy default stream
        stream = (torch.cuda.default_stream(device) if handle in (0, 1) else
                  torch.cuda.ExternalStream(handle, device=device))
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _result(shape, dtype, device, stream) -> torch.Tensor:
    """An output of a call on ``stream``, which the current stream may read after the
    caller has ordered the two: its memory is not used again before that read."""
    t = _empty(shape, dtype, device, stream)
    if stream is not None:
        t.record_stream(torch.cuda.current_stream(device))
    return t


def _dense(t: torch.Tensor, name: str, dtypes, numel: int, device) -> None:
    """A dense tensor argument: one of ``dtypes``, contiguous, holding at least
    ``numel`` elements (what the call reads or writes through its pointer), on
    the CUDA device of the call.  The C ABI sees only the address, so a tensor
    that is too small would be read or written past its end on the device."""
    if t.dtype not in dtypes:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {' or '.join(map(str, dtypes))}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    if t.numel() < numel:
        raise ValueError(f"{name}: {t.numel()} elements, the call reaches {numel}")
    _on(t, name, device)


def _extent(t: torch.Tensor, name: str, dtypes, numel: int, device) -> None:
    """A strided cache argument: one of ``dtypes``, with at least ``numel``
    elements of storage from its first element on (the rows the call may reach
    through ``cache_batch_stride``), on the CUDA device of the call."""
    if t.dtype not in dtypes:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {' or '.join(map(str, dtypes))}")
    have = t.untyped_storage().nbytes() // t.element_size() - t.storage_offset()
    if have < numel:
        raise ValueError(f"{name}: storage holds {have} elements, the call reaches {numel}")
    _on(t, name, device)


def _on(t: torch.Tensor, name: str, device) -> None:
    if not t.is_cuda:
        raise ValueError(f"{name}: must be a CUDA tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name}: on {t.device}, the call runs on {device}")


def _cache_elems(batch: int, desc: "LayerDesc") -> int:
    """Elements of a cache that sequences 0..batch-1 span: sequence b starts at
    b * cache_batch_stride (0 = C * Hkv * D) and holds C * Hkv * D."""
    rows = int(desc.cache_capacity) * int(desc.n_kv_heads) * int(desc.head_dim)
    stride = int(desc.cache_batch_stride) or rows
    return (batch - 1) * stride + rows if batch > 0 else 0


_BF16 = (torch.bfloat16,)
_F32 = (torch.float32,)
_I32 = (torch.int32,)
_CODES = (torch.uint8, torch.float8_e4m3fn)


def _check_layer(q, k, v, seqlens, out, lse, desc, n_seq: int, n_cache: int) -> None:
    """The arguments every decode entry point shares: q and out are bf16
    [n_seq, Hq, D] (possibly with a leading token axis folded into n_seq), lse fp32
    [n_seq, Hq] or None, seqlens int32 [n_cache], and bf16 K / V caches spanning
    n_cache sequences."""
    dev = q.device
    hq, d = int(desc.n_q_heads), int(desc.head_dim)
    _dense(q, "q", _BF16, n_seq * hq * d, dev)
    _extent(k, "k", _BF16, _cache_elems(n_cache, desc), dev)
    if v is not None:
        _extent(v, "v", _BF16, _cache_elems(n_cache, desc), dev)
    _dense(seqlens, "seqlens", _I32, n_cache, dev)
    _dense(out, "out", _BF16, n_seq * hq * d, dev)
    if lse is not None:
        _dense(lse, "lse", _F32, n_seq * hq, dev)


def _check_new_rows(k_new, v_new, desc, batch: int, device) -> None:
    """gdattn_decode_append's rows: bf16 [batch, Hkv, D] (v_new None when K = V)."""
    rows = batch * int(desc.n_kv_heads) * int(desc.head_dim)
    _dense(k_new, "k_new", _BF16, rows, device)
    if v_new is not None:
        _dense(v_new, "v_new", _BF16, rows, device)


def _check_fp8(q, k_codes, v_codes, k_scale, v_scale, seqlens, out, lse, desc,
               batch: int) -> None:
    """gdattn_decode_fp8's arguments: e4m3 code caches (uint8 or float8_e4m3fn)
    spanning ``batch`` sequences, fp32 scales [batch, Hkv, C], the rest as for
    gdattn_decode."""
    dev = q.device
    hq, d = int(desc.n_q_heads), int(desc.head_dim)
    _dense(q, "q", _BF16, batch * hq * d, dev)
    n_scales = batch * int(desc.n_kv_heads) * int(desc.cache_capacity)
    _extent(k_codes, "k_codes", _CODES, _cache_elems(batch, desc), dev)
    _dense(k_scale, "k_scale", _F32, n_scales, dev)
    if v_codes is not None:  # None is the C ABI's to refuse (no fp8 path for K = V)
        _extent(v_codes, "v_codes", _CODES, _cache_elems(batch, desc), dev)
    if v_scale is not None:
        _dense(v_scale, "v_scale", _F32, n_scales, dev)
    _dense(seqlens, "seqlens", _I32, batch, dev)
    _dense(out, "out", _BF16, batch * hq * d, dev)
    if lse is not None:
        _dense(lse, "lse", _F32, batch * hq, dev)


def _check_combine(o_partial, lse_partial, out, lse) -> None:
    """gdattn_combine's arguments: fp32 partials [B, Hq, S, D] and [B, Hq, S],
    bf16 out [B, Hq, D], fp32 lse [B, Hq]."""
    B, Hq, S, D = o_partial.shape
    dev = o_partial.device
    _dense(o_partial, "o_partial", _F32, B * Hq * S * D, dev)
    _dense(lse_partial, "lse_partial", _F32, B * Hq * S, dev)
    _dense(out, "out", _BF16, B * Hq * D, dev)
    if lse is not None:
        _dense(lse, "lse", _F32, B * Hq, dev)


GDATTN_FLAG_EVEN_UNITS = 1
GDATTN_FLAG_TEST_WITHHOLD_KV = 2


def make_desc(n_q_heads: int, n_kv_heads: int, head_dim: int, window: int, softcap: float,
              scale: float, kv_shared: bool, cache_capacity: int, cache_batch_stride: int = 0,
              split_ctas: int = 0, flags: int = 0) -> LayerDesc:
    return LayerDesc(int(n_q_heads), int(n_kv_heads), int(head_dim), int(window),
                     float(softcap), float(scale), 1 if kv_shared else 0, int(cache_capacity),
                     int(cache_batch_stride), int(split_ctas), int(flags))


def desc_from_spec(spec, split_ctas: int = 0, capacity: Optional[int] = None,
                   flags: int = 0) -> LayerDesc:
    """Descriptor for a ``workloads.LayerSpec``."""
    return make_desc(spec.n_q_heads, spec.n_kv_heads, spec.head_dim, spec.window, spec.softcap,
                     spec.scale, spec.kv_shared,
                     capacity if capacity is not None else spec.capacity, 0, split_ctas, flags)


def workspace_size(batch: int, max_seqlen: int, desc: LayerDesc) -> int:
    return int(lib().gdattn_workspace_size(int(batch), int(max_seqlen), ctypes.byref(desc)))


def plan_splits(batch: int, max_seqlen: int, desc: LayerDesc) -> int:
    """CTAs the planner splits the KV range across (0 on invalid arguments)."""
    return int(lib().gdattn_plan_splits(int(batch), int(max_seqlen), ctypes.byref(desc)))


def launches_per_call(batch: int, max_seqlen: int, desc: LayerDesc) -> int:
    """Kernel launches one gdattn_decode call makes (1, or 2 with a separate combine)."""
    return int(lib().gdattn_plan_launches(int(batch), int(max_seqlen), ctypes.byref(desc)))


def workspace_init(workspace: torch.Tensor, stream=None) -> None:
    st = lib().gdattn_workspace_init(_ptr(workspace), workspace.numel() * workspace.element_size(),
                                     _stream_handle(stream))
    if st != GDATTN_OK:
        raise GdattnError(st, "gdattn_workspace_init")


def alloc_workspace(batch: int, max_seqlen: int, desc: LayerDesc, device="cuda",
                    stream=None) -> torch.Tensor:
    n = workspace_size(batch, max_seqlen, desc)
    if n == 0:
        raise GdattnError(GDATTN_ERR_INVALID_ARG, "gdattn_workspace_size")
    ws = _empty((n,), torch.uint8, device, stream)
    workspace_init(ws, stream)
    return ws


def decode_raw(q, k, v, seqlens, batch, max_seqlen, desc, out, lse, workspace, workspace_bytes,
               stream) -> int:
    """gdattn_decode on raw addresses (ints); returns the status code."""
    return int(lib().gdattn_decode(q, k, v, seqlens, int(batch), int(max_seqlen),
                                   ctypes.byref(desc), out, lse, workspace,
                                   int(workspace_bytes), stream))


def decode(q: torch.Tensor, k: torch.Tensor, v: Optional[torch.Tensor], seqlens: torch.Tensor,
           desc: LayerDesc, max_seqlen: int, out: Optional[torch.Tensor] = None,
           lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
           stream=None, want_lse: bool = True):
    """One decode-attention layer through gdattn_decode.  Returns (out, lse)."""
    B, Hq, D = q.shape
    if out is None:
        out = _result((B, Hq, D), torch.bfloat16, q.device, stream)
    if lse is None and want_lse:
        lse = _result((B, Hq), torch.float32, q.device, stream)
    _check_layer(q, k, v, seqlens, out, lse, desc, B, B)
    if workspace is None:
        workspace = alloc_workspace(B, max_seqlen, desc, q.device, stream)
    _on(workspace, "workspace", q.device)
    st = decode_raw(_ptr(q), _ptr(k), _ptr(v), _ptr(seqlens), B, max_seqlen, desc, _ptr(out),
                    _ptr(lse), _ptr(workspace), workspace.numel(), _stream_handle(stream))
    if st != GDATTN_OK:
        raise GdattnError(st, "gdattn_decode")
    return out, lse


def decode_append(q: torch.Tensor, k_new: torch.Tensor, v_new: Optional[torch.Tensor],
                  k: torch.Tensor, v: Optional[torch.Tensor], seqlens: torch.Tensor,
                  desc: LayerDesc, max_seqlen: int, out: Optional[torch.Tensor] = None,
                  lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                  stream=None):
    """gdattn_decode_append: write k_new / v_new ([B, Hkv, D]) into slot
    (L - 1) mod C of the caches, then decode.  Returns (out, lse)."""
    B, Hq, D = q.shape
    if out is None:
        out = _result((B, Hq, D), torch.bfloat16, q.device, stream)
    if lse is None:
        lse = _result((B, Hq), torch.float32, q.device, stream)
    _check_layer(q, k, v, seqlens, out, lse, desc, B, B)
    _check_new_rows(k_new, v_new, desc, B, q.device)
    if workspace is None:
        workspace = alloc_workspace(B, max_seqlen, desc, q.device, stream)
    _on(workspace, "workspace", q.device)
    st = int(lib().gdattn_decode_append(_ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k), _ptr(v),
                                        _ptr(seqlens), B, int(max_seqlen), ctypes.byref(desc),
                                        _ptr(out), _ptr(lse), _ptr(workspace),
                                        workspace.numel(), _stream_handle(stream)))
    if st != GDATTN_OK:
        raise GdattnError(st, "gdattn_decode_append")
    return out, lse


def decode_fp8_raw(q, k_codes, v_codes, k_scale, v_scale, seqlens, batch, max_seqlen, desc, out,
                   lse, workspace, workspace_bytes, stream) -> int:
    """gdattn_decode_fp8 on raw addresses (ints); returns the status code."""
    return int(lib().gdattn_decode_fp8(q, k_codes, v_codes, k_scale, v_scale, seqlens,
                                       int(batch), int(max_seqlen), ctypes.byref(desc), out, lse,
                                       workspace, int(workspace_bytes), stream))


def decode_fp8(q: torch.Tensor, k_codes: torch.Tensor, v_codes: torch.Tensor,
               k_scale: torch.Tensor, v_scale: torch.Tensor, seqlens: torch.Tensor,
               desc: LayerDesc, max_seqlen: int, out: Optional[torch.Tensor] = None,
               lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
               stream=None):
    """One layer over an fp8 e4m3 cache through gdattn_decode_fp8.  Returns (out, lse).

    k_codes / v_codes: uint8 (or float8_e4m3fn) [B, C, Hkv, D]; k_scale / v_scale:
    float32 [B, Hkv, C], the scale of each cache row.
    """
    B, Hq, D = q.shape
    if out is None:
        out = _result((B, Hq, D), torch.bfloat16, q.device, stream)
    if lse is None:
        lse = _result((B, Hq), torch.float32, q.device, stream)
    _check_fp8(q, k_codes, v_codes, k_scale, v_scale, seqlens, out, lse, desc, B)
    if workspace is None:
        workspace = alloc_workspace(B, max_seqlen, desc, q.device, stream)
    _on(workspace, "workspace", q.device)
    st = decode_fp8_raw(_ptr(q), _ptr(k_codes), _ptr(v_codes), _ptr(k_scale), _ptr(v_scale),
                        _ptr(seqlens), B, max_seqlen, desc, _ptr(out), _ptr(lse),
                        _ptr(workspace), workspace.numel(), _stream_handle(stream))
    if st != GDATTN_OK:
        raise GdattnError(st, "gdattn_decode_fp8")
    return out, lse


def multi_workspace_size(batch: int, n_tokens: int, max_seqlen: int, desc: LayerDesc) -> int:
    return int(lib().gdattn_multi_workspace_size(int(batch), int(n_tokens), int(max_seqlen),
                                                 ctypes.byref(desc)))


def decode_multi_raw(q, k, v, seqlens, batch, n_tokens, max_seqlen, desc, out, lse, workspace,
                     workspace_bytes, stream) -> int:
    """gdattn_decode_multi on raw addresses (ints); returns the status code."""
    return int(lib().gdattn_decode_multi(q, k, v, seqlens, int(batch), int(n_tokens),
                                         int(max_seqlen), ctypes.byref(desc), out, lse, workspace,
                                         int(workspace_bytes), stream))


def decode_multi(q: torch.Tensor, k: torch.Tensor, v: Optional[torch.Tensor],
                 seqlens: torch.Tensor, desc: LayerDesc, max_seqlen: int,
                 out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                 workspace: Optional[torch.Tensor] = None, stream=None):
    """Multi-token step through gdattn_decode_multi: a verify step, or a prompt chunk
    (flash prefill).  q bf16 [T, B, Hq, D]: token t of sequence b at position
    L_b - T + t, attending causally.  Returns (out, lse), token-major."""
    T, B, Hq, D = q.shape
    if out is None:
        out = _result((T, B, Hq, D), torch.bfloat16, q.device, stream)
    if lse is None:
        lse = _result((T, B, Hq), torch.float32, q.device, stream)
    _check_layer(q, k, v, seqlens, out, lse, desc, T * B, B)
    if workspace is None:
        n = multi_workspace_size(B, T, max_seqlen, desc)
        if n == 0:
            raise GdattnError(GDATTN_ERR_INVALID_ARG, "gdattn_multi_workspace_size")
        workspace = _empty((n,), torch.uint8, q.device, stream)
        workspace_init(workspace, stream)
    _on(workspace, "workspace", q.device)
    st = decode_multi_raw(_ptr(q), _ptr(k), _ptr(v), _ptr(seqlens), B, T, max_seqlen, desc,
                          _ptr(out), _ptr(lse), _ptr(workspace), workspace.numel(),
                          _stream_handle(stream))
    if st != GDATTN_OK:
        raise GdattnError(st, "gdattn_decode_multi")
    return out, lse


NOALLOC_SCRATCH_BYTES = 8 << 20  # GDATTN_NOALLOC_SCRATCH_BYTES


def decode_noalloc_raw(q, k, v, seqlens, batch, max_seqlen, desc, out, lse, stream) -> int:
    """gdattn_decode_noalloc on raw addresses (ints); returns the status code."""
    return int(lib().gdattn_decode_noalloc(q, k, v, seqlens, int(batch), int(max_seqlen),
                                           ctypes.byref(desc), out, lse, stream))


def decode_noalloc(q: torch.Tensor, k: torch.Tensor, v: Optional[torch.Tensor],
                   seqlens: torch.Tensor, desc: LayerDesc, max_seqlen: int,
                   out: torch.Tensor, lse: Optional[torch.Tensor] = None, stream=None):
    """One layer through gdattn_decode_noalloc (scratch inside the library).

    `out` (and `lse`, if wanted) are caller-owned; nothing is allocated here.
    Calls that can overlap in time on one device race on the shared scratch.
    """
    B = q.shape[0]
    _check_layer(q, k, v, seqlens, out, lse, desc, B, B)
    st = decode_noalloc_raw(_ptr(q), _ptr(k), _ptr(v), _ptr(seqlens), B, max_seqlen, desc,
                            _ptr(out), _ptr(lse), _stream_handle(stream))
    if st != GDATTN_OK:
        raise GdattnError(st, "gdattn_decode_noalloc")
    return out, lse


def combine(o_partial: torch.Tensor, lse_partial: torch.Tensor, out: Optional[torch.Tensor] = None,
            lse: Optional[torch.Tensor] = None, stream=None):
    """gdattn_combine: o_partial fp32 [B,Hq,S,D], lse_partial fp32 [B,Hq,S]."""
    B, Hq, S, D = o_partial.shape
    if out is None:
        out = _result((B, Hq, D), torch.bfloat16, o_partial.device, stream)
    if lse is None:
        lse = _result((B, Hq), torch.float32, o_partial.device, stream)
    _check_combine(o_partial, lse_partial, out, lse)
    st = lib().gdattn_combine(_ptr(o_partial), _ptr(lse_partial), B, Hq, S, D, _ptr(out), _ptr(lse),
                              _stream_handle(stream))
    if st != GDATTN_OK:
        raise GdattnError(st, "gdattn_combine")
    return out, lse


def check_device_status(workspace: Optional[torch.Tensor], stream=None) -> int:
    """Read and clear a workspace's status word (None: the no-alloc scratch)."""
    return int(lib().gdattn_check_device_status(_ptr(workspace), _stream_handle(stream)))


def read_probe(src: torch.Tensor, mode: int, sink: torch.Tensor, stream=None) -> None:
    """gdattn_read_probe over the whole of ``src`` (a contiguous device tensor);
    ``sink``: int32 tensor of 2 elements on the same device."""
    _on(sink, "sink", src.device)
    if not src.is_contiguous() or sink.numel() < 2 or sink.dtype != torch.int32:
        raise ValueError("read_probe: contiguous src and an int32 sink of 2 elements")
    st = lib().gdattn_read_probe(_ptr(src), src.numel() * src.element_size(), int(mode),
                                 _ptr(sink), _stream_handle(stream))
    if st != GDATTN_OK:
        raise GdattnError(st, "gdattn_read_probe")


# ------------------------------------------------------ continuous batching
# These wrappers are called once per layer and step, so what they cost the host counts:
# an argument is first tested as a whole (``_fits``), and only one that fails goes
# through the checks that name what is wrong with it.
def _call(fn, what: str, index: int, stream, *args) -> None:
    """fn(*args, stream) with device ``index`` current: the library launches on the
    current device, so a call follows its tensors.  stream None: the device's current one."""
    if index != torch._C._cuda_getDevice():
        with torch.cuda.device(index):
            return _call(fn, what, index, stream, *args)
    if stream is None:
        stream = torch._C._cuda_getCurrentRawStream(index)
    elif hasattr(stream, "cuda_stream"):
        stream = stream.cuda_stream
    st = fn(*args, stream)
    if st != GDATTN_OK:
        raise GdattnError(st, what)


def _fits(t: torch.Tensor, dtype, numel: int, index: int) -> bool:
    return (t.dtype is dtype and t.get_device() == index and t.is_contiguous()
            and t.numel() >= numel)


def _need(t: torch.Tensor, name: str, dtype, numel: int, like: torch.Tensor, index: int) -> None:
    """A dense argument on the device of ``like``, which is device ``index``."""
    if not _fits(t, dtype, numel, index):
        _dense(t, name, (dtype,), numel, like.device)


def _need_cache(t: torch.Tensor, name: str, dtypes, numel: int, like: torch.Tensor,
                index: int, desc: LayerDesc) -> None:
    if not _fits(t, dtypes[0], numel, index):  # dense caches; strided ones reach further
        _extent(t, name, dtypes, numel, like.device)
        if t.dim() == 4 and not t.is_contiguous():
            _cache_strides(t, name, desc)


def _cache_strides(t: torch.Tensor, name: str, desc: LayerDesc) -> None:
    """A cache [B, C, Hkv, D] that is not contiguous: the library goes by the descriptor,
    so any other order or distance of the rows would be read as something else."""
    H, D = int(desc.n_kv_heads), int(desc.head_dim)
    batch = int(desc.cache_batch_stride) or int(desc.cache_capacity) * H * D
    for n, have, want in zip(t.shape, t.stride(), (batch, H * D, D, 1)):
        if n > 1 and have != want:
            raise ValueError(f"{name}: strides {tuple(t.stride())}, the descriptor says "
                             f"{(batch, H * D, D, 1)}")


_bf16, _f32, _i32, _u8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


def _check_tokens(q, k, v, seqlens, out, lse, desc, stream=None):
    """The arguments both continuous-batching attention calls share: q and out bf16
    [T, B, Hq, D], lse fp32 [T, B, Hq] or None, caches spanning B sequences.  Returns
    (T, B, device index, out, lse), with out and lse allocated where they are None, for
    a call on ``stream``."""
    T, B, Hq, D = q.shape
    index = q.get_device()
    if Hq != desc.n_q_heads or D != desc.head_dim:
        raise ValueError(f"q: heads and head_dim {(Hq, D)}, the descriptor has "
                         f"{(int(desc.n_q_heads), int(desc.head_dim))}")
    if index < 0 or q.dtype is not _bf16 or not q.is_contiguous():
        _dense(q, "q", _BF16, q.numel(), q.device)
    if out is None:
        out = (torch.empty_like(q) if stream is None else
               _result(q.shape, _bf16, q.device, stream))
    else:
        _need(out, "out", _bf16, T * B * Hq * D, q, index)
    if lse is None:
        lse = (q.new_empty((T, B, Hq), dtype=_f32) if stream is None else
               _result((T, B, Hq), _f32, q.device, stream))
    else:
        _need(lse, "lse", _f32, T * B * Hq, q, index)
    n = _cache_elems(B, desc)
    _need_cache(k, "k", _BF16, n, q, index, desc)
    if v is not None:
        _need_cache(v, "v", _BF16, n, q, index, desc)
    _need(seqlens, "seqlens", _i32, B, q, index)
    return T, B, index, out, lse


_MOST = 2 ** 31 - 1  # of the ABI's counts: ctypes would cut higher bits off silently


def _too_many(name: str, n: int) -> None:
    raise ValueError(f"{name}: {n}, at most {_MOST}")


def _check_workspace(workspace, like, index: int) -> None:
    _need(workspace, "workspace", _u8, 0, like, index)


def sink_workspace_size(batch: int, n_tokens: int, max_seqlen: int, desc: LayerDesc,
                        n_sink: int) -> int:
    return int(lib().gdattn_sink_workspace_size(int(batch), int(n_tokens), int(max_seqlen),
                                                ctypes.byref(desc), int(n_sink)))


def alloc_sink_workspace(batch: int, n_tokens: int, max_seqlen: int, desc: LayerDesc,
                         n_sink: int, device="cuda", stream=None) -> torch.Tensor:
    """A zeroed workspace for ``decode_sink`` calls of these sizes."""
    return _zeroed_workspace(
        lambda: sink_workspace_size(batch, n_tokens, max_seqlen, desc, n_sink),
        "gdattn_sink_workspace_size", device, stream)


def prefix_workspace_size(batch: int, n_tokens: int, max_seqlen: int, prefix_rows: int,
                          desc: LayerDesc) -> int:
    return int(lib().gdattn_prefix_workspace_size(int(batch), int(n_tokens), int(max_seqlen),
                                                  int(prefix_rows), ctypes.byref(desc)))


def alloc_prefix_workspace(batch: int, n_tokens: int, max_seqlen: int, prefix_rows: int,
                           desc: LayerDesc, device="cuda", stream=None) -> torch.Tensor:
    """A zeroed workspace for ``decode_prefix`` calls of these sizes."""
    return _zeroed_workspace(
        lambda: prefix_workspace_size(batch, n_tokens, max_seqlen, prefix_rows, desc),
        "gdattn_prefix_workspace_size", device, stream)


def _zeroed_workspace(size, what: str, device, stream) -> torch.Tensor:
    device = torch.device(device)
    with torch.cuda.device(device):
        n = size()
        if n == 0:
            raise GdattnError(GDATTN_ERR_INVALID_ARG, what)
        ws = _empty((n,), torch.uint8, device, stream)
        workspace_init(ws, stream)
    return ws


def decode_sink_raw(q, k, v, seqlens, batch, n_tokens, max_seqlen, desc, n_sink, out, lse,
                    workspace, workspace_bytes, stream) -> int:
    """gdattn_decode_sink on raw addresses (ints); returns the status code."""
    return lib().gdattn_decode_sink(q, k, v, seqlens, int(batch), int(n_tokens), int(max_seqlen),
                                    ctypes.byref(desc), int(n_sink), out, lse, workspace,
                                    int(workspace_bytes), stream)


def decode_sink(q: torch.Tensor, k: torch.Tensor, v: Optional[torch.Tensor],
                seqlens: torch.Tensor, desc: LayerDesc, max_seqlen: int, n_sink: int,
                out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                workspace: Optional[torch.Tensor] = None, stream=None):
    """Sliding-window attention with n_sink pinned first tokens through
    gdattn_decode_sink.  q bf16 [T, B, Hq, D]: token t of sequence b at position
    L_b - T + t.  Returns (out, lse), token-major."""
    T, B, index, out, lse = _check_tokens(q, k, v, seqlens, out, lse, desc, stream)
    if max_seqlen > _MOST or n_sink > _MOST:
        _too_many("max_seqlen or n_sink", max(max_seqlen, n_sink))
    if workspace is None:
        workspace = alloc_sink_workspace(B, T, max_seqlen, desc, n_sink, q.device, stream)
    _check_workspace(workspace, q, index)
    _call(lib().gdattn_decode_sink, "gdattn_decode_sink", index, stream, q.data_ptr(),
          k.data_ptr(), _ptr(v), seqlens.data_ptr(), B, T, max_seqlen, ctypes.byref(desc), n_sink,
          out.data_ptr(), lse.data_ptr(), workspace.data_ptr(), workspace.numel())
    return out, lse


def decode_prefix_raw(q, k_prefix, v_prefix, prefix_len, prefix_rows, k, v, seqlens, batch,
                      n_tokens, max_seqlen, desc, out, lse, workspace, workspace_bytes,
                      stream) -> int:
    """gdattn_decode_prefix on raw addresses (ints); returns the status code."""
    return lib().gdattn_decode_prefix(q, k_prefix, v_prefix, prefix_len, int(prefix_rows), k, v,
                                      seqlens, int(batch), int(n_tokens), int(max_seqlen),
                                      ctypes.byref(desc), out, lse, workspace,
                                      int(workspace_bytes), stream)


def decode_prefix(q: torch.Tensor, k_prefix: torch.Tensor, v_prefix: Optional[torch.Tensor],
                  prefix_len: torch.Tensor, k: torch.Tensor, v: Optional[torch.Tensor],
                  seqlens: torch.Tensor, desc: LayerDesc, max_seqlen: int,
                  out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                  workspace: Optional[torch.Tensor] = None, stream=None):
    """Attention behind a prefix that the batch shares, through gdattn_decode_prefix.

    q bf16 [T, B, Hq, D]; k_prefix / v_prefix bf16 [prefix_rows, Hkv, D] (v_prefix None
    when K = V); prefix_len int32 [1] on the device; k, v, seqlens the sequences' own
    caches and lengths.  Returns (out, lse), token-major."""
    T, B, index, out, lse = _check_tokens(q, k, v, seqlens, out, lse, desc, stream)
    shape = k_prefix.shape
    rows = shape[0]
    if len(shape) != 3 or shape[1] != desc.n_kv_heads or shape[2] != desc.head_dim:
        raise ValueError(f"k_prefix: shape {tuple(shape)}, expected "
                         f"{('prefix_rows', int(desc.n_kv_heads), int(desc.head_dim))}")
    if max_seqlen > _MOST or rows > _MOST:
        _too_many("max_seqlen or k_prefix rows", max(max_seqlen, rows))
    n = rows * desc.n_kv_heads * desc.head_dim
    _need(k_prefix, "k_prefix", _bf16, n, q, index)
    if v_prefix is not None:
        _need(v_prefix, "v_prefix", _bf16, n, q, index)
    _need(prefix_len, "prefix_len", _i32, 1, q, index)
    if workspace is None:
        workspace = alloc_prefix_workspace(B, T, max_seqlen, rows, desc, q.device, stream)
    _check_workspace(workspace, q, index)
    _call(lib().gdattn_decode_prefix, "gdattn_decode_prefix", index, stream, q.data_ptr(),
          k_prefix.data_ptr(), _ptr(v_prefix), prefix_len.data_ptr(), rows, k.data_ptr(), _ptr(v),
          seqlens.data_ptr(), B, T, max_seqlen, ctypes.byref(desc), out.data_ptr(),
          lse.data_ptr(), workspace.data_ptr(), workspace.numel())
    return out, lse


class RowMap(NamedTuple):
    """Where the packed rows of a step go (gdattn_slot_map), all int32."""

    start: torch.Tensor  # [B + 1]: first row of each sequence, then the step's rows
    seq: torch.Tensor    # [n_rows]: the row's sequence, -1 behind the last row
    pos: torch.Tensor    # [n_rows]: its position in the sequence
    slot: torch.Tensor   # [n_rows]: its slot in the sequence's cache, or -1


def slot_map(seqlens: torch.Tensor, new_lens: torch.Tensor, n_rows: int, capacity: int,
             n_sink: int = 0, out: Optional[RowMap] = None, stream=None) -> RowMap:
    """gdattn_slot_map: the slots of a step in which new_lens[b] tokens join sequence
    b (seqlens[b] long with them), packed into n_rows rows."""
    B, index = seqlens.numel(), seqlens.get_device()
    _need(seqlens, "seqlens", _i32, B, seqlens, index)
    _need(new_lens, "new_lens", _i32, B, seqlens, index)
    if index < 0:
        _on(seqlens, "seqlens", None)
    if n_rows < 0:
        raise ValueError(f"n_rows: {n_rows}")
    if n_rows > _MOST or capacity > _MOST or n_sink > _MOST:
        _too_many("n_rows, capacity or n_sink", max(n_rows, capacity, n_sink))
    if out is None:
        n = B + 1 + 3 * n_rows
        flat = (seqlens.new_empty(n) if stream is None else
                _result((n,), _i32, seqlens.device, stream))
        out = RowMap(*flat.split_with_sizes((B + 1, n_rows, n_rows, n_rows)))
        start = flat.data_ptr()
        seq = start + 4 * (B + 1)
        pos, slot = seq + 4 * n_rows, seq + 8 * n_rows
    else:
        _need(out.start, "out.start", _i32, B + 1, seqlens, index)
        for name in ("seq", "pos", "slot"):
            _need(getattr(out, name), f"out.{name}", _i32, n_rows, seqlens, index)
        start, seq, pos, slot = (t.data_ptr() for t in out)
    _call(lib().gdattn_slot_map, "gdattn_slot_map", index, stream, seqlens.data_ptr(),
          new_lens.data_ptr(), B, n_rows, capacity, n_sink, start, seq, pos, slot)
    return out


def _row_stride(rows: torch.Tensor, name: str, desc: LayerDesc, n_rows: int, like,
                index: int) -> int:
    """Elements between the rows of a bf16 [n_rows, Hkv, D] tensor whose heads are
    next to one another (a slice of a fused projection is)."""
    H, D = desc.n_kv_heads, desc.head_dim
    if rows.dtype is not _bf16:
        raise ValueError(f"{name}: dtype {rows.dtype}, expected torch.bfloat16")
    if rows.dim() != 3 or rows.shape[0] < n_rows or rows.shape[1] != H or rows.shape[2] != D:
        raise ValueError(f"{name}: shape {tuple(rows.shape)}, expected at least {(n_rows, H, D)}")
    stride = rows.stride()
    if stride[2] != 1 or (H > 1 and stride[1] != D):
        raise ValueError(f"{name}: the heads of a row must be next to one another")
    if index < 0 or rows.get_device() != index:
        _on(rows, name, like.device)
    return stride[0] if rows.shape[0] > 1 else H * D


def _check_write(k_rows, v_rows, row_seq, row_slot, desc, k, v, dtypes):
    """The arguments both cache writes share; returns (n_rows, batch, row stride)."""
    index = k.get_device()
    n_rows, batch = row_slot.numel(), k.shape[0]
    if n_rows > _MOST:
        _too_many("row_slot", n_rows)
    _need(row_seq, "row_seq", _i32, n_rows, k, index)
    _need(row_slot, "row_slot", _i32, n_rows, k, index)
    stride = _row_stride(k_rows, "k_rows", desc, n_rows, k, index)
    n = _cache_elems(batch, desc)
    _need_cache(k, "k", dtypes, n, k, index, desc)
    if v_rows is not None and _row_stride(v_rows, "v_rows", desc, n_rows, k, index) != stride:
        raise ValueError("v_rows: must have the row stride of k_rows")
    if v is not None:
        _need_cache(v, "v", dtypes, n, k, index, desc)
    return n_rows, batch, stride


def cache_write_raw(k_rows, v_rows, row_stride, row_seq, row_slot, n_rows, batch, desc, k, v,
                    stream) -> int:
    """gdattn_cache_write on raw addresses (ints); returns the status code."""
    return lib().gdattn_cache_write(k_rows, v_rows, int(row_stride), row_seq, row_slot,
                                    int(n_rows), int(batch), ctypes.byref(desc), k, v, stream)


def cache_write(k_rows: torch.Tensor, v_rows: Optional[torch.Tensor], row_seq: torch.Tensor,
                row_slot: torch.Tensor, desc: LayerDesc, k: torch.Tensor,
                v: Optional[torch.Tensor] = None, stream=None) -> None:
    """gdattn_cache_write: rows bf16 [n_rows, Hkv, D] (any row stride) into the caches
    k, v [B, C, Hkv, D] by a slot map; v_rows and v None when K = V."""
    n_rows, batch, stride = _check_write(k_rows, v_rows, row_seq, row_slot, desc, k, v, _BF16)
    _call(lib().gdattn_cache_write, "gdattn_cache_write", k.get_device(), stream, k_rows.data_ptr(),
          _ptr(v_rows), stride, row_seq.data_ptr(), row_slot.data_ptr(), n_rows, batch,
          ctypes.byref(desc), k.data_ptr(), _ptr(v))


def cache_write_fp8_raw(k_rows, v_rows, row_stride, row_seq, row_slot, n_rows, batch, desc,
                        k_codes, v_codes, k_scale, v_scale, stream) -> int:
    """gdattn_cache_write_fp8 on raw addresses (ints); returns the status code."""
    return lib().gdattn_cache_write_fp8(k_rows, v_rows, int(row_stride), row_seq, row_slot,
                                        int(n_rows), int(batch), ctypes.byref(desc), k_codes,
                                        v_codes, k_scale, v_scale, stream)


def cache_write_fp8(k_rows: torch.Tensor, v_rows: Optional[torch.Tensor], row_seq: torch.Tensor,
                    row_slot: torch.Tensor, desc: LayerDesc, k_codes: torch.Tensor,
                    v_codes: Optional[torch.Tensor], k_scale: torch.Tensor,
                    v_scale: Optional[torch.Tensor] = None, stream=None) -> None:
    """gdattn_cache_write_fp8: rows into the e4m3 caches [B, C, Hkv, D] (uint8 or
    float8_e4m3fn) and their scales, fp32 [B, Hkv, C].  ``decode_fp8`` reads such a cache
    in its own geometry and only when the slot map had no pinned slots (n_sink 0)."""
    n_rows, batch, stride = _check_write(k_rows, v_rows, row_seq, row_slot, desc, k_codes,
                                         v_codes, _CODES)
    index = k_codes.get_device()
    scales = batch * desc.n_kv_heads * desc.cache_capacity
    _need(k_scale, "k_scale", _f32, scales, k_codes, index)
    if v_scale is not None:
        _need(v_scale, "v_scale", _f32, scales, k_codes, index)
    _call(lib().gdattn_cache_write_fp8, "gdattn_cache_write_fp8", index, stream,
          k_rows.data_ptr(), _ptr(v_rows), stride, row_seq.data_ptr(), row_slot.data_ptr(),
          n_rows, batch, ctypes.byref(desc), k_codes.data_ptr(), _ptr(v_codes),
          k_scale.data_ptr(), _ptr(v_scale))
