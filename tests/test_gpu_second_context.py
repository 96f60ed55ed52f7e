"""The library in a second context on the same device: what it keeps of a context (the
kernels' shared-memory limits, how many blocks fit) is found again there."""
import os
import subprocess
import sys

import pytest

from gpu_helpers import require_gpu

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))

SCRIPT = r"""
import ctypes, sys
sys.path[:0] = [%r, %r]
import numpy as np
import torch
import serving_ref as ref
from decode_attention_09_b200 import binding
from test_gpu_serving import GLOBAL, SLIDING, Call

cu = ctypes.CDLL("libcuda.so.1")
u64 = ctypes.c_uint64


def ok(r):
    assert r == 0, f"driver call: {r}"


def alloc(n):
    p = u64()
    ok(cu.cuMemAlloc_v2(ctypes.byref(p), ctypes.c_size_t(n)))
    return p


def upload(t):
    t = t.cpu().contiguous().view(torch.uint8).reshape(-1)
    p = alloc(max(16, t.numel()))
    ok(cu.cuMemcpyHtoD_v2(p, ctypes.c_void_p(t.data_ptr()), ctypes.c_size_t(t.numel())))
    return p.value


def download(p, like):
    t = torch.empty(like.numel() * like.element_size(), dtype=torch.uint8)
    ok(cu.cuMemcpyDtoH_v2(ctypes.c_void_p(t.data_ptr()), u64(p), ctypes.c_size_t(t.numel())))
    return t.view(like.dtype).view(like.shape)


calls = [Call(ref.make_case(1, T=1, lens=[900, 70], window=500, sinks=4, **SLIDING)),
         Call(ref.make_case(2, T=1, lens=[9, 300], prefix=333, softcap=50.0, **GLOBAL))]
want = [[t.cpu() for t in c.run()] for c in calls]
# the sliding layer's plain decode, whose kernel keeps its limits elsewhere
c0 = calls[0]
d0 = binding.make_desc(16, 8, 256, 500, 0.0, 1 / 16, False, c0.desc.cache_capacity)
q0, k0, v0 = (t.cpu() for t in c0.args[:3])
k0, v0 = (torch.nan_to_num(t, 0.5) for t in (k0, v0))
want0 = binding.decode(q0[0].cuda(), k0.cuda(), v0.cuda(), c0.args[3], d0, 900)
want0 = [t.cpu() for t in want0]
torch.cuda.synchronize()

first, ctx = ctypes.c_void_p(), ctypes.c_void_p()
ok(cu.cuCtxGetCurrent(ctypes.byref(first)))
ok(cu.cuCtxCreate_v2(ctypes.byref(ctx), 0, 0))  # and makes it current
null = ctypes.c_void_p(0)
for call, w in list(zip(calls, want)) + [(None, want0)]:
    out, lse = (alloc(t.numel() * t.element_size()).value for t in w)
    if call is None:
        n = binding.workspace_size(2, 900, d0)
        assert n > 0
        ws = alloc(n).value
        st = binding.lib().gdattn_workspace_init(ws, n, null)
        assert st == 0, st
        st = binding.decode_raw(upload(q0), upload(k0), upload(v0),
                                upload(torch.tensor([900, 70], dtype=torch.int32)), 2, 900, d0,
                                out, lse, ws, n, null)
    else:
        n = call.ws.t.numel()
        ws = alloc(n).value
        st = binding.lib().gdattn_workspace_init(ws, n, null)
        assert st == 0, st
        c = call.c
        T, B = c.q.shape[:2]
        q, k, lens = upload(c.q), upload(c.k), upload(c.lens)
        v = None if c.v is None else upload(c.v)
        if c.pk is None:
            st = binding.decode_sink_raw(q, k, v, lens, B, T, call.max_seqlen, call.desc, c.sinks,
                                         out, lse, ws, n, null)
        else:
            pv = None if c.pv is None else upload(c.pv)
            plen = upload(torch.tensor([c.plen], dtype=torch.int32))
            st = binding.decode_prefix_raw(q, upload(c.pk), pv, plen, c.pk.shape[0], k, v, lens,
                                           B, T, call.max_seqlen, call.desc, out, lse, ws, n,
                                           null)
    assert st == 0, binding.status_string(st)
    ok(cu.cuCtxSynchronize())
    for p, t in zip((out, lse), w):
        assert torch.equal(download(p, t), t)
ok(cu.cuCtxSetCurrent(first))
for call, w in zip(calls, want):  # and in the first one again
    assert all(torch.equal(a.cpu(), b) for a, b in zip(call.run(), w))
ok(cu.cuCtxSetCurrent(ctx))
ok(cu.cuCtxDestroy_v2(ctx))
ok(cu.cuCtxSetCurrent(first))
print("same")
"""


def test_second_context():
    require_gpu()
    r = subprocess.run([sys.executable, "-c", SCRIPT % (os.path.dirname(HERE), HERE)],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-3000:]
    assert r.stdout.strip() == "same"
