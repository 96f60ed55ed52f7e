"""Float64 definitions of the continuous-batching operators and their test inputs.

Written from the definitions in include/gdattn.h over *logical* rows (a sequence's
K and V by position); the caches the library reads are filled from those rows, and
every slot that a call may not read holds NaN.
"""
from __future__ import annotations

import math
from dataclasses import dataclass
from typing import List, Optional

import torch

NAN = float("nan")


def slot_of(pos, sinks, capacity):
    """Slot of each position: pinned below ``sinks``, a ring behind."""
    return torch.where(pos < sinks, pos, sinks + (pos - sinks) % (capacity - sinks))


@dataclass
class Case:
    q: torch.Tensor                 # bf16 [T, B, Hq, D]
    k_rows: List[torch.Tensor]      # per sequence bf16 [L, Hkv, D]
    v_rows: Optional[List[torch.Tensor]]
    k: torch.Tensor                 # bf16 [B, C, Hkv, D], NaN where nothing may be read
    v: Optional[torch.Tensor]
    lens: torch.Tensor              # int32 [B]
    window: int
    sinks: int
    capacity: int
    softcap: float
    scale: float
    pk: Optional[torch.Tensor] = None   # prefix rows [rows, Hkv, D], NaN behind plen
    pv: Optional[torch.Tensor] = None
    plen: int = 0


def make_case(seed, T, lens, hq, hkv, dim, window, sinks=0, capacity=None, shared=False,
              softcap=0.0, prefix=None, prefix_rows=None, heavy=1.0, growth=0.0, scale=None,
              q_scale=1.0) -> Case:
    """lens: own tokens per sequence.  The ring holds what the T tokens' windows reach.
    heavy multiplies the pinned rows of K, and growth makes K rows grow with their
    position (to 1 + growth times as large), so that a row's maximum keeps moving."""
    g = torch.Generator().manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g).to(torch.bfloat16)

    B = len(lens)
    if capacity is None:
        capacity = max([1 + sinks] + list(lens))
        if window:
            capacity = min(capacity, sinks + window + T - 1)
            capacity = max(capacity, sinks + 1)
    k_rows, v_rows = [], []
    k = torch.full((B, capacity, hkv, dim), NAN, dtype=torch.bfloat16)
    v = None if shared else torch.full_like(k, NAN)
    for b, L in enumerate(lens):
        kr = normal(max(L, 0), hkv, dim)
        kr[:sinks] *= heavy
        if growth:
            kr *= (1 + growth * torch.arange(len(kr)) / max(1, len(kr)))[:, None, None].to(kr.dtype)
        vr = kr if shared else normal(max(L, 0), hkv, dim)
        pos = torch.arange(max(L, 0))
        low = max(0, L - T + 1 - window) if window else 0  # first window's start
        pos = pos[(pos < sinks) | (pos >= max(low, L - (capacity - sinks)))]
        at = slot_of(pos, sinks, capacity)
        k[b, at] = kr[pos]
        if not shared:
            v[b, at] = vr[pos]
        k_rows.append(kr)
        v_rows.append(vr)
    c = Case(normal(T, B, hq, dim) * q_scale, k_rows, v_rows, k, v, torch.tensor(lens, dtype=torch.int32),
             window, sinks, capacity, softcap,
             1.0 / math.sqrt(dim) if scale is None else scale)
    if prefix is not None:
        rows = prefix_rows or max(1, prefix)
        c.pk = torch.full((rows, hkv, dim), NAN, dtype=torch.bfloat16)
        c.pk[:prefix] = normal(prefix, hkv, dim)
        if not shared:
            c.pv = torch.full_like(c.pk, NAN)
            c.pv[:prefix] = normal(prefix, hkv, dim)
        c.plen = prefix
    return c


@dataclass
class Ref:
    out: torch.Tensor      # float64 [T, B, Hq, D]
    lse: torch.Tensor      # float64 [T, B, Hq]
    out_tol: torch.Tensor
    lse_tol: torch.Tensor


def reference(c: Case, device="cpu") -> Ref:
    """The definition in float64, with the error a correct kernel may have.

    Scores: a dot product of D bf16 products (exact in fp32) accumulated in fp32, in
    D / 16 steps of at most 2^-23 of the sum of magnitudes each (a truncating adder),
    plus 8 such steps for the adds inside a step and the scale; plus 2^-20 for the
    exponential and the soft-cap's tanh.  That is delta.  A weight is then off by at
    most delta relative, its two stored bf16 parts by 2^-14, and the same again for the
    normalisation; the output is rounded once to bf16, by at most 2^-8 relative.
    The log-sum-exp is off by delta plus its own fp32 rounding, 2^-22 of its size and
    2^-20 for the logarithm of the sum."""
    T, B, Hq, D = c.q.shape
    G = Hq // c.k.shape[2]
    out = torch.zeros((T, B, Hq, D), dtype=torch.float64)
    lse = torch.full((T, B, Hq), -math.inf, dtype=torch.float64)
    out_tol, lse_tol = torch.zeros_like(out), torch.zeros_like(lse)
    for b, L in enumerate(c.lens.tolist()):
        p = L - T + torch.arange(T, device=device)
        rows = torch.nonzero((p >= 0) & (L > 0)).flatten()
        if not rows.numel():
            continue
        P = c.plen
        j = torch.arange(P + max(L, 0), device=device)
        at = p[rows][:, None] + P  # position with the prefix in front
        see = j <= at
        if c.window:
            see &= (j > at - c.window) | ((j >= P) & (j < P + c.sinks))
        k, v = c.k_rows[b].to(device), c.v_rows[b].to(device)
        if c.pk is not None:
            k = torch.cat([c.pk[:P].to(device), k])
            v = torch.cat([(c.pk if c.pv is None else c.pv)[:P].to(device), v])
        k, v = k.double(), v.double()
        q = c.q[:, b].to(device)[rows].double()
        for h in range(Hq):
            kh, vh = k[:, h // G], v[:, h // G]
            x = q[:, h] @ kh.T * c.scale
            mag = (q[:, h].abs() @ kh.abs().T * abs(c.scale)).masked_fill(~see, 0.0).amax(-1)
            if c.softcap:
                x = c.softcap * torch.tanh(x / c.softcap)
            x = x.masked_fill(~see, -math.inf)
            z = torch.logsumexp(x, -1)
            w = torch.exp(x - z[:, None])
            o = w @ vh
            delta = (D / 16 + 8) * 2.0 ** -23 * mag + 2.0 ** -20
            spread = w @ vh.abs()
            out[rows.cpu(), b, h] = o.cpu()
            lse[rows.cpu(), b, h] = z.cpu()
            out_tol[rows.cpu(), b, h] = (2.0 ** -8 * o.abs() + spread *
                                         (2 * delta + 2.0 ** -13)[:, None]).cpu()
            lse_tol[rows.cpu(), b, h] = (delta + 2.0 ** -22 * z.abs() + 2.0 ** -20).cpu()
    return Ref(out, lse, out_tol, lse_tol)


def check(out, lse, ref: Ref, what=""):
    out, lse = out.double().cpu(), lse.double().cpu()
    assert torch.isfinite(out).all(), f"{what}: out has values that are not finite"
    empty = ref.lse == -math.inf
    assert torch.equal(lse == -math.inf, empty), f"{what}: empty rows differ"
    assert (out[empty] == 0).all(), f"{what}: an empty row is not zero"
    over = (out - ref.out).abs() - ref.out_tol
    assert over.max() <= 0, f"{what}: out off by {float((out - ref.out).abs().max()):.3g}, " \
                            f"{float(over.max()):.3g} over its tolerance"
    full = ~empty
    d = (lse[full] - ref.lse[full]).abs() - ref.lse_tol[full]
    assert d.numel() == 0 or d.max() <= 0, f"{what}: lse {float(d.max()):.3g} over its tolerance"


def slot_map(lens, new, n_rows, capacity, sinks):
    """gdattn_slot_map, row by row."""
    start, seq, pos, slot = [0], [], [], []
    for b, (L, n) in enumerate(zip(lens, new)):
        n = max(0, n)
        start.append(start[-1] + n)
        for i in range(n):
            p = L - n + i
            seq.append(b)
            pos.append(p)
            keep = p >= 0 and (p < sinks or p >= L - (capacity - sinks))
            slot.append((p if p < sinks else sinks + (p - sinks) % (capacity - sinks))
                        if keep else -1)
    pad = max(0, n_rows - len(seq))
    return [torch.tensor(start, dtype=torch.int32)] + [
        torch.tensor((x + [-1] * pad)[:n_rows], dtype=torch.int32) for x in (seq, pos, slot)]


def e4m3_rows(x):
    """(codes as their values, scale) of rows [..., D], the definition in float64: the
    scale and the quotients are rounded to fp32, the code to the nearest e4m3 number."""
    x = x.double()
    scale = (x.abs().amax(-1) / 448.0).float().double()
    y = torch.where(scale[..., None] > 0, x / scale[..., None], torch.zeros_like(x))
    y = y.float().double()
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(y / step) * step, scale
