"""Measured cases of the continuous-batching operators: attention with pinned
first tokens (sinks), attention over a prefix that a batch shares, slot maps
from request lengths, and the cache write that goes by them.

``run`` computes a case either in plain torch operations (``own`` false) or
through the library's entry points (``own`` true).  Geometries are those of the
layer stacks in ``workloads.py``: sliding layers (head_dim 256, windows of 512
and 1024) and global layers (head_dim 512, one KV head, K = V).
"""
import math

import torch

own = False

BF16 = torch.bfloat16
E4M3_MAX = 448.0


# ------------------------------------------------------------------- cases
def _sink(name, batch, tokens, window, sinks, len_lo, len_hi, capacity, hq=16, hkv=8, dim=256,
          shared=False, softcap=0.0):
    return {"name": name, "op": "sink", "batch": batch, "tokens": tokens, "window": window,
            "sinks": sinks, "len_lo": len_lo, "len_hi": len_hi, "capacity": capacity, "hq": hq,
            "hkv": hkv, "dim": dim, "shared": shared, "softcap": softcap}


def _prefix(name, batch, tokens, prefix, len_lo, len_hi, window=0, hq=16, hkv=1, dim=512,
            shared=True, softcap=0.0):
    # The sequences' own caches: a ring where a window allows one.
    capacity = min(len_hi, window + tokens - 1) if window else len_hi
    return {"name": name, "op": "prefix", "batch": batch, "tokens": tokens, "prefix": prefix,
            "prefix_rows": -(-prefix // 64) * 64, "len_lo": len_lo, "len_hi": len_hi,
            "window": window, "capacity": capacity, "hq": hq, "hkv": hkv, "dim": dim,
            "shared": shared, "softcap": softcap}


def _slots(name, batch, new_lo, new_hi, old_hi, rows, capacity, sinks):
    return {"name": name, "op": "slots", "batch": batch, "new_lo": new_lo, "new_hi": new_hi,
            "old_hi": old_hi, "rows": rows, "capacity": capacity, "sinks": sinks}


def _write(name, batch, new_lo, new_hi, capacity, sinks, hq=16, hkv=8, dim=256, shared=False,
           fp8=False):
    return {"name": name, "op": "write", "batch": batch, "new_lo": new_lo, "new_hi": new_hi,
            "old_hi": 4096, "rows": batch * new_hi, "capacity": capacity, "sinks": sinks,
            "hq": hq, "hkv": hkv, "dim": dim, "shared": shared, "fp8": fp8}


def listed():
    return [
        # One chat on a sliding layer: the smallest decode call, where latency counts.
        _sink("sink_decode_b1_w512", 1, 1, 512, 4, 2048, 2048, 516, softcap=50.0),
        # The 12B stack's sliding layer in steady state: batch 8, every window full.
        _sink("sink_decode_b8_w1024", 8, 1, 1024, 4, 8192, 8192, 1028),
        # A busy server's verify step of speculative decoding: ragged contexts, some
        # shorter than the window, 4 tokens each.
        _sink("sink_verify4_b64_w1024", 64, 4, 1024, 16, 300, 32768, 1100, softcap=50.0),
        # A whole prompt through a sliding layer.
        _sink("sink_prompt_8192_w1024", 1, 8192, 1024, 4, 8192, 8192, 8192),
        # A few chats under one system prompt, global layer: bound by reading the prefix.
        _prefix("prefix_global_b4_p8191", 4, 1, 8191, 1, 300),
        # The same with a full batch: bound by the prefix's products.
        _prefix("prefix_global_b64_p8192", 64, 1, 8192, 1, 1024),
        # A full batch on a sliding layer whose windows still reach into the prefix.
        _prefix("prefix_sliding_b64_p2000", 64, 1, 2000, 1, 700, window=1024, hkv=8, dim=256,
                shared=False, softcap=50.0),
        # Eight users' questions of 64 tokens, read against one long document.
        _prefix("prefix_global_b8_t64_p8192", 8, 64, 8192, 64, 500),
        # Slots of one decode step of a batch of 64.
        _slots("slots_decode_b64", 64, 1, 1, 32768, 64, 1028, 4),
        # Slots of a step that mixes prompts with decoding sequences.
        _slots("slots_mixed_b256", 256, 0, 1000, 32768, 160000, 1028, 4),
        # A step's K and V rows, cut out of the fused projection, into sliding rings.
        _write("write_b16_t1000", 16, 500, 1000, 1028, 4),
        # The same into an fp8 cache: a scale per row, e4m3 codes.
        _write("write_fp8_b16_t1000", 16, 500, 1000, 1024, 0, fp8=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


#: (query heads, KV heads, head_dim, K serves as V)
_LAYERS = [(16, 8, 256, False), (16, 8, 256, False), (16, 8, 256, False), (8, 8, 256, False),
           (8, 2, 256, False), (16, 1, 256, True), (32, 4, 256, False)]
_GLOBALS = [(16, 1, 512, True), (16, 1, 512, True), (16, 1, 512, True), (8, 1, 512, True),
            (16, 2, 512, False), (16, 8, 256, False), (8, 2, 256, False)]


def draw(rng):
    op = rng.choice(["sink", "sink", "sink", "prefix", "prefix", "prefix", "slots", "write"])
    softcap = rng.choice([0.0, 50.0])
    if op == "sink":
        tokens = rng.choice([1, 1, 1, rng.randint(2, 8), _log_int(rng, 9, 4096)])
        batch = _log_int(rng, 1, 64 if tokens <= 8 else max(1, min(16, 8192 // tokens)))
        window = _log_int(rng, 32, 1500)
        sinks = rng.choice([1, 4, 4, 8, rng.randint(1, 70)])
        hi = tokens + _log_int(rng, 1, 32768)
        lo = rng.choice([hi, tokens, tokens])
        hq, hkv, dim, shared = rng.choice(_LAYERS + [(16, 1, 512, True)])
        capacity = sinks + window + tokens - 1 + rng.choice([0, 0, rng.randint(1, 100)])
        c = _sink("", batch, tokens, window, sinks, lo, hi, capacity, hq, hkv, dim, shared,
                  softcap)
    elif op == "prefix":
        tokens = rng.choice([1, 1, 1, rng.randint(2, 8), _log_int(rng, 9, 64)])
        batch = _log_int(rng, 1, 128 if tokens <= 8 else 8)
        hq, hkv, dim, shared = rng.choice(_GLOBALS)
        window = rng.choice([0, _log_int(rng, 128, 2000)]) if dim == 256 else 0
        prefix = _log_int(rng, 30, 8192 if batch * tokens * hq * dim > 1 << 20 else 16384)
        hi = tokens + _log_int(rng, 1, 1000)
        c = _prefix("", batch, tokens, prefix, rng.choice([hi, tokens, tokens]), hi, window, hq,
                    hkv, dim, shared, softcap)
    elif op == "slots":
        batch = _log_int(rng, 1, 512)
        new_hi = rng.choice([1, _log_int(rng, 1, 300)])
        sinks = rng.choice([0, 4, rng.randint(1, 64)])
        c = _slots("", batch, rng.choice([0, 1]), new_hi, _log_int(rng, 1, 100000),
                   batch * new_hi + rng.choice([0, rng.randint(1, 50)]),
                   sinks + _log_int(rng, 16, 8192), sinks)
    else:
        fp8 = rng.choice([False, True])
        hq, hkv, dim, shared = rng.choice(_LAYERS[:5] if fp8 else _LAYERS + _GLOBALS[:4])
        new_hi = rng.choice([1, _log_int(rng, 1, 1000)])
        sinks = rng.choice([0, 4])
        c = _write("", _log_int(rng, 1, 16), rng.choice([0, new_hi]), new_hi,
                   sinks + _log_int(rng, 64, 1500), sinks, hq, hkv, dim, shared, fp8)
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs
class _Inputs:
    def __init__(self, seed):
        self.g = torch.Generator(device="cuda").manual_seed(int(seed))

    def ints(self, n, lo, hi):
        return torch.randint(lo, hi + 1, (n,), generator=self.g, device="cuda",
                             dtype=torch.int32)

    def normal(self, *shape):
        return torch.randn(shape, generator=self.g, device="cuda", dtype=BF16)

    def rows(self, *shape):
        """Cache rows: N(0, 1), one in a hundred four times as large."""
        x = self.normal(*shape)
        heavy = torch.rand(shape[:2], generator=self.g, device="cuda") < 0.01
        return x * (1 + 3 * heavy.to(BF16))[:, :, None, None]


def _prepare_sink(c, g):
    B, C = c["batch"], c["capacity"]
    s = {"q": g.normal(c["tokens"], B, c["hq"], c["dim"]),
         "k": g.rows(B, C, c["hkv"], c["dim"])}
    s["v"] = None if c["shared"] else g.normal(B, C, c["hkv"], c["dim"])
    s["lens"] = g.ints(B, c["len_lo"], c["len_hi"])
    return s


def _prepare_prefix(c, g):
    B, P = c["batch"], c["prefix_rows"]
    s = _prepare_sink(c, g)
    s["pk"] = g.rows(1, P, c["hkv"], c["dim"])[0]
    s["pv"] = None if c["shared"] else g.normal(P, c["hkv"], c["dim"])
    s["plen"] = torch.full((1,), c["prefix"], dtype=torch.int32, device="cuda")
    return s


def _prepare_slots(c, g):
    new = g.ints(c["batch"], c["new_lo"], c["new_hi"])
    return {"new": new, "lens": new + g.ints(c["batch"], 0, c["old_hi"])}


def _prepare_write(c, g):
    s = _prepare_slots(c, g)
    B, C, N, H, D = c["batch"], c["capacity"], c["rows"], c["hkv"], c["dim"]
    parts = 1 if c["shared"] else 2
    # Rows of the fused Q, K, V projection; K's spread differs from row to row.
    fused = g.normal(N, c["hq"] + parts * H, D)
    fused = fused * torch.exp2(torch.rand((N, 1, 1), generator=g.g, device="cuda") * 4 - 2).to(BF16)
    s["k_rows"] = fused[:, c["hq"]:c["hq"] + H]
    s["v_rows"] = None if c["shared"] else fused[:, c["hq"] + H:]
    _, s["seq"], _, s["slot"] = _slot_map(s["lens"], s["new"], N, C, c["sinks"])
    # One row more than the caches have: where the plain form puts rows without a slot.
    kind = torch.uint8 if c["fp8"] else BF16
    for n in ("k", "v")[:parts]:
        s[n + "_flat"] = torch.zeros((B * C + 1, H, D), dtype=kind, device="cuda")
        s[n] = s[n + "_flat"][:B * C].view(B, C, H, D)
        if c["fp8"]:
            s[n + "_scale_flat"] = torch.zeros(B * H * C + 1, device="cuda")
            s[n + "_scale"] = s[n + "_scale_flat"][:B * H * C].view(B, H, C)
    return s


def prepare(case, seed):
    make = {"sink": _prepare_sink, "prefix": _prepare_prefix, "slots": _prepare_slots,
            "write": _prepare_write}[case["op"]]
    return {"case": dict(case), **make(case, _Inputs(seed))}


# ------------------------------------------------------------- plain forms
def _scores(x, c):
    x = x * (1.0 / math.sqrt(c["dim"]))
    return c["softcap"] * torch.tanh(x / c["softcap"]) if c["softcap"] else x


def _weights(s, mask):
    """Softmax weights over the last axis and its log-sum-exp; rows without a key get zeros."""
    s = s.masked_fill(~mask, -math.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = torch.exp(s - m)
    n = p.sum(-1, keepdim=True)
    return p / torch.where(n > 0, n, torch.ones_like(n)), (m + torch.log(n)).squeeze(-1)


def _run_sink(s):
    c = s["case"]
    T, B, Hq, D = s["q"].shape
    H, S, W, C = c["hkv"], c["sinks"], c["window"], c["capacity"]
    block = min(T, 1024)
    nb = -(-T // block)
    q = torch.nn.functional.pad(s["q"].float(), (0, 0, 0, 0, 0, 0, 0, nb * block - T))
    q = q.view(nb, block, B, H, Hq // H, D)
    lens = s["lens"].long()
    dev = lens.device
    first = lens[:, None] - T + block * torch.arange(nb, device=dev)  # [B, nb]
    qpos = first[:, :, None] + torch.arange(block, device=dev)
    near = first[:, :, None] - (W - 1) + torch.arange(block + W - 1, device=dev)
    pinned = torch.arange(S, device=dev).expand(B, nb, S)
    pos = torch.cat([pinned, near], -1)  # [B, nb, n]
    is_pinned = torch.arange(pos.shape[-1], device=dev) < S
    slot = torch.where(pos < S, pos.clamp(min=0), S + (pos - S).clamp(min=0) % (C - S))
    b = torch.arange(B, device=dev)[:, None, None]
    k = s["k"][b, slot].float()
    v = k if s["v"] is None else s["v"][b, slot].float()
    x = _scores(torch.einsum("nqbhgd,bnkhd->bnhgqk", q, k), c)
    seen = (pos[:, :, None] <= qpos[..., None]) & (pos[:, :, None] >= 0)
    seen &= torch.where(is_pinned, pos[:, :, None] < S,
                        (pos[:, :, None] >= S) & (pos[:, :, None] > qpos[..., None] - W))
    p, lse = _weights(x, seen[:, :, None, None])
    o = torch.einsum("bnhgqk,bnkhd->nqbhgd", p, v).reshape(nb * block, B, Hq, D)[:T]
    lse = lse.permute(1, 4, 0, 2, 3).reshape(nb * block, B, Hq)[:T]
    return {"out": o.to(BF16), "lse": lse.contiguous()}


def _run_prefix(s):
    c = s["case"]
    T, B, Hq, D = s["q"].shape
    H, W, C = c["hkv"], c["window"], c["capacity"]
    n = min(c["len_hi"], W + T - 1) if W else c["len_hi"]
    lens = s["lens"].long()
    dev = lens.device
    q = s["q"].float().view(T, B, H, Hq // H, D)
    qpos = (lens - T) + torch.arange(T, device=dev)[:, None]  # [T, B], behind the prefix
    pos = (lens - n)[:, None] + torch.arange(n, device=dev)  # [B, n]
    slot = pos.clamp(min=0) % C
    b = torch.arange(B, device=dev)[:, None]
    k = s["k"][b, slot].float()
    v = k if s["v"] is None else s["v"][b, slot].float()
    pk = s["pk"].float()
    pv = pk if s["pv"] is None else s["pv"].float()
    own_keys = (pos >= 0) & (pos <= qpos[..., None])
    ppos = torch.arange(pk.shape[0], device=dev)
    plen = s["plen"].long()
    shared_keys = ((ppos < plen) & (qpos[..., None] >= 0)).expand(T, B, -1)
    if W:
        own_keys &= pos > qpos[..., None] - W
        shared_keys = shared_keys & (ppos - plen > qpos[..., None] - W)
    x = torch.cat([torch.einsum("tbhgd,khd->tbhgk", q, pk),
                   torch.einsum("tbhgd,bkhd->tbhgk", q, k)], -1)
    p, lse = _weights(_scores(x, c), torch.cat([shared_keys, own_keys], -1)[:, :, None, None])
    o = torch.einsum("tbhgk,khd->tbhgd", p[..., :pk.shape[0]], pv)
    o = o + torch.einsum("tbhgk,bkhd->tbhgd", p[..., pk.shape[0]:], v)
    return {"out": o.reshape(T, B, Hq, D).to(BF16), "lse": lse.reshape(T, B, Hq)}


def _slot_map(lens, new, rows, C, S):
    """Where each row of a step goes: its sequence, position and slot (-1: none)."""
    start = torch.zeros(new.numel() + 1, dtype=torch.int64, device=new.device)
    start[1:] = torch.cumsum(new.long(), 0)
    r = torch.arange(rows, device=new.device)
    seq = torch.searchsorted(start[1:], r, right=True)
    real = seq < new.numel()
    b = seq.clamp(max=new.numel() - 1)
    L = lens.long()[b]
    pos = L - new.long()[b] + r - start[b]
    ring = S + (pos - S).clamp(min=0) % (C - S)
    slot = torch.where(pos < S, pos, torch.where(pos >= L - (C - S), ring, -1))
    return [x.to(torch.int32) for x in (start, torch.where(real, seq, -1),
                                        torch.where(real, pos, -1), torch.where(real, slot, -1))]


def _run_slots(s):
    c = s["case"]
    start, seq, pos, slot = _slot_map(s["lens"], s["new"], c["rows"], c["capacity"], c["sinks"])
    return {"start": start, "seq": seq, "pos": pos, "slot": slot}


def _written(s):
    names = ("k",) if s["case"]["shared"] else ("k", "v")
    if s["case"]["fp8"]:
        return {**{n: s[n].view(torch.float8_e4m3fn) for n in names},
                **{n + "_scale": s[n + "_scale"] for n in names}}
    return {n: s[n] for n in names}


def _run_write(s):
    c = s["case"]
    B, C, H = c["batch"], c["capacity"], c["hkv"]
    seq, slot = s["seq"].long(), s["slot"].long()
    at = torch.where(slot < 0, B * C, seq * C + slot)
    heads = torch.arange(H, device=at.device)
    scale_at = torch.where(slot[:, None] < 0, B * H * C,
                           (seq[:, None] * H + heads) * C + slot[:, None])
    for n in ("k",) if c["shared"] else ("k", "v"):
        rows = s[n + "_rows"]
        if c["fp8"]:
            x = rows.float()
            amax = x.abs().amax(-1)
            scale = amax / torch.full_like(amax, E4M3_MAX)  # a quotient: no product with 1/448
            x = torch.where(scale[..., None] > 0, x / scale[..., None], torch.zeros_like(x))
            rows = x.to(torch.float8_e4m3fn).view(torch.uint8)
            s[n + "_scale_flat"].index_copy_(0, scale_at.reshape(-1), scale.reshape(-1))
        s[n + "_flat"].index_copy_(0, at, rows)
    return _written(s)


# ------------------------------------------------------- the library's calls
def _plan(s):
    """What a program that runs this layer keeps: the descriptor and the workspace."""
    from decode_attention_09_b200 import binding
    if "plan" not in s:
        c = s["case"]
        desc = binding.make_desc(c["hq"], c["hkv"], c["dim"], c.get("window", 0),
                                 c.get("softcap", 0.0), 1.0 / math.sqrt(c["dim"]), c["shared"],
                                 c["capacity"])
        ws = None
        if c["op"] == "sink":
            ws = binding.alloc_sink_workspace(c["batch"], c["tokens"], c["len_hi"], desc,
                                              c["sinks"])
        elif c["op"] == "prefix":
            ws = binding.alloc_prefix_workspace(c["batch"], c["tokens"], c["len_hi"],
                                                c["prefix_rows"], desc)
        s["plan"] = binding, desc, ws
    return s["plan"]


def _own_sink(s):
    binding, desc, ws = _plan(s)
    out, lse = binding.decode_sink(s["q"], s["k"], s["v"], s["lens"], desc, s["case"]["len_hi"],
                                   s["case"]["sinks"], workspace=ws)
    return {"out": out, "lse": lse}


def _own_prefix(s):
    binding, desc, ws = _plan(s)
    out, lse = binding.decode_prefix(s["q"], s["pk"], s["pv"], s["plen"], s["k"], s["v"],
                                     s["lens"], desc, s["case"]["len_hi"], workspace=ws)
    return {"out": out, "lse": lse}


def _own_slots(s):
    from decode_attention_09_b200 import binding
    c = s["case"]
    m = binding.slot_map(s["lens"], s["new"], c["rows"], c["capacity"], c["sinks"])
    return {"start": m.start, "seq": m.seq, "pos": m.pos, "slot": m.slot}


def _own_write(s):
    binding, desc, _ = _plan(s)
    if s["case"]["fp8"]:
        binding.cache_write_fp8(s["k_rows"], s["v_rows"], s["seq"], s["slot"], desc, s["k"],
                                s["v"], s["k_scale"], s["v_scale"])
    else:
        binding.cache_write(s["k_rows"], s["v_rows"], s["seq"], s["slot"], desc, s["k"],
                            s.get("v"))
    return _written(s)


def run(state):
    op = state["case"]["op"]
    if own:
        return {"sink": _own_sink, "prefix": _own_prefix, "slots": _own_slots,
                "write": _own_write}[op](state)
    return {"sink": _run_sink, "prefix": _run_prefix, "slots": _run_slots,
            "write": _run_write}[op](state)


# -------------------------------------------------------------------- work
def _mean(lo, hi, f, n=64):
    return sum(f(lo + (hi - lo) * (i + 0.5) / n) for i in range(n)) / n


def work(case):
    c = case
    B = c["batch"]
    if c["op"] == "slots":
        return {"bytes": 8.0 * B + 4.0 * (B + 1) + 12.0 * c["rows"], "flops": 0.0}
    H, D = c["hkv"], c["dim"]
    if c["op"] == "write":
        rows = B * (c["new_lo"] + c["new_hi"]) / 2.0
        kept = B * _mean(c["new_lo"], c["new_hi"], lambda n: min(n, c["capacity"]))
        tensors = 1 if c["shared"] else 2
        out = D + 4 if c["fp8"] else 2 * D
        return {"bytes": tensors * kept * H * (2.0 * D + out) + 8.0 * rows, "flops": 0.0}
    T, W, S = c["tokens"], c["window"], c.get("sinks", 0)
    row = H * D * 2 * (1 if c["shared"] else 2)

    def keys(p):  # keys of a query at position p
        return min(p + 1, W + min(S, max(0, p + 1 - W))) if W else p + 1

    def union(length):
        return min(length, W + T - 1 + S) if W else length

    pairs = B * T * _mean(c["len_lo"], c["len_hi"], lambda n: _mean(n - T, n - 1, keys))
    read = B * _mean(c["len_lo"], c["len_hi"], union) * row
    if c["op"] == "prefix":
        P = c["prefix"]

        def seen(p):  # prefix keys of a query at position p behind it
            return min(P, max(0.0, W - 1 - p)) if W else P

        pairs += B * T * _mean(c["len_lo"], c["len_hi"], lambda n: _mean(n - T, n - 1, seen))
        read += (min(P, W) if W else P) * row
    return {"bytes": read + T * B * c["hq"] * (4.0 * D + 4) + 4 * B,
            "flops": 4.0 * D * c["hq"] * pairs}


# ------------------------------------------------------------ in 64 bits
def _exact_sink(c, s):
    q, lens, S, W = s["q"].double(), s["lens"].tolist(), c["sinks"], c["window"]
    T, B, Hq, D = q.shape
    G, C = Hq // c["hkv"], c["capacity"]
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    lse = torch.full((T, B, Hq), -math.inf, dtype=torch.float64, device=q.device)
    for b, L in enumerate(lens):
        for t0 in range(0, T, 512):
            p = torch.arange(t0, min(T, t0 + 512), device=q.device) + L - T
            lo = max(0, int(p[0]) + 1 - W)
            j = torch.arange(int(p[-1]) + 1, device=q.device)
            j = j[(j < S) | (j >= lo)]
            at = torch.where(j < S, j, S + (j - S) % (C - S))
            see = (j <= p[:, None]) & ((j < S) | (j > p[:, None] - W))
            _exact_rows(c, q[t0:t0 + 512, b], s["k"][b, at],
                        (s["k"] if s["v"] is None else s["v"])[b, at], see,
                        out[t0:t0 + 512, b], lse[t0:t0 + 512, b], G)
    return {"out": out, "lse": lse}


def _exact_rows(c, q, k, v, see, out, lse, G):
    """q [t, Hq, D] over keys k, v [n, H, D] where see [t, n]; written into out and lse."""
    if not k.shape[0]:
        return
    for h in range(q.shape[1]):
        x = q[:, h] @ k[:, h // G].double().T / math.sqrt(c["dim"])
        if c["softcap"]:
            x = c["softcap"] * torch.tanh(x / c["softcap"])
        x = torch.where(see, x, -math.inf)
        z = torch.logsumexp(x, -1)
        lse[:, h] = z
        p = torch.where(see, torch.exp(x - z[:, None]), 0.0)
        out[:, h] = p @ v[:, h // G].double()


def _exact_prefix(c, s):
    q, lens, W, P = s["q"].double(), s["lens"].tolist(), c["window"], c["prefix"]
    T, B, Hq, D = q.shape
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    lse = torch.full((T, B, Hq), -math.inf, dtype=torch.float64, device=q.device)
    for b, L in enumerate(lens):
        p = P + L - T + torch.arange(T, device=q.device)  # in prefix and own tokens together
        j = torch.arange(max(0, L - c["capacity"]), L, device=q.device)
        k = torch.cat([s["pk"][:P], s["k"][b, j % c["capacity"]]])
        v = k
        if s["v"] is not None:
            v = torch.cat([s["pv"][:P], s["v"][b, j % c["capacity"]]])
        j = torch.cat([torch.arange(P, device=q.device), P + j])
        see = j <= p[:, None]
        if W:
            see &= j > p[:, None] - W
        _exact_rows(c, q[:, b], k, v, see, out[:, b], lse[:, b], Hq // c["hkv"])
    return {"out": out, "lse": lse}


def _exact_write(c, s):
    got = {n: x.double() for n, x in _written(s).items()}  # zeros
    seq, slot = s["seq"].long(), s["slot"].long()
    keep = slot >= 0
    seq, slot = seq[keep], slot[keep]
    for n in ("k",) if c["shared"] else ("k", "v"):
        x = s[n + "_rows"][keep].double()
        if c["fp8"]:
            # By definition the scale is the 32-bit quotient, and a code is the nearest
            # e4m3 number (ties to even) to the 32-bit quotient of value and scale.
            scale = (x.abs().amax(-1) / E4M3_MAX).float().double()
            x = (x / scale[..., None]).float().double()
            step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
            x = torch.round(x / step) * step
            got[n + "_scale"][seq, :, slot] = scale
        got[n][seq, slot] = x
    return got


def exact(case, seed):
    if case["op"] == "slots":
        return None
    s = prepare(case, seed)
    return {"sink": _exact_sink, "prefix": _exact_prefix, "write": _exact_write}[case["op"]](
        s["case"], s)
