"""Measured cases of the key/value cache operators: appending rotated keys and values to a paged
cache (bf16 or 4 bits), reading rows back, and attention of new tokens over the cache.

A case is a dict; `prepare` makes its inputs from a seed, `run` makes one pass (elementary torch
operations in 32 bits, or with `own` the calls a user makes of KVCache), `exact` gives the same
outputs from the definitions in 64 bits, `work` the bytes and operations no form can do without.

The definitions:
  append   the key of the new token at position p is rotated by the table row cos_sin[p] (the
           pairs (j, j + rot/2)), rounded to bf16 and stored in its page; 4 bits: per group of
           32 values lo, hi = min, max; s = bf16((hi - lo) * (1/15)); z = bf16(lo + 8 s);
           code = clamp(round((x - z) * (1 / s)) + 8, 0, 15), which stands for s (code - 8) + z.
  read     the values of the last n tokens of each sequence, rounded to bf16.
  attend   query i of n at position p = len - n + i; key u in [max(0, p - window + 1), p]:
           score = scale q.k, then cap tanh(score / cap), then + slope (u - p); softmax.
"""
import math
import random

import torch

own = False

GROUP = 32          # values that share one scale in the 4-bit format
DEV = "cuda"


# --------------------------------------------------------------------------- cases

def _attend(name, fmt, B, L, h_q, h_kv, d_k, d_v, page=64, n_new=1, ragged=False, window=0, cap=0.0, slopes=False):
    c = dict(kind="attend", fmt=fmt, B=B, L=L, h_q=h_q, h_kv=h_kv, d_k=d_k, d_v=d_v, page=page, n_new=n_new,
             ragged=ragged, window=window, cap=cap, slopes=slopes)
    return dict(c, name=name) if name else c


def _append(name, fmt, B, L, n_new, h_q, h_kv, d_k, d_v, page=64, ragged=False, rot=None):
    c = dict(kind="append", fmt=fmt, B=B, L=L, n_new=n_new, h_q=h_q, h_kv=h_kv, d_k=d_k, d_v=d_v, page=page,
             ragged=ragged, rot=d_k if rot is None else rot)
    return dict(c, name=name) if name else c


def _read(name, fmt, B, L, h_kv, d_k, d_v, page=64, ragged=False):
    c = dict(kind="read", fmt=fmt, B=B, L=L, h_kv=h_kv, d_k=d_k, d_v=d_v, page=page, ragged=ragged)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one short chat turn of a small model: latency alone counts
        _attend("attend_int4_b1_short", "int4", 1, 257, 4, 1, 64, 64),
        # a decode step of the serving workload: 32 sequences with a full 64K cache
        _attend("attend_int4_b32_64k", "int4", 32, 65536, 64, 4, 192, 128),
        # one long document, no grouping: the generation stage of a MoBA layer at 128K
        _attend("attend_int4_b1_128k_mha", "int4", 1, 131072, 32, 32, 128, 128),
        # drafts of a speculative step under a sliding window, unequal lengths
        _attend("attend_int4_drafts_window", "int4", 16, 20011, 32, 4, 128, 128, n_new=4, ragged=True, window=4096),
        # continuous batching with small pages, capped and distance-biased scores
        _attend("attend_bf16_ragged_capped", "bf16", 48, 9001, 32, 4, 128, 128, page=16, ragged=True, cap=30.0,
                slopes=True),
        # a decode step over a bf16 cache in the serving head layout
        _attend("attend_bf16_b32_16k", "bf16", 32, 16384, 64, 4, 192, 128),
        # the new token of each sequence in a bf16 cache, queries rotated too
        _append("append_bf16_token", "bf16", 32, 1000, 1, 64, 4, 192, 128),
        # the same into a 4-bit cache, a large batch of small heads
        _append("append_int4_token", "int4", 128, 517, 1, 16, 4, 64, 64, rot=32),
        # packed prompts of unequal lengths into a 4-bit cache
        _append("append_int4_prompts", "int4", 8, 16384, 16384, 64, 4, 192, 128, ragged=True),
        # one prompt of a layer without grouping into a bf16 cache
        _append("append_bf16_prompt_mha", "bf16", 1, 8192, 8192, 32, 32, 128, 128),
        # a long shared prefix back out of the 4-bit cache, for a prompt that continues it
        _read("read_int4_prefix", "int4", 4, 32768, 4, 192, 128),
        # unequal short histories out of small bf16 pages
        _read("read_bf16_ragged", "bf16", 24, 3001, 8, 128, 128, page=16, ragged=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    d_k, d_v = rng.choice([(64, 64), (128, 128), (192, 128)])
    fmt = rng.choice(["int4", "int4", "bf16"])
    page = rng.choice([16, 48, 64, 256])
    h_kv = rng.choice([1, 2, 4, 8, 32])
    kind = rng.choice(["attend", "attend", "attend", "append", "append", "read"])
    B = _log_int(rng, 1, 96)
    ragged = rng.random() < 0.6
    if kind == "attend":
        G = rng.choice([1, 2, 4, 7, 8, 16]) if h_kv < 32 else 1
        n_new = rng.choice([1, 1, 1, 2, 5])
        # cached values over all sequences and heads: 2^15 .. 2^30, so no more than the largest listed case's
        tokens = max(1, _log_int(rng, 2 ** 15, 2 ** 30) // (B * h_kv * (d_k + d_v)))
        L = max(n_new, min(tokens, 131072))
        return _attend(None, fmt, B, L, h_kv * G, h_kv, d_k, d_v, page=page, n_new=n_new, ragged=ragged,
                       window=rng.choice([0, 0, _log_int(rng, 1, 8192)]), cap=rng.choice([0.0, 0.0, 20.0, 50.0]),
                       slopes=rng.random() < 0.3)
    if kind == "append":
        h_q = h_kv * (rng.choice([1, 2, 8]) if h_kv < 32 else 1)
        if rng.random() < 0.5:
            return _append(None, fmt, B, _log_int(rng, 1, 2000), 1, h_q, h_kv, d_k, d_v, page=page, ragged=ragged,
                           rot=rng.choice([d_k, 32]))
        tokens = max(B, _log_int(rng, 2 ** 14, 2 ** 26) // (h_kv * (d_k + d_v)))
        n = max(1, min(tokens // B, 16384))
        return _append(None, fmt, B, n + rng.choice([0, 0, 100]), n, h_q, h_kv, d_k, d_v, page=page, ragged=ragged,
                       rot=rng.choice([d_k, 32]))
    tokens = max(B, _log_int(rng, 2 ** 14, 2 ** 27) // (h_kv * (d_k + d_v)))
    return _read(None, fmt, B, max(1, min(tokens // B, 32768)), h_kv, d_k, d_v, page=page, ragged=ragged)


def _lens(case):
    """Lengths of the sequences (new tokens included): all L, or spread over 0 .. L with the ends among them."""
    B, L = case["B"], case["L"]
    if not case["ragged"]:
        return [L] * B
    rng = random.Random(B * 1000003 + L)
    lens = [rng.randint(0, L) for _ in range(B)]
    lens[0] = L
    if B > 2:
        lens[1] = 0
    return lens


def _counts(case):
    """Rows that an append or a read takes of each sequence."""
    lens = _lens(case)
    if case["kind"] == "read":
        return lens
    return [min(n, case["n_new"]) for n in lens]


def _packed(case):
    return case["kind"] != "attend" and case["ragged"]


# --------------------------------------------------------------------------- layout of the cache

def _code_order(d, kind):
    """Which value each nibble of a stored row holds, in the order of the row's nibbles.  Keys: the
    32-bit words (8 values) of a row are stored transposed as a [4, groups] matrix; values: its
    16-bit halves (4 values) as an [8, groups] one."""
    per = 8 if kind == "k" else 4
    across = GROUP // per
    return torch.arange(d).view(d // GROUP, across, per).transpose(0, 1).reshape(-1)


def _pack(codes, kind):
    d = codes.shape[-1]
    c = codes[..., _code_order(d, kind).to(codes.device)].to(torch.uint8)
    return c[..., 0::2] | (c[..., 1::2] << 4)


def _unpack(rows, kind):
    d = rows.shape[-1] * 2
    c = torch.stack((rows & 15, rows >> 4), dim=-1).flatten(-2)
    out = torch.empty_like(c)
    out[..., _code_order(d, kind).to(rows.device)] = c
    return out


def _quantise(x):
    """x bf16 [..., d] -> codes (float) [..., d], (s, z) bf16 [..., d / 32, 2]."""
    g = x.float().unflatten(-1, (-1, GROUP))
    lo, hi = g.amin(-1), g.amax(-1)
    s = ((hi - lo) * (1.0 / 15.0)).bfloat16().float()
    s = torch.where(s < 2.0 ** -100, torch.zeros_like(s), s)
    z = (lo + 8.0 * s).bfloat16().float()
    inv = torch.where(s > 0, 1.0 / s, torch.zeros_like(s))
    c = (torch.round((g - z[..., None]) * inv[..., None]) + 8.0).clamp(0, 15)
    return c.flatten(-2), torch.stack((s, z), dim=-1).bfloat16()


def _dequantise(codes, sz, dtype=torch.float32):
    g = codes.to(dtype).unflatten(-1, (-1, GROUP))
    sz = sz.to(dtype)
    return ((g - 8.0) * sz[..., 0:1] + sz[..., 1:2]).flatten(-2)


def _places(st, seq, pos):
    """Pages and places in them of positions `pos` of sequences `seq`."""
    return st["table"][seq, pos // st["page"]].long(), pos % st["page"]


def _values(st, seq, pos, dtype=torch.float32):
    """Keys and values of positions `pos` of sequences `seq` as [n, h_kv, d]."""
    pg, off = _places(st, seq, pos)
    if st["fmt"] == "bf16":
        return st["k"][pg, off].to(dtype), st["v"][pg, off].to(dtype)
    return (_dequantise(_unpack(st["k"][pg, :, off], "k"), st["k_scale"][pg, :, off], dtype),
            _dequantise(_unpack(st["v"][pg, :, off], "v"), st["v_scale"][pg, :, off], dtype))


# --------------------------------------------------------------------------- inputs

def _keys(g, n, h, d):
    """N(0, 1) plus one offset vector for each 64 tokens, as real keys cluster along a text."""
    x = torch.randn((n, h, d), generator=g, device=DEV)
    off = torch.randn(((n + 63) // 64, h, d), generator=g, device=DEV) * 0.5
    return (x + off.repeat_interleave(64, 0)[:n]).bfloat16()


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    B, page, h_kv, d_k, d_v = (case[n] for n in ("B", "page", "h_kv", "d_k", "d_v"))
    lens = _lens(case)
    max_pages = max(1, -(-case["L"] // page))
    n_pages = B * max_pages
    st = dict(kind=case["kind"], fmt=case["fmt"], page=page, lens=lens, max_len=max(case["L"], 1), n_new=case.get("n_new", 1),
              window=case.get("window", 0), cap=case.get("cap", 0.0), rot=case.get("rot", 0), d_k=d_k, d_v=d_v, h_kv=h_kv,
              scale=1.0 / math.sqrt(d_k))
    # the pages of a sequence lie anywhere in the pool
    st["table"] = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32).view(B, max_pages)
    st["seqlens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    if case["fmt"] == "bf16":
        st["k"] = torch.zeros((n_pages, page, h_kv, d_k), dtype=torch.bfloat16, device=DEV)
        st["v"] = torch.zeros((n_pages, page, h_kv, d_v), dtype=torch.bfloat16, device=DEV)
        st["k_scale"] = st["v_scale"] = None
    else:
        st["k"] = torch.zeros((n_pages, h_kv, page, d_k // 2), dtype=torch.uint8, device=DEV)
        st["v"] = torch.zeros((n_pages, h_kv, page, d_v // 2), dtype=torch.uint8, device=DEV)
        st["k_scale"] = torch.zeros((n_pages, h_kv, page, d_k // GROUP, 2), dtype=torch.bfloat16, device=DEV)
        st["v_scale"] = torch.zeros((n_pages, h_kv, page, d_v // GROUP, 2), dtype=torch.bfloat16, device=DEV)
    if case["kind"] != "append":
        for b, n in enumerate(lens):
            if n:
                _store(st, b, torch.arange(n, device=DEV), _keys(g, n, h_kv, d_k),
                       torch.randn((n, h_kv, d_v), generator=g, device=DEV).bfloat16())
    counts = _counts(case)
    st["counts"] = counts
    st["cu"] = None
    if _packed(case):
        cu = [0]
        for n in counts:
            cu.append(cu[-1] + n)
        st["cu"] = torch.tensor(cu, dtype=torch.int32, device=DEV)
    if case["kind"] == "attend":
        st["q"] = torch.randn((B, case["n_new"], case["h_q"], d_k), generator=g, device=DEV).bfloat16()
        st["slopes"] = None
        if case["slopes"]:
            st["slopes"] = torch.exp2(-8.0 * torch.arange(1, case["h_q"] + 1, device=DEV, dtype=torch.float64) / case["h_q"]).float()
    elif case["kind"] == "append":
        rows = sum(counts) if _packed(case) else B * case["n_new"]
        lead = (rows,) if _packed(case) else (B, case["n_new"])
        # one projection's output holds the queries, keys and values of a token side by side
        wide = case["h_q"] * d_k + h_kv * (d_k + d_v)
        qkv = torch.randn((rows, wide), generator=g, device=DEV).bfloat16().view(*lead, wide)
        nq, nk = case["h_q"] * d_k, h_kv * d_k
        st["q"] = qkv[..., :nq].unflatten(-1, (case["h_q"], d_k))
        st["k_new"] = qkv[..., nq:nq + nk].unflatten(-1, (h_kv, d_k))
        st["v_new"] = qkv[..., nq + nk:].unflatten(-1, (h_kv, d_v))
        inv_freq = 10000.0 ** (-torch.arange(0, case["rot"], 2, device=DEV, dtype=torch.float64) / case["rot"])
        ang = torch.arange(st["max_len"], device=DEV, dtype=torch.float64)[:, None] * inv_freq
        st["cos_sin"] = torch.cat((ang.cos(), ang.sin()), dim=-1).float()
    if own:
        from block_sparse_attention_compress_b200.torch_ops import KVCache
        st["cache"] = KVCache(B, max_pages * page, h_kv, d_k, d_v, fmt=case["fmt"], page_size=page, n_pages=n_pages,
                              device=DEV)
        st["cache"].page_table.copy_(st["table"])
        for n in ("k", "v", "k_scale", "v_scale"):
            if st[n] is not None:
                getattr(st["cache"], n).copy_(st[n])
                st[n] = None
    return st


def _store(st, seq, pos, k, v):
    """Plain writing of bf16 keys and values [n, h_kv, d] at positions `pos` of sequences `seq`."""
    pg, off = _places(st, seq, pos)
    if st["fmt"] == "bf16":
        st["k"][pg, off] = k
        st["v"][pg, off] = v
        return
    for name, x in (("k", k), ("v", v)):
        codes, sz = _quantise(x)
        st[name][pg, :, off] = _pack(codes, name)
        st[name + "_scale"][pg, :, off] = sz


# --------------------------------------------------------------------------- one pass

def _rotate(x, cs):
    """x bf16 [n, h, d], cs [n, rot] (cosines, then sines): the pairs (j, j + rot/2) rotated, rounded to bf16."""
    half = cs.shape[-1] // 2
    c, s = cs[:, None, :half], cs[:, None, half:]
    x = x.to(cs.dtype)
    a, b, rest = x[..., :half], x[..., half:2 * half], x[..., 2 * half:]
    return torch.cat((a * c - b * s, b * c + a * s, rest), dim=-1).bfloat16()


def _row_index(st, rows):
    """Sequence and position of each of the rows (the last ones of every sequence, one sequence after another)."""
    if st["cu"] is None:
        n = rows // len(st["lens"])
        seq = torch.arange(rows, device=DEV) // n
        return seq, st["seqlens"].long()[seq] - n + torch.arange(rows, device=DEV) % n
    cu = st["cu"].long()
    seq = torch.repeat_interleave(torch.arange(len(st["lens"]), device=DEV), cu[1:] - cu[:-1], output_size=rows)
    return seq, st["seqlens"].long()[seq] - cu[seq + 1] + torch.arange(rows, device=DEV)


def _run_append(st):
    if own:
        c = st["cache"]
        q = c.append(st["k_new"], st["v_new"], st["seqlens"], cu_seqlens=st["cu"], cos_sin=st["cos_sin"], q=st["q"])
        if st["fmt"] == "bf16":
            return {"k": c.k, "v": c.v, "q": q}
        k, v = c.read(st["seqlens"], st["n_new"], cu_seqlens=st["cu"], total=st["k_new"].shape[0])
        return {"k": k, "v": v, "q": q}
    q, k, v = (x.flatten(0, -3) for x in (st["q"], st["k_new"], st["v_new"]))
    seq, pos = _row_index(st, k.shape[0])
    cs = st["cos_sin"][pos]
    q = _rotate(q, cs).view(st["q"].shape)
    _store(st, seq, pos, _rotate(k, cs), v)
    if st["fmt"] == "bf16":
        return {"k": st["k"], "v": st["v"], "q": q}
    k, v = _values(st, seq, pos)
    return {"k": k.bfloat16().view(st["k_new"].shape), "v": v.bfloat16().view(st["v_new"].shape), "q": q}


def _run_read(st):
    total = sum(st["counts"]) if st["cu"] is not None else None
    if own:
        k, v = st["cache"].read(st["seqlens"], st["max_len"], cu_seqlens=st["cu"], total=total)
        return {"k": k, "v": v}
    seq, pos = _row_index(st, sum(st["counts"]))
    k, v = _values(st, seq, pos)
    lead = (len(st["lens"]), st["max_len"]) if total is None else (total,)
    return {"k": k.bfloat16().view(*lead, *k.shape[1:]), "v": v.bfloat16().view(*lead, *v.shape[1:])}


def _attend_one(st, b, dtype):
    """Outputs [n_new, h_q, d_v] and log-sum-exps [n_new, h_q] of sequence b in `dtype`."""
    n_new, L, h_kv = st["n_new"], st["lens"][b], st["h_kv"]
    q = st["q"][b].to(dtype)
    h_q = q.shape[1]
    out = torch.zeros((n_new, h_q, st["d_v"]), dtype=dtype, device=DEV)
    lse = torch.full((n_new, h_q), -math.inf, dtype=dtype, device=DEV)
    if L == 0:
        return out, lse
    first = 0 if st["window"] == 0 else max(0, L - n_new - st["window"] + 1)
    k, v = _values(st, b, torch.arange(first, L, device=DEV), dtype)
    live = max(0, n_new - L)     # queries before the first token have nothing to attend
    q = q[live:].view(n_new - live, h_kv, -1, st["d_k"]).permute(1, 2, 0, 3)       # [h_kv, G, n, d]
    s = torch.matmul(q.flatten(1, 2), k.permute(1, 2, 0)) * st["scale"]            # [h_kv, G n, tokens]
    s = s.unflatten(1, (-1, n_new - live))
    if st["cap"] > 0:
        s = st["cap"] * torch.tanh(s / st["cap"])
    u = torch.arange(first, L, device=DEV)
    p = torch.arange(L - n_new + live, L, device=DEV)
    dist = u[None, :] - p[:, None]
    if st["slopes"] is not None:
        s = s + st["slopes"].to(dtype).view(h_kv, -1, 1, 1) * dist.to(dtype)
    seen = dist <= 0
    if st["window"]:
        seen &= dist > -st["window"]
    s = s.masked_fill(~seen, -math.inf)
    m = s.amax(-1, keepdim=True)
    e = torch.exp(s - m)
    l = e.sum(-1, keepdim=True)
    o = torch.matmul(e.flatten(1, 2), v.permute(1, 0, 2)).unflatten(1, (-1, n_new - live)) / l   # [h_kv, G, n, d_v]
    out[live:] = o.permute(2, 0, 1, 3).reshape(n_new - live, h_q, -1)
    lse[live:] = (m + torch.log(l)).squeeze(-1).permute(2, 0, 1).reshape(n_new - live, h_q)
    return out, lse


def _run_attend(st):
    q = st["q"]
    if own:
        lse = torch.empty(q.shape[:3], dtype=torch.float32, device=DEV)
        out = st["cache"].attend(q, st["seqlens"], st["max_len"], window=st["window"], softcap=st["cap"],
                                 slopes=st["slopes"], lse=lse)
        return {"out": out, "lse": lse}
    out = torch.empty((*q.shape[:3], st["d_v"]), dtype=torch.bfloat16, device=DEV)
    lse = torch.empty(q.shape[:3], dtype=torch.float32, device=DEV)
    for b in range(q.shape[0]):
        o, l = _attend_one(st, b, torch.float32)
        out[b], lse[b] = o.bfloat16(), l
    return {"out": out, "lse": lse}


def run(state):
    return {"attend": _run_attend, "append": _run_append, "read": _run_read}[state["kind"]](state)


# --------------------------------------------------------------------------- 64 bits

def _exact_quantised(x):
    """What 4 bits keep of x (float64 values that bf16 holds): written from the definition, value by value of a group."""
    g = x.reshape(*x.shape[:-1], -1, GROUP)
    lo, hi = g.min(dim=-1, keepdim=True).values, g.max(dim=-1, keepdim=True).values
    s = ((hi - lo) / 15).float().bfloat16().double()
    s[s < 2.0 ** -100] = 0
    z = (lo + 8 * s).float().bfloat16().double()
    steps = torch.where(s > 0, (g - z) / s, torch.zeros_like(g))
    return (z + s * steps.round().clamp(-8, 7)).reshape(x.shape)


def _exact_rotated(x, pos, rot):
    x = x.double().clone()
    j = torch.arange(rot // 2, device=DEV, dtype=torch.float64)
    ang = pos.double()[:, None] * torch.exp(-math.log(10000.0) * 2 * j / rot)
    turned = torch.complex(x[..., :rot // 2], x[..., rot // 2:rot]) * torch.polar(torch.ones_like(ang), ang)[:, None]
    x[..., :rot // 2], x[..., rot // 2:rot] = turned.real, turned.imag
    return x


def _spans(st):
    """(sequence, first row, number of rows, first position) of the sequences' new rows."""
    r = 0
    for b, n in enumerate(st["counts"]):
        if n:
            yield b, r, n, st["lens"][b] - n
        r += n


def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    if case["kind"] == "attend":
        both = [_exact_attend(st, b) for b in range(case["B"])]
        return {"out": torch.stack([o for o, _ in both]), "lse": torch.stack([l for _, l in both])}
    if case["kind"] == "read":
        k = torch.zeros((sum(st["counts"]), st["h_kv"], st["d_k"]), dtype=torch.float64, device=DEV)
        v = torch.zeros((sum(st["counts"]), st["h_kv"], st["d_v"]), dtype=torch.float64, device=DEV)
        r = 0
        for b, n in enumerate(st["counts"]):
            k[r:r + n], v[r:r + n] = _exact_values(st, b, n)
            r += n
        if st["cu"] is None:
            k, v = (x.view(case["B"], case["L"], *x.shape[1:]) for x in (k, v))
        return {"k": k, "v": v}
    q = torch.zeros(st["q"].shape, dtype=torch.float64, device=DEV)
    k = torch.zeros(st["k_new"].shape, dtype=torch.float64, device=DEV)
    v = torch.zeros(st["v_new"].shape, dtype=torch.float64, device=DEV)
    pool_k, pool_v = st["k"].double() if st["fmt"] == "bf16" else None, st["v"].double() if st["fmt"] == "bf16" else None
    flat = lambda x: x.reshape(-1, *x.shape[-2:])
    for b, r, n, p in _spans(st):
        pos = torch.arange(p, p + n, device=DEV)
        flat(q)[r:r + n] = _exact_rotated(flat(st["q"])[r:r + n], pos, st["rot"])
        kr, vr = _exact_rotated(flat(st["k_new"])[r:r + n], pos, st["rot"]), flat(st["v_new"])[r:r + n].double()
        if st["fmt"] == "bf16":
            pg, off = st["table"][b].long()[pos // st["page"]], pos % st["page"]
            pool_k[pg, off], pool_v[pg, off] = kr, vr
        else:
            flat(k)[r:r + n] = _exact_quantised(kr.float().bfloat16().double())
            flat(v)[r:r + n] = _exact_quantised(vr)
    return {"k": pool_k, "v": pool_v, "q": q} if st["fmt"] == "bf16" else {"k": k, "v": v, "q": q}


def _exact_values(st, b, n):
    """Keys and values of the first n positions of sequence b in 64 bits, whole pages at a time."""
    pages = st["table"][b, :-(-n // st["page"])].long()
    both = []
    for name in ("k", "v"):
        if st["fmt"] == "bf16":
            both.append(st[name][pages].double().flatten(0, 1)[:n])
            continue
        byte = st[name][pages]                                                       # [pages, h, page, d / 2]
        nib = torch.stack((byte % 16, byte // 16), dim=-1).flatten(-2)
        per = 8 if name == "k" else 4
        nib = nib.unflatten(-1, (GROUP // per, -1, per)).transpose(-3, -2)           # [.., groups, across, per]
        sz = st[name + "_scale"][pages].double()
        val = (nib.double() - 8) * sz[..., 0, None, None] + sz[..., 1, None, None]
        both.append(val.flatten(-3).transpose(1, 2).flatten(0, 1)[:n])
    return both


def _exact_attend(st, b):
    n_new, L, h_kv, h_q = st["n_new"], st["lens"][b], st["h_kv"], st["q"].shape[2]
    out = torch.zeros((n_new, h_q, st["d_v"]), dtype=torch.float64, device=DEV)
    lse = torch.full((n_new, h_q), -math.inf, dtype=torch.float64, device=DEV)
    if L == 0:
        return out, lse
    k, v = _exact_values(st, b, L)
    G = h_q // h_kv
    for i in range(n_new):
        p = L - n_new + i
        if p < 0:
            continue
        a = max(0, p - st["window"] + 1) if st["window"] else 0
        qi = st["q"][b, i].double().view(h_kv, G, -1)
        s = torch.einsum("hgd,uhd->hgu", qi, k[a:p + 1]) / math.sqrt(st["d_k"])
        if st["cap"] > 0:
            s = torch.tanh(s / st["cap"]) * st["cap"]
        if st["slopes"] is not None:
            s += st["slopes"].double().view(h_kv, G, 1) * torch.arange(a - p, 1, device=DEV, dtype=torch.float64)
        lse[i] = torch.logsumexp(s, -1).view(-1)
        out[i] = torch.einsum("hgu,uhd->hgd", torch.softmax(s, -1), v[a:p + 1]).reshape(h_q, -1)
    return out, lse


# --------------------------------------------------------------------------- the least work

def _row_bytes(case):
    """Bytes of one token's key and value of one head in the cache."""
    d = case["d_k"] + case["d_v"]
    return 2 * d if case["fmt"] == "bf16" else d // 2 + 4 * d // GROUP


def work(case):
    lens, d = _lens(case), case["d_k"] + case["d_v"]
    if case["kind"] == "attend":
        pairs = tokens = 0
        for L in lens:
            n = case["n_new"]
            w = case["window"] or L + 1
            for p in range(max(0, L - n), L):
                pairs += min(p + 1, w)
            tokens += L - max(0, max(0, L - n) - w + 1) if L else 0
        rows = case["B"] * case["n_new"] * case["h_q"]
        return {"bytes": tokens * case["h_kv"] * _row_bytes(case) + rows * (2 * d + 4), "flops": 2 * pairs * case["h_q"] * d}
    rows = sum(_counts(case))
    cache = rows * case["h_kv"] * _row_bytes(case)
    plain = rows * case["h_kv"] * 2 * d
    if case["kind"] == "read":
        return {"bytes": cache + plain, "flops": 0}
    table = min(rows, case["L"]) * case["rot"] * 4
    rotated = rows * (case["h_q"] + case["h_kv"])
    # 4 bits: the stored rows are also read back as the values they stand for
    back = cache + plain if case["fmt"] == "int4" else 0
    return {"bytes": plain + cache + back + table + rows * case["h_q"] * case["d_k"] * 4, "flops": rotated * case["rot"] * 3}
