"""The paged key/value cache on the GPU: append, read and attention against the fp64 oracle.

Tolerances.  Stored values are checked exactly where the definition fixes every rounding, else by
half a step (2^-8 of the value in bf16) plus fp32's error of the products.  Attention: the output
is rounded once to bf16 (2^-8 |out|) and the weights once before the product with the values
(bf16: 2^-8 sum P |v|; 4 bits, where the weight is rounded together with the group's scale and meets
a code c - 8 in [-8, 7]: 2^-8 sum P 8 s); a score that is off by e changes a weight by a factor
exp(e), so the output by up to 2 e sum P |v|.  e: fp32 sums of up to 192 products, 2^-17 of
scale sum |q||k| (192 roundings or truncations of 2^-24.4 each), and 2^-20 of the bias or cap.
"""
import math

import pytest
import torch

import block_sparse_attention_compress_b200 as nsa
from block_sparse_attention_compress_b200 import build
from block_sparse_attention_compress_b200.torch_ops import KVCache, compress_torch
from oracle import cache_oracle as co

pytestmark = pytest.mark.gpu
DEV = "cuda"
DIMS = [(64, 64), (128, 128), (192, 128)]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()


def gen(seed):
    return torch.Generator().manual_seed(seed)


def bf(shape, g, scale=1.0):
    return (torch.randn(shape, generator=g) * scale).bfloat16()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def table(n, rot, base=10000.0):
    ang = torch.arange(n).double()[:, None] * base ** (-torch.arange(0, rot, 2).double() / rot)
    return torch.cat((ang.cos(), ang.sin()), -1).float()


def shuffled(batch, max_len, h_kv, dk, dv, fmt, page, seed, spare=3):
    """A cache whose sequences' pages lie anywhere in a pool with some pages to spare."""
    max_pages = -(-max_len // page)
    c = KVCache(batch, max_len, h_kv, dk, dv, fmt=fmt, page_size=page, n_pages=batch * max_pages + spare, device=DEV)
    order = torch.randperm(batch * max_pages + spare, generator=gen(seed))[:batch * max_pages]
    c.page_table.copy_(order.view(batch, max_pages))
    return c


def cu_of(counts):
    return i32([0] + torch.tensor(counts).cumsum(0).tolist())


def pools(c):
    return [t for t in (c.k, c.v, c.k_scale, c.v_scale) if t is not None]


def bits(t):
    return t.contiguous().view(torch.uint8)


def stored_row(c, name, b, p):
    """What the pool holds for position p of sequence b: [h, d] bf16, or codes [h, d], s, z [h, d / 32]."""
    page, off = int(c.page_table[b, p // c.page_size]), p % c.page_size
    pool = getattr(c, name)
    if c.fmt == "bf16":
        return pool[page, off].cpu()
    byte = pool[page, :, off].cpu()
    nib = torch.stack((byte & 15, byte >> 4), -1).flatten(-2)
    d = nib.shape[-1]
    order = co.nibble_order_keys(d) if name == "k" else co.nibble_order_values(d)
    codes = torch.empty_like(nib)
    codes[:, torch.tensor(order)] = nib
    sz = getattr(c, name + "_scale")[page, :, off].cpu()
    return codes, sz[..., 0], sz[..., 1]


# ------------------------------------------------------------------ append and read

@pytest.mark.parametrize("fmt", ["bf16", "int4"])
@pytest.mark.parametrize("dk,dv", DIMS)
@pytest.mark.parametrize("rot,interleaved", [(0, False), (16, False), (None, False), (None, True), (48, True)])
def test_append_stores_rotated_rows(fmt, dk, dv, rot, interleaved):
    rot = dk if rot is None else rot
    g = gen(dk + rot)
    B, h_kv, h_q, page = 3, 3, 6, 16
    lens, counts = [37, 5, 20], [21, 5, 1]
    c = shuffled(B, 48, h_kv, dk, dv, fmt, page, 1)
    n = sum(counts)
    # slices of one projection's output, tokens a wide row apart
    wide = bf((n, h_q * dk + h_kv * (dk + dv)), g)
    q, k, v = (x.unflatten(-1, (-1, d)) for x, d in
               zip(wide.split([h_q * dk, h_kv * dk, h_kv * dv], -1), (dk, dk, dv)))
    dev = wide.to(DEV)
    qd, kd, vd = (x.unflatten(-1, (-1, d)) for x, d in
                  zip(dev.split([h_q * dk, h_kv * dk, h_kv * dv], -1), (dk, dk, dv)))
    cs = table(64, rot) if rot else None
    qo = c.append(kd, vd, i32(lens), cu_seqlens=cu_of(counts), cos_sin=cs.to(DEV) if rot else None,
                  interleaved=interleaved, q=qd).cpu()
    assert c.device_status() == 0
    row = 0
    for b in range(B):
        for i in range(counts[b]):
            p = lens[b] - counts[b] + i
            for got, x in ((qo[row], q[row]), (None, k[row])):
                exact = co.rotate(x, cs[p], interleaved) if rot else x.double()
                mag = x.double().abs().amax(-1, keepdim=True)
                if got is None:
                    if fmt == "int4":
                        continue
                    got = stored_row(c, "k", b, p)
                # products and their sum in fp32 (three roundings of at most 2 max|x|), then half a step
                assert ((got.double() - exact).abs() <= exact.abs() * 2 ** -8 * 1.001 + mag * 2 ** -21).all(), (b, p)
                assert torch.equal(got[:, rot:], x[:, rot:])
            if fmt == "bf16":
                assert torch.equal(stored_row(c, "v", b, p), v[row])
            else:
                want_v = co.quantise(v[row].unflatten(-1, (-1, 32)))
                codes, s, z = stored_row(c, "v", b, p)
                assert torch.equal(codes, want_v[0].flatten(-2)) and torch.equal(s.float(), want_v[1]) and \
                    torch.equal(z.float(), want_v[2])
            row += 1
    if fmt == "int4":   # the keys' codes are those of the rotated rows that a bf16 cache holds
        c16 = shuffled(B, 48, h_kv, dk, dv, "bf16", page, 1)
        c16.append(kd, vd, i32(lens), cu_seqlens=cu_of(counts), cos_sin=cs.to(DEV) if rot else None,
                   interleaved=interleaved)
        for b in range(B):
            for p in range(lens[b] - counts[b], lens[b]):
                want = co.quantise(stored_row(c16, "k", b, p).unflatten(-1, (-1, 32)))
                codes, s, z = stored_row(c, "k", b, p)
                assert torch.equal(codes, want[0].flatten(-2)) and torch.equal(s.float(), want[1]) and \
                    torch.equal(z.float(), want[2]), (b, p)


@pytest.mark.parametrize("fmt", ["bf16", "int4"])
@pytest.mark.parametrize("page,h_kv,lens,n", [(16, 1, [1, 0, 40], 1), (64, 4, [64, 65, 63], 63), (48, 2, [100, 7, 33], 9),
                                              (256, 8, [300, 256, 1], 2)])
def test_padded_rows_go_where_they_belong(fmt, page, h_kv, lens, n):
    """Rows before position 0 are not written, everything else in the pools stays as it was, and the
    padded queries are zeros; a read of the same rows gives them back, padding as zeros."""
    dk = dv = 64
    B, g = len(lens), gen(page)
    c = shuffled(B, 320, h_kv, dk, dv, fmt, page, 2)
    for t in pools(c):
        bits(t).random_(0, 255)
        if t.dtype == torch.bfloat16:
            t.copy_(torch.randn(t.shape, device=DEV))
    before = [t.clone() for t in pools(c)]
    k, v, q = bf((B, n, h_kv, dk), g), bf((B, n, h_kv, dv), g), bf((B, n, 2, dk), g)
    cs = table(320, 64)
    qo = c.append(k.to(DEV), v.to(DEV), i32(lens), cos_sin=cs.to(DEV), q=q.to(DEV)).cpu()
    assert c.device_status() == 0
    mask = [torch.zeros(t.shape[:3], dtype=torch.bool) for t in before]
    for b in range(B):
        for i in range(n):
            p = lens[b] - n + i
            if p < 0:
                assert not qo[b, i].any()
                continue
            pg, off = int(c.page_table[b, p // page]), p % page
            for m in mask:
                if fmt == "bf16":
                    m[pg, off] = True
                else:
                    m[pg, :, off] = True
            if p == 0:
                assert torch.equal(qo[b, i], q[b, i])
    for was, now, m in zip(before, pools(c), mask):
        assert torch.equal(bits(was)[~m.to(DEV)], bits(now)[~m.to(DEV)])
    ko, vo = (x.cpu() for x in c.read(i32(lens), n))
    for b in range(B):
        for i in range(n):
            p = lens[b] - n + i
            if p < 0:
                assert not ko[b, i].any() and not vo[b, i].any()
            elif fmt == "bf16":
                assert torch.equal(vo[b, i], v[b, i]) and torch.equal(ko[b, i], stored_row(c, "k", b, p))
            else:
                for got, name in ((ko, "k"), (vo, "v")):
                    codes, s, z = stored_row(c, name, b, p)
                    want = co.dequantise(codes.unflatten(-1, (-1, 32)), s, z).flatten(-2)
                    assert torch.equal(got[b, i], want.bfloat16()), (b, i, name)


def test_rows_of_no_sequence_stay(fmt="int4"):
    """Packed rows outside [cu[0], cu[B]) are neither written to the cache nor to the outputs."""
    g = gen(5)
    c = shuffled(2, 64, 2, 64, 64, fmt, 16, 3)
    before = [t.clone() for t in pools(c)]
    k, v, q = bf((12, 2, 64), g).to(DEV), bf((12, 2, 64), g).to(DEV), bf((12, 4, 64), g).to(DEV)
    cu, lens = i32([3, 3, 8]), i32([9, 20])
    q_out = torch.full_like(q, 7.0)
    assert c.append(k, v, lens, cu_seqlens=cu, q=q, q_out=q_out) is q_out
    assert (q_out[:3] == 7).all() and (q_out[8:] == 7).all() and torch.equal(q_out[3:8], q[3:8])
    # only positions 15 .. 19 of sequence 1 changed: pages 0 and 1 of it
    pages = set(c.page_table[1, :2].tolist())
    for was, now in zip(before, pools(c)):
        for pg in range(was.shape[0]):
            assert pg in pages or torch.equal(bits(was[pg]), bits(now[pg]))
    ko, vo = (torch.full((12, 2, 64), 5.0, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    c.read(lens, cu_seqlens=cu, total=12, k_out=ko, v_out=vo)
    for x in (ko, vo):
        assert (x[:3] == 5).all() and (x[8:] == 5).all() and not (x[3:8] == 5).all()
    assert c.device_status() == 0


def test_four_bit_groups_at_the_edges_of_the_type():
    """Constant, tiny, huge and non-finite groups, against the definition."""
    g = gen(6)
    rows = bf((12, 1, 64), g)
    rows[0], rows[1], rows[2] = 0.0, 3.0, -1e30
    rows[3] *= 1e-30
    rows[4] *= 1e36
    rows[5, 0, :32] = torch.linspace(-3.3e38, 3.3e38, 32).bfloat16()        # a span beyond fp32
    rows[6, 0, 3], rows[7, 0, 40], rows[8, 0, 63] = math.nan, math.inf, -math.inf
    rows[9, 0, 0] = 100.0
    rows[10] = rows[10] * 1e-3 + 5.0
    rows[11] *= 1e-38
    c = KVCache(1, 16, 1, 64, 64, fmt="int4", page_size=16, device=DEV)
    c.append(rows.to(DEV)[None], rows.to(DEV)[None], i32([12]))
    assert c.device_status() == 0
    ko, vo = (x.cpu()[0] for x in c.read(i32([12]), 12))
    for name, got in (("k", ko), ("v", vo)):
        for p in range(12):
            want = co.quantise(rows[p].unflatten(-1, (-1, 32)))
            codes, s, z = stored_row(c, name, 0, p)
            assert torch.equal(codes, want[0].flatten(-2)), p
            assert torch.equal(s.float().nan_to_num(9), want[1].nan_to_num(9)) and \
                torch.equal(z.float().nan_to_num(9), want[2].nan_to_num(9)), p
            val = co.dequantise(*want).flatten(-2).bfloat16()
            assert torch.equal(got[p].nan_to_num(9), val.nan_to_num(9)), p


def test_tokens_that_have_no_place_are_skipped_and_told():
    g = gen(7)
    k, v = bf((2, 4, 1, 64), g).to(DEV), bf((2, 4, 1, 64), g).to(DEV)
    q = bf((2, 4, 1, 64), g).to(DEV)

    def fresh(fmt="bf16"):
        c = shuffled(2, 32, 1, 64, 64, fmt, 16, 4)
        return c, [t.clone() for t in pools(c)]

    for fmt in ("bf16", "int4"):
        for bad in (-1, 10 ** 6, 2 ** 31 - 1, -2 ** 31):                # a page out of the pool
            c, before = fresh(fmt)
            c.page_table[1, 1] = bad
            qo = c.append(k, v, i32([0, 18]), q=q)                      # positions 14, 15 | 16, 17 of sequence 1
            assert c.device_status() == nsa.NSA_CODE_CACHE
            assert nsa.nsa_device_status(c.status) == (nsa.NSA_ERR_INVALID_ARG, nsa.NSA_CODE_CACHE)
            assert torch.equal(qo[1, :2], q[1, :2]) and not qo[1, 2:].any() and not qo[0].any()
            c.status.zero_()
            ko, _ = c.read(i32([0, 18]), 4)
            assert c.device_status() == nsa.NSA_CODE_CACHE and not ko[1, 2:].any() and ko[1, :2].any()
        for length in (33, 2 ** 31 - 1):                                # beyond the capacity
            c, before = fresh(fmt)
            c.append(k, v, i32([0, length]))
            assert c.device_status() == nsa.NSA_CODE_CACHE
        c, before = fresh(fmt)
        c.append(k, v, i32([-5, -2 ** 31]))                             # nothing there: all padding
        assert c.device_status() == 0 and all(torch.equal(a, b) for a, b in zip(before, pools(c)))
        c, _ = fresh(fmt)
        c.append(k, v, i32([4, 12]), cos_sin=table(10, 64).to(DEV))     # positions 10, 11 have no angles
        assert c.device_status() == nsa.NSA_CODE_CACHE
        ko, vo = c.read(i32([4, 12]), 4)
        assert torch.equal(vo[1, :2], v[1, :2]) or fmt == "int4"
        assert not vo[1, 2:].any()


# ------------------------------------------------------------------ attention

def filled(c, lens, g, k_scale=1.0, v_scale=1.0):
    """Random tokens in the cache; what the cache then holds, fp64 per sequence."""
    n = sum(lens)
    k, v = bf((max(n, 1), c.h_kv, c.d_k), g, k_scale), bf((max(n, 1), c.h_kv, c.d_v), g, v_scale)
    if n:
        c.append(k.to(DEV), v.to(DEV), i32(lens), cu_seqlens=cu_of(lens))
    held, r = [], 0
    for L in lens:
        kk, vv = k[r:r + L], v[r:r + L]
        if c.fmt == "int4":
            sv = co.quantise(vv.unflatten(-1, (-1, 32)))[1].double().repeat_interleave(32, -1) * 8
            held.append((co.through_4_bits(kk), co.through_4_bits(vv), sv))
        else:
            held.append((kk.double(), vv.double(), vv.double().abs()))
        r += L
    return held


def check_attention(out, lse, q, held, lens, *, scale=0.0, softcap=0.0, slopes=None, window=0, seen=None):
    out, q = out.cpu().double(), q.cpu()
    for b, L in enumerate(lens):
        k, v, unit = held[b]
        kw = dict(scale=scale, softcap=softcap, slopes=slopes, window=window, seen=None if seen is None else seen[b])
        ref, ref_lse, mag = co.attend(q[b], k, v, **kw)
        _, _, mag8 = co.attend(q[b], k, unit, **kw)
        sc = scale or 1 / math.sqrt(k.shape[-1])
        G = q.shape[2] // k.shape[1]
        raw = 0.0
        if L:   # the largest scale sum |q||k| of any score
            raw = float(torch.einsum("nhgd,uhd->nhgu", q[b].double().abs().unflatten(1, (k.shape[1], G)), k.abs()).max()) * sc
        reach = L if not window else min(L, window)
        e = raw * 2 ** -17 + 2 ** -20 * (min(softcap, raw) + (float(slopes.abs().max()) * reach if slopes is not None else 0)) + 1e-5
        bound = ref.abs() * 2 ** -8 + mag8 * 2 ** -8 + 2 * e * mag + 1e-30
        diff = (out[b] - ref).abs()
        assert (diff <= bound * 1.01).all(), (b, L, float((diff / bound).max()))
        if lse is not None:
            got = lse[b].cpu().double()
            assert torch.equal(got == -math.inf, ref_lse == -math.inf)
            ok = ref_lse != -math.inf
            assert ((got - ref_lse).abs()[ok] <= e + ref_lse.abs()[ok] * 2 ** -20).all(), (b, L)


def run_attention(fmt, dk, dv, page, h_kv, G, lens, n_new, seed=0, max_len=None, k_scale=1.0, v_scale=1.0, q_scale=1.0, **kw):
    g = gen(seed)
    B, max_len = len(lens), max_len or max(max(lens), 1)
    c = shuffled(B, max_len, h_kv, dk, dv, fmt, page, seed)
    held = filled(c, lens, g, k_scale, v_scale)
    q = bf((B, n_new, h_kv * G, dk), g, q_scale).to(DEV)
    lse = torch.full((B, n_new, h_kv * G), math.nan, device=DEV)
    slopes = kw.pop("slopes", None)
    out = c.attend(q, i32(lens), kw.pop("max_seqlen", max(max(lens), 1)), lse=lse,
                   slopes=slopes.to(DEV) if slopes is not None else None, softmax_scale=kw.pop("scale", 0.0), **kw)
    assert c.device_status() == 0
    return c, q, held, out, lse, slopes


@pytest.mark.parametrize("fmt", ["bf16", "int4"])
@pytest.mark.parametrize("dk,dv", DIMS)
@pytest.mark.parametrize("G,n_new", [(1, 1), (16, 1), (7, 1), (3, 3), (2, 5), (16, 2), (5, 16), (16, 16)])
def test_attention_head_layouts(fmt, dk, dv, G, n_new):
    lens = [300, 0, 17, 129, 1] if n_new < 16 else [75, 9]
    _, q, held, out, lse, _ = run_attention(fmt, dk, dv, 48, 2, G, lens, n_new, seed=G * 100 + n_new)
    check_attention(out, lse, q, held, lens)


@pytest.mark.parametrize("fmt", ["bf16", "int4"])
@pytest.mark.parametrize("page,lens", [(16, [1, 2, 15, 16, 17, 31, 33]), (64, [128, 127, 129, 512, 513]), (256, [2000, 0, 1, 1025]),
                                       (4096, [4096, 4095, 1537])])
def test_attention_lengths(fmt, page, lens):
    _, q, held, out, lse, _ = run_attention(fmt, 128, 128, page, 1, 4, lens, 1, seed=page)
    check_attention(out, lse, q, held, lens)


@pytest.mark.parametrize("fmt", ["bf16", "int4"])
@pytest.mark.parametrize("window,n_new", [(1, 1), (1, 4), (15, 3), (16, 16), (100, 1), (128, 5), (700, 2)])
def test_attention_windows(fmt, window, n_new):
    lens = [700, 65, 3, 0, 128]
    _, q, held, out, lse, _ = run_attention(fmt, 64, 64, 16, 1, 4, lens, n_new, seed=window, window=window)
    check_attention(out, lse, q, held, lens, window=window)


@pytest.mark.parametrize("fmt", ["bf16", "int4"])
@pytest.mark.parametrize("cap,steep,scale", [(30.0, 0, 0.0), (0.5, 0, 0.0), (1e6, 0, 0.0), (0.0, 1, 0.0), (20.0, 1, 0.3), (0.0, 0, 1.0),
                                             (1e-3, 0, 0.0)])
def test_attention_caps_and_slopes(fmt, cap, steep, scale):
    lens = [450, 33, 4]
    slopes = torch.exp2(-torch.arange(1, 9).float()) * (1 - 2 * (torch.arange(8) % 2)) * 0.25 if steep else None
    _, q, held, out, lse, slopes = run_attention(fmt, 128, 128, 48, 2, 4, lens, 3, seed=9, softcap=cap, slopes=slopes, scale=scale)
    check_attention(out, lse, q, held, lens, softcap=cap, slopes=slopes, scale=scale)


@pytest.mark.parametrize("fmt", ["bf16", "int4"])
def test_options_at_the_ends_of_their_ranges(fmt):
    """Windows that reach everything are none; caps far above the scores change nothing, far below make them equal."""
    lens = [130, 20, 3, 0]
    c, q, held, out, lse, _ = run_attention(fmt, 64, 64, 16, 2, 2, lens, 5, seed=40)
    check_attention(out, lse, q, held, lens)
    for window in (130, 131, 2 ** 31 - 1):
        assert torch.equal(c.attend(q, i32(lens), 130, window=window), out)
    for cap in (1e32, 3e38):
        assert torch.equal(c.attend(q, i32(lens), 130, softcap=cap), out)
    for cap in (1e-30, 1e-44):
        flat = c.attend(q, i32(lens), 130, softcap=cap)
        check_attention(flat, None, torch.zeros_like(q), held, lens)
    check_attention(c.attend(q, i32(lens), 130, softcap=1e20), None, q, held, lens)


@pytest.mark.parametrize("fmt", ["bf16", "int4"])
@pytest.mark.parametrize("odd", [math.nan, math.inf])
def test_a_query_that_is_not_finite_spoils_its_row_alone(fmt, odd):
    lens = [700, 40]
    c, q, _, out, _, _ = run_attention(fmt, 128, 128, 16, 2, 4, lens, 3, seed=41)
    q[0, 1, 3, 17] = odd
    again = c.attend(q, i32(lens), 700)
    assert torch.isnan(again[0, 1, 3].float()).all()
    same = torch.ones(out.shape[:3], dtype=torch.bool)
    same[0, 1, 3] = False
    assert torch.equal(again[same.to(DEV)], out[same.to(DEV)])


@pytest.mark.parametrize("fmt", ["bf16", "int4"])
@pytest.mark.parametrize("ks,vs,qs", [(1e-4, 1e3, 1.0), (30.0, 1.0, 1.0), (1.0, 1e-20, 1e3), (1e10, 1e20, 1e-10), (1.0, 1.0, 0.0)])
def test_attention_magnitudes(fmt, ks, vs, qs):
    """Small, large and lopsided inputs: weights from flat to one token taking all."""
    lens = [290, 40]
    _, q, held, out, lse, _ = run_attention(fmt, 192, 128, 64, 1, 16, lens, 1, seed=4, k_scale=ks, v_scale=vs, q_scale=qs)
    check_attention(out, lse, q, held, lens)


@pytest.mark.parametrize("fmt", ["bf16", "int4"])
def test_attention_many_sequences(fmt):
    """More sequences and heads than blocks fit at once, lengths all over the place."""
    g = gen(12)
    lens = torch.randint(0, 150, (150,), generator=g).tolist()
    lens[3], lens[149] = 900, 0
    _, q, held, out, lse, _ = run_attention(fmt, 64, 64, 16, 3, 2, lens, 1, seed=12)
    check_attention(out, lse, q, held, lens)


@pytest.mark.parametrize("fmt", ["bf16", "int4"])
def test_attention_long_sequence_beside_short_ones(fmt):
    lens = [40000, 0, 5, 1000]
    _, q, held, out, lse, _ = run_attention(fmt, 128, 128, 256, 1, 2, lens, 1, seed=13)
    check_attention(out, lse, q, held, lens)


@pytest.mark.parametrize("fmt", ["bf16", "int4"])
@pytest.mark.parametrize("B,h_kv,G,n_new,top,window,dk,dv", [
    (2, 1, 16, 16, 3000, 0, 192, 128),      # 256 rows a head: four row tiles, cut sequences
    (2, 1, 16, 16, 3000, 333, 128, 128),
    (3, 1, 8, 4, 2500, 0, 64, 64),          # 32 rows: two row groups
    (3, 2, 7, 5, 2500, 700, 64, 64),        # 35 rows: four row groups, the last ones partly empty
    (70, 1, 3, 1, 1100, 0, 64, 64),         # runs that end with their items
    (40, 8, 1, 1, 3000, 0, 64, 64),         # runs that do not
    (20, 16, 2, 1, 6000, 2000, 64, 64),
])
def test_attention_cut_over_blocks(fmt, B, h_kv, G, n_new, top, window, dk, dv):
    """Work that is shared out over blocks in runs, with empty and short sequences between the long ones."""
    g = gen(B + top)
    lens = torch.randint(0, top + 1, (B,), generator=g).tolist()
    lens[0], lens[-1] = top, top - 1
    if B > 3:
        lens[1], lens[2] = 0, 1
    _, q, held, out, lse, _ = run_attention(fmt, dk, dv, 16, h_kv, G, lens, n_new, seed=B, window=window)
    picks = list(range(B)) if B < 5 else [0, 1, 2, B // 2, B - 2, B - 1]
    check_attention(out[picks], lse[picks], q[picks], [held[b] for b in picks], [lens[b] for b in picks], window=window)
    assert torch.isfinite(out.float()).all() and not torch.isnan(lse).any()


@pytest.mark.parametrize("shape", ["rising", "falling", "offset", "mixed"])
def test_four_bit_values_of_changing_scales(shape):
    """A warp's long run over values whose scales grow or shrink by tokens and groups, or whose offsets dwarf
    their spans, with weights from flat to steep: the accumulators' common factors have to follow."""
    g = gen(30)
    B, h_kv, L, d = 80, 8, 3000, 128
    k, v = bf((L, 1, d), g), bf((L, 1, d), g)
    f = torch.arange(L).float()[:, None, None]
    if shape == "rising":
        v = (v.float() * torch.exp2(f * (16 / L))).bfloat16()
    elif shape == "falling":
        v = (v.float() * torch.exp2(-f * (16 / L))).bfloat16()
    elif shape == "offset":
        v = (v.float() * 0.02 + 30.0).bfloat16()
    else:
        v = (v.float() * torch.tensor([1e-20, 1.0, 1e20, 1e5]).repeat_interleave(32)).bfloat16()
    c = KVCache(B, L, h_kv, d, d, fmt="int4", page_size=64, device=DEV)
    kk, vv = (x.to(DEV).expand(L, h_kv, d).contiguous() for x in (k, v))
    for b in range(B):
        c.append(kk, vv, i32([L] * B), cu_seqlens=i32([0] * (b + 1) + [L] * (B - b)))
    q = bf((1, 1, h_kv, d), g).to(DEV).expand(B, 1, h_kv, d).contiguous()
    out = c.attend(q, i32([L] * B), L)
    assert c.device_status() == 0
    unit = co.quantise(v.unflatten(-1, (-1, 32)))[1].double().repeat_interleave(32, -1) * 8
    held = [tuple(x.expand(L, h_kv, d) for x in (co.through_4_bits(k), co.through_4_bits(v), unit))]
    for b in (0, 37, B - 1):
        check_attention(out[b:b + 1], None, q[b:b + 1], held, [L])


@pytest.mark.parametrize("fmt", ["bf16", "int4"])
def test_attention_bound_above_lengths_and_repeats(fmt):
    """max_seqlen is only a bound, and the same call gives the same bits, workspace dirty or not."""
    lens = [900, 33, 0, 412]
    c, q, held, out, lse, _ = run_attention(fmt, 128, 128, 16, 2, 8, lens, 2, seed=14, max_len=5000)
    check_attention(out, lse, q, held, lens)
    for bound in (900, 901, 2048, 5000):
        need = c.attend_workspace(2, 16, bound)
        ws = torch.full((need + 256,), 255, dtype=torch.uint8, device=DEV)     # NaNs wherever it is read unset
        a = c.attend(q, i32(lens), bound, workspace=ws)
        check_attention(a, None, q, held, lens)
        for _ in range(3):
            assert torch.equal(c.attend(q, i32(lens), bound), a)
        if bound == 900:
            assert torch.equal(a, out)


@pytest.mark.parametrize("fmt", ["bf16", "int4"])
def test_what_no_query_attends_never_matters(fmt):
    """NaN and infinities in places behind the lengths, before the window and in foreign pages."""
    g = gen(15)
    lens, window = [333, 70, 1], 50
    c, q, held, out, lse, _ = run_attention(fmt, 128, 128, 16, 1, 4, lens, 2, seed=15, window=window)
    check_attention(out, lse, q, held, lens, window=window)
    want = out.clone()
    keep = torch.zeros((c.k.shape[0], c.page_size), dtype=torch.bool)
    for b, L in enumerate(lens):
        for p in range(max(0, L - 2 - window + 1), L):
            keep[int(c.page_table[b, p // 16]), p % 16] = True
    for t in pools(c):
        m = (~keep).to(DEV)
        if fmt == "int4":
            m = m[:, None, :].expand(t.shape[:3])
        bits(t)[m] = 255                                   # bf16: NaN; codes: 15
    assert torch.equal(c.attend(q, i32(lens), 333, window=window), want)
    for val in (math.inf, -math.inf):
        for t in pools(c):
            if t.dtype == torch.bfloat16:
                m = (~keep).to(DEV)
                t[m[:, None, :].expand(t.shape[:3]) if fmt == "int4" else m] = val
        assert torch.equal(c.attend(q, i32(lens), 333, window=window), want)


@pytest.mark.parametrize("fmt", ["bf16", "int4"])
def test_attended_nan_shows(fmt):
    lens = [200, 40]
    c, q, held, out, _, _ = run_attention(fmt, 64, 64, 16, 1, 2, lens, 1, seed=16)
    bad = torch.full((1, 1, 64), math.nan, dtype=torch.bfloat16, device=DEV)
    c.append(bad, bad, i32([150, 0]), cu_seqlens=i32([0, 1, 1]))
    again = c.attend(q, i32(lens), 200)
    assert torch.isnan(again[0].float()).all() and torch.equal(again[1], out[1])


@pytest.mark.parametrize("fmt", ["bf16", "int4"])
def test_attention_over_missing_pages(fmt):
    """Tokens on pages out of range are as if not there; lengths out of range are clamped."""
    lens = [100, 64, 30]
    c, q, held, out, lse, _ = run_attention(fmt, 64, 64, 16, 2, 2, lens, 1, seed=17)
    c.page_table[0, 2], c.page_table[0, 5], c.page_table[1] = -1, 2 ** 31 - 1, c.k.shape[0]
    seen = [torch.ones(L, dtype=torch.bool) for L in lens]
    seen[0][32:48] = seen[0][80:96] = False
    seen[1][:] = False
    out = c.attend(q, i32(lens), 100, lse=lse)
    assert c.device_status() == nsa.NSA_CODE_CACHE
    check_attention(out, lse, q, held, lens, seen=seen)
    assert not out[1].any() and (lse[1] == -math.inf).all()
    c, q, held, out, lse, _ = run_attention(fmt, 64, 64, 16, 2, 2, [48, 64, 30], 1, seed=17, max_len=64)
    clamped = c.attend(q, i32([-3, 100, 30]), 64, lse=lse)
    assert c.device_status() == nsa.NSA_CODE_CACHE
    assert not clamped[0].any() and torch.equal(clamped[1:], out[1:])


# ------------------------------------------------------------------ how they are called

def test_refusals_of_the_python_calls():
    c = KVCache(2, 64, 2, 64, 64, device=DEV)
    bfz = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device=DEV)
    ok = i32([1, 1])
    bad = [
        lambda: c.append(bfz(2, 1, 2, 64), bfz(2, 1, 2, 32), ok),
        lambda: c.append(bfz(2, 1, 2, 64).float(), bfz(2, 1, 2, 64), ok),
        lambda: c.append(bfz(2, 1, 2, 64), bfz(2, 2, 2, 64), ok),
        lambda: c.append(bfz(2, 1, 2, 64), bfz(2, 1, 2, 64), ok.long()),
        lambda: c.append(bfz(2, 1, 2, 64), bfz(2, 1, 2, 64), i32([1])),
        lambda: c.append(bfz(2, 1, 2, 64).cpu(), bfz(2, 1, 2, 64), ok),
        lambda: c.append(bfz(2, 1, 64, 2).transpose(2, 3), bfz(2, 1, 2, 64), ok),
        lambda: c.append(bfz(2, 1, 2, 64), bfz(2, 1, 2, 64), ok, q=bfz(2, 2, 2, 64)),
        lambda: c.append(bfz(2, 1, 2, 64), bfz(2, 1, 2, 64), ok, q=bfz(2, 1, 2, 64), q_out=bfz(2, 1, 4, 64)),
        lambda: c.append(bfz(2, 1, 2, 64), bfz(2, 1, 2, 64), ok, cos_sin=torch.zeros(4, 64, dtype=torch.float64, device=DEV)),
        lambda: c.append(bfz(2, 1, 2, 64), bfz(2, 1, 2, 64), ok, cu_seqlens=i32([0, 1, 2])),
        lambda: c.read(ok), lambda: c.read(ok, cu_seqlens=i32([0, 1, 2])), lambda: c.read(ok, -1),
        lambda: c.read(ok, 1, k_out=bfz(2, 1, 2, 32)),
        lambda: c.attend(bfz(2, 1, 2, 32), ok), lambda: c.attend(bfz(1, 1, 2, 64), ok), lambda: c.attend(bfz(2, 0, 2, 64), ok),
        lambda: c.attend(bfz(2, 1, 4, 64)[:, :, ::2], ok), lambda: c.attend(bfz(2, 1, 2, 64).float(), ok),
        lambda: c.attend(bfz(2, 1, 2, 64), ok, slopes=torch.zeros(3, device=DEV)),
        lambda: c.attend(bfz(2, 1, 2, 64), ok, lse=torch.zeros(2, 2, device=DEV)),
        lambda: c.attend(bfz(2, 1, 2, 64), ok, out=bfz(2, 1, 2, 32)),
        lambda: c.attend(bfz(2, 1, 2, 64), ok, workspace=torch.zeros(1 << 20, dtype=torch.uint8)),
    ]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    refused = [
        lambda: c.attend(bfz(2, 1, 3, 64), ok), lambda: c.attend(bfz(2, 17, 2, 64), ok), lambda: c.attend(bfz(2, 1, 34, 64), ok),
        lambda: c.attend(bfz(2, 1, 2, 64), ok, 65), lambda: c.attend(bfz(2, 1, 2, 64), ok, window=-1),
        lambda: c.attend(bfz(2, 1, 2, 64), ok, softcap=-1.0),
        lambda: c.append(bfz(2, 1, 2, 64), bfz(2, 1, 2, 64), ok, cos_sin=torch.zeros(4, 8, device=DEV)),
    ]
    for call in refused:
        with pytest.raises(nsa.NsaError):
            call()
    # nothing to do is not an error
    assert c.append(bfz(2, 0, 2, 64), bfz(2, 0, 2, 64), ok) is None
    k, v = c.read(ok, 0)
    assert k.shape == v.shape == (2, 0, 2, 64)
    assert c.device_status() == 0


def test_strides_of_new_rows():
    """A batch whose rows lie apart by token (one new token, sequences far apart; heads one)."""
    g = gen(20)
    big = bf((3, 5, 4, 64), g).to(DEV)
    lens = i32([4, 9, 1])
    a, b = (KVCache(3, 16, 4, 64, 64, page_size=16, device=DEV) for _ in range(2))
    a.append(big[:, 2:3], big[:, 4:5], lens, q=big[:, 0:1])
    b.append(big[:, 2:3].contiguous(), big[:, 4:5].contiguous(), lens)
    assert torch.equal(a.k, b.k) and torch.equal(a.v, b.v)
    one = KVCache(3, 16, 1, 64, 64, page_size=16, device=DEV)
    with pytest.raises(ValueError):
        one.append(big[:, :2, 1:2], big[:, 1:3, 3:4], lens)     # sequences at another stride than tokens


@pytest.mark.parametrize("fmt", ["bf16", "int4"])
def test_graph_replays_decode_steps(fmt):
    """Append and attention of a step captured once, replayed while the lengths grow; two graphs of
    two layers share one workspace; the results are those of eager calls."""
    g = gen(21)
    B, h_kv, G, d, steps = 3, 2, 4, 128, 5
    start = [500, 16, 0]
    cs = table(600, d).to(DEV)

    def layer():
        c = KVCache(B, 600, h_kv, d, d, fmt=fmt, page_size=16, device=DEV)
        return c

    pre = bf((sum(start), h_kv, d), g).to(DEV)
    layers = [layer(), layer()]
    eager = [layer(), layer()]
    for c in layers + eager:
        c.append(pre, pre, i32(start), cu_seqlens=cu_of(start), cos_sin=cs)
    lens = i32(start)
    qkv = torch.zeros((B, 1, (h_kv * G + 2 * h_kv) * d), dtype=torch.bfloat16, device=DEV)
    split = lambda x: [t.unflatten(-1, (-1, d)) for t in x.split([h_kv * G * d, h_kv * d, h_kv * d], -1)]
    ws = torch.empty(max(c.attend_workspace(1, h_kv * G, 600) for c in layers), dtype=torch.uint8, device=DEV)

    def step(c, workspace=None):
        q, k, v = split(qkv)
        q = c.append(k, v, lens, cos_sin=cs, q=q)
        return c.attend(q, lens, 600, workspace=workspace, window=200)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):        # lengths 0 new tokens yet: the warm-up writes the last tokens again
        for c in layers:
            step(c, ws)
    torch.cuda.current_stream().wait_stream(side)
    for c in layers:
        c.append(pre, pre, i32(start), cu_seqlens=cu_of(start), cos_sin=cs)
    graphs, outs = [], []
    for c in layers:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(step(c, ws))
        graphs.append(gr)
    for s in range(steps):
        lens += 1
        qkv.copy_(bf(qkv.shape, g))
        for i in range(2):
            graphs[i].replay()
            assert torch.equal(step(eager[i]), outs[i]), (s, i)
    assert all(c.device_status() == 0 for c in layers + eager)


def test_calls_on_other_streams():
    """Two caches worked on at once on two streams, given as objects and as handles."""
    lens = [2000, 100]
    one = run_attention("int4", 128, 128, 64, 2, 4, lens, 1, seed=22)
    two = run_attention("bf16", 64, 64, 16, 1, 8, lens, 2, seed=23)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    lens_d = i32(lens)
    torch.cuda.synchronize()
    for _ in range(10):
        for i, (c, q, *_r) in enumerate((one, two)):
            s = streams[i]
            got[i].append(c.attend(q, lens_d, 2000, stream=s if len(got[i]) % 2 else s.cuda_stream))
    torch.cuda.synchronize()
    for i, run in enumerate((one, two)):
        assert all(torch.equal(x, run[3]) for x in got[i])


@pytest.mark.parametrize("fmt", ["bf16", "int4"])
def test_far_pages(fmt):
    """Pages whose offsets pass 2^32 bytes and 2^32 elements: the pool is larger, three pages are used."""
    d, h_kv, page = 128, 8, 256
    per_page = page * h_kv * d                             # elements of keys in a page
    n_pages = 2 ** 32 // per_page * (1 if fmt == "bf16" else 2) + 4
    c = KVCache(1, 3 * page, h_kv, d, d, fmt=fmt, page_size=page, n_pages=n_pages, device=DEV)
    c.page_table.copy_(i32([[n_pages - 1, 0, n_pages // 2 + 1]]))
    near = KVCache(1, 3 * page, h_kv, d, d, fmt=fmt, page_size=page, device=DEV)
    g = gen(24)
    L = 3 * page - 5
    k, v, q = bf((L, h_kv, d), g).to(DEV), bf((L, h_kv, d), g).to(DEV), bf((1, 2, 16, d), g).to(DEV)
    res = []
    for x in (c, near):
        x.append(k, v, i32([L]), cu_seqlens=i32([0, L]))
        res.append((x.attend(q, i32([L]), L), *x.read(i32([L]), L)))
        assert x.device_status() == 0
    assert all(torch.equal(a, b) for a, b in zip(*res))


def test_contiguous_caches_of_decode_as_pools():
    """nsa_decode's [B, L_max, h_kv, d] caches are pools as they stand, whatever L_max is."""
    g = gen(25)
    B, L_max, h_kv, d = 2, 83, 2, 64
    k, v = bf((B, L_max, h_kv, d), g), bf((B, L_max, h_kv, d), g)
    c = KVCache.from_pools(k.to(DEV), v.to(DEV), i32([[0], [1]]))
    lens = [83, 50]
    q = bf((B, 2, 8, d), g).to(DEV)
    out = c.attend(q, i32(lens))
    held = [(k[b, :L].double(), v[b, :L].double(), v[b, :L].double().abs()) for b, L in enumerate(lens)]
    check_attention(out, None, q, held, lens)
    new = bf((B, 1, h_kv, d), g).to(DEV)
    c.append(new, new, i32([83, 51]))
    assert torch.equal(c.k[0, 82], new[0, 0]) and torch.equal(c.v[1, 50], new[1, 0])
    ko, vo = c.read(i32([83, 51]), 83)
    assert torch.equal(ko[0], c.k[0]) and torch.equal(vo[1, 32:], c.v[1, :51]) and not vo[1, :32].any()


@pytest.mark.parametrize("fmt", ["bf16", "int4"])
def test_a_prompt_then_steps_then_its_compressed_blocks(fmt):
    """As a serving loop uses the calls: packed prompts, drafts of unequal lengths, single tokens; every
    step against the oracle on what was fed in; at the end the history goes to the block compression."""
    g = gen(26)
    B, h_kv, G, dk, dv, page = 3, 2, 4, 192, 128, 16
    c = shuffled(B, 200, h_kv, dk, dv, fmt, page, 26)
    c16 = shuffled(B, 200, h_kv, dk, dv, "bf16", page, 27)
    cs = table(200, 64).to(DEV)
    lens = [0, 0, 0]
    fed = [[] for _ in range(B)]     # (rotated keys as the bf16 cache holds them, values)
    for counts in ([120, 0, 33], [1, 1, 1], [3, 0, 2], [1, 1, 1]):
        n = sum(counts)
        lens = [a + b for a, b in zip(lens, counts)]
        q, k, v = bf((n, h_kv * G, dk), g).to(DEV), bf((n, h_kv, dk), g).to(DEV), bf((n, h_kv, dv), g).to(DEV)
        kw = dict(cu_seqlens=cu_of(counts), cos_sin=cs)
        q_rot = c.append(k, v, i32(lens), q=q, **kw)
        assert torch.equal(c16.append(k, v, i32(lens), q=q, **kw), q_rot)
        k16, v16 = (x.cpu() for x in c16.read(i32(lens), cu_seqlens=kw["cu_seqlens"], total=n))
        r = 0
        for b in range(B):
            fed[b].append((k16[r:r + counts[b]], v16[r:r + counts[b]]))
            r += counts[b]
        if max(counts) <= 3:         # the new tokens attend; unequal counts stand at the end of a padded row
            m = max(counts)
            qp = torch.zeros((B, m, h_kv * G, dk), dtype=torch.bfloat16, device=DEV)
            r = 0
            for b in range(B):
                if counts[b]:
                    qp[b, m - counts[b]:] = q_rot[r:r + counts[b]]
                r += counts[b]
            out = c.attend(qp, i32(lens), max(lens))
            held = []
            for b in range(B):
                kk, vv = (torch.cat(x) for x in zip(*fed[b]))
                if fmt == "int4":
                    unit = co.quantise(vv.unflatten(-1, (-1, 32)))[1].double().repeat_interleave(32, -1) * 8
                    held.append((co.through_4_bits(kk), co.through_4_bits(vv), unit))
                else:
                    held.append((kk.double(), vv.double(), vv.double().abs()))
            check_attention(out, None, qp, held, lens)
    hist, _ = c.read(i32(lens), lens[0])
    want = torch.cat([x for x, _ in fed[0]])
    want = co.through_4_bits(want).bfloat16() if fmt == "int4" else want
    assert torch.equal(hist[0].cpu(), want)
    w = bf((32 * dk, dk), g, 0.02)
    assert torch.equal(compress_torch(hist[:1], w.to(DEV)), compress_torch(want[None].to(DEV), w.to(DEV)))
    assert c.device_status() == 0
