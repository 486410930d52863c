"""The paged cache where a call can go wrong although the ordinary ones are right: other streams, values and
options at the ends of their ranges, the shapes that plain decoding takes, and errors below the outputs' own rounding."""
import math

import pytest
import torch

import block_sparse_attention_compress_b200 as nsa
from block_sparse_attention_compress_b200 import build
from block_sparse_attention_compress_b200.torch_ops import KVCache
from oracle import cache_oracle as co
from tests.test_gpu_cache import DEV, bf, check_attention, gen, i32, run_attention

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()


@pytest.mark.parametrize("handle", [False, True])
def test_memory_freed_behind_a_queue_of_another_stream_is_left_alone(handle):
    """A tensor of the workspace's size, freed while its kernels still wait on the current stream, and a call on another
    stream at once: neither sees the other's writes."""
    lens = [2000, 100]
    c, q, _, want, _, _ = run_attention("int4", 128, 128, 64, 2, 4, lens, 1, seed=50)
    lens_d, need = i32(lens), c.attend_workspace(1, 8, 2000)
    assert need > 0
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        torch.cuda._sleep(20_000_000)                    # ten milliseconds or so
        sums = []
        for shape, dtype in (((need,), torch.uint8), (tuple(want.shape), torch.bfloat16)):
            x = torch.full(shape, 7, dtype=dtype, device=DEV)
            sums.append((x == 7).sum())
            del x
        got = c.attend(q, lens_d, 2000, stream=side.cuda_stream if handle else side)
        side.synchronize()
        assert torch.equal(got, want)
        assert [int(s) for s in sums] == [need, want.numel()]
        torch.cuda.synchronize()


@pytest.mark.parametrize("fmt", ["bf16", "int4"])
@pytest.mark.parametrize("cap", [1e-30, 2e-39, 1e-44])
def test_the_smallest_caps_leave_zero_scores_alone(fmt, cap):
    """A query of zeros and a key of zeros score exactly 0, which any cap leaves at 0: equal weights, the mean of the values."""
    lens = [70, 20]
    g = gen(51)
    c = KVCache(2, 70, 1, 64, 64, fmt=fmt, page_size=16, device=DEV)
    k, v = bf((90, 1, 64), g), bf((90, 1, 64), g)
    k[5] = k[80] = 0
    c.append(k.to(DEV), v.to(DEV), i32(lens), cu_seqlens=i32([0, 70, 90]))
    kept = (lambda x: co.through_4_bits(x)) if fmt == "int4" else (lambda x: x.double())
    unit = co.quantise(v.unflatten(-1, (-1, 32)))[1].double().repeat_interleave(32, -1) * 8 if fmt == "int4" else v.double().abs()
    held = [(kept(k)[a:b], kept(v)[a:b], unit[a:b]) for a, b in ((0, 70), (70, 90))]
    q = bf((2, 2, 4, 64), g)
    q[0, 0] = q[1, 1, 2] = 0
    lse = torch.full((2, 2, 4), math.nan, device=DEV)
    out = c.attend(q.to(DEV), i32(lens), 70, softcap=cap, lse=lse)
    check_attention(out, lse, torch.zeros_like(q), held, lens)     # scores of 1e-30 and less: as if all were 0


def looped(fmt, L, h_kv, d, page_rows, per_page=256):
    """A cache of one sequence of L tokens whose pages are those of `page_rows` (lists of (k, v) [per_page, d] rows) over
    and over: long runs of a warp without their memory."""
    n = len(page_rows)
    c = KVCache(1, L, h_kv, d, d, fmt=fmt, page_size=per_page, n_pages=n, device=DEV)
    c.page_table.copy_((torch.arange(c.page_table.shape[1], device=DEV, dtype=torch.int32) % n)[None])
    k, v = (torch.cat(x)[:, None].expand(-1, h_kv, -1).contiguous().to(DEV) for x in zip(*page_rows))
    c.append(k, v, i32([n * per_page]), cu_seqlens=i32([0, n * per_page]))
    return c


@pytest.mark.parametrize("z", [29952.0, -1e20, 1e-20])
def test_long_runs_of_constant_values_stay_what_they_are(z):
    """Groups without a span (s = 0) over ten thousand and more tokens of a warp, equal weights: the value itself."""
    L, d = 14_000_000, 64
    v = torch.full((256, d), z).bfloat16()
    v[:, 32:] = torch.tensor(3.0)
    c = looped("int4", L, 1, d, [(torch.zeros(256, d).bfloat16(), v)])
    lse = torch.zeros((1, 1, 1), device=DEV)
    out = c.attend(torch.zeros((1, 1, 1, d), dtype=torch.bfloat16, device=DEV), i32([L]), L, lse=lse)
    assert c.device_status() == 0
    # weights of 1 and their sums in fp32: sums of up to 2^24 units are exact, the rest far below half a step of bf16
    assert torch.equal(out.cpu()[0, 0, 0], v[0])
    assert abs(float(lse) - math.log(L)) <= math.log(L) * 2 ** -20


def key_reach(fmt, q, k):
    """The largest scale sum |q||k| of q [h, d] over k [L, d]; 4 bits: |k| as the kernel adds it up, 15 s + |z - 8 s|."""
    k = k.double().abs()
    if fmt == "int4":
        _, s, z = co.quantise(k.bfloat16().unflatten(-1, (-1, 32)))
        k = (15 * s + (z - 8 * s).abs()).double().repeat_interleave(32, -1)
    return float((q.double().abs() @ k.T).max()) / math.sqrt(k.shape[-1])


@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (192, 128)])
@pytest.mark.parametrize("G,n", [(1, 1), (4, 1), (8, 1), (16, 1), (16, 4)])
@pytest.mark.parametrize("fmt", ["bf16", "int4"])
def test_weights_are_exact_far_below_the_outputs_rounding(fmt, dk, dv, G, n):
    """Values that almost cancel under the weights of the (equal) queries, so that the output's own rounding (2^-8 of little)
    hides nothing.  Allowed: weights of two terms, bf16 2^-18 each (2^-16 granted), f16 2^-22; a score's error e twice, with
    e = 16 roundings of 2^-23 or less of scale sum |q||k| and 2^-20 for the exponential; sums of few terms, 2^-20."""
    g = gen(60 + G + dk)
    L, h_kv = 5 + n, 2
    k, q = bf((L, h_kv, dk), g), bf((1, 1, 1, dk), g, 0.1).expand(1, n, h_kv * G, dk).contiguous()
    k[:, 1] = k[:, 0]
    v = bf((L, h_kv, dv), g)
    kept = (lambda x: co.through_4_bits(x)) if fmt == "int4" else (lambda x: x.double())
    kk = kept(k)
    x = kk[:, 0] @ q[0, 0, 0].double() / math.sqrt(dk)
    p = torch.exp(x - x.max())
    # the first token is seen by every query; what the others up to the first query's position weigh, it takes back
    seen = slice(1, L - n + 1)
    v[0] = (-(p[seen, None, None] * kept(v)[seen]).sum(0) / p[0]).bfloat16()
    v[L - n + 1:] = 0
    c = KVCache(1, L, h_kv, dk, dv, fmt=fmt, page_size=16, device=DEV)
    c.append(k.to(DEV), v.to(DEV), i32([L]), cu_seqlens=i32([0, L]))
    out = c.attend(q.to(DEV), i32([L]), L).cpu().double()[0]
    ref, _, mag = co.attend(q[0], kk, kept(v))
    e = key_reach(fmt, q[0, 0, :1], k[:, 0]) * 2 ** -19 + 2 ** -20
    unit = mag
    if fmt == "int4":
        s = co.quantise(v.unflatten(-1, (-1, 32)))[1].double().repeat_interleave(32, -1) * 8
        unit = co.attend(q[0], kk, s)[2] + mag
    bound = ref.abs() * 2 ** -8 + (2 ** -16 if fmt == "bf16" else 2 ** -20) * unit + (2 * e + 2 ** -20) * mag
    worst = float(((out - ref).abs() / bound).max())
    assert worst <= 1.01, worst


@pytest.mark.parametrize("fmt", ["bf16", "int4"])
@pytest.mark.parametrize("G,pages", [(1, 1024), (8, 1024), (16, 1024), (16, 1)])
def test_long_sums_do_not_drift(fmt, G, pages):
    """Equal weights over 60 million tokens (3,200 tiles a warp) whose values cancel exactly: `up` pages of positive values
    from 2^-12 to 1, then a page of the negatives of one of them times `up`, and so on until each of the `pages` different
    ones has come up as often as down.  A warp's sum of a dim climbs to A, about 256 up mean values, and falls again.

    Cut off, a sum or its addends lose up to a unit of the sum's last place (2^-23 A) at every tile, always towards zero.
    Rounded, a tile's error is at most half a unit either way: 2^-24 A / 16 a token whatever the tiles, 2^-15 (up = 32) or 2^-20
    (up = 1) mean values.  With the sum a multiple of its unit, that error is the tile's own wherever it comes, so those of T = 16
    pages different tiles average out: eight standard deviations, 8 2^-23 A / (16 sqrt(12 T)), with A 1.3 times as large as
    above for what is left over from one climb to the next: 2^-19.4 or 2^-24.4 for 1024 pages.  A step of one or two tiles
    (32 tokens) cut off at each of up to three products is less than 3 2^-23 32 / 32 = 2^-21.4."""
    g = gen(70)
    d, page, up = 64, 256, 32 if fmt == "bf16" else 1
    cycle = torch.arange(pages)
    climbs = (cycle[:, None] * up + torch.arange(up)) % pages
    order = torch.cat((climbs, cycle[:, None] + pages), 1).flatten().int()
    order = order.repeat(60_000_000 // (page * order.numel()))
    L = page * order.numel()
    c = KVCache(1, L, 1, d, d, fmt=fmt, page_size=page, n_pages=2 * pages, device=DEV)
    c.page_table.copy_(order[None])
    spread = lambda *shape: torch.exp2(-12 * torch.rand(shape, generator=g))
    if fmt == "bf16":
        v = spread(pages, page, 1, d).bfloat16()
        c.v.copy_(torch.cat((v, -up * v)))
        mean = v.double().mean((0, 1, 2))
    else:     # codes 1 .. 15 and 16 less them; s (c - 8) + z with z above 8 s, and z negated
        nib = torch.randint(1, 16, (pages, 1, page, d), generator=g, dtype=torch.uint8)
        s = spread(pages, 1, page, d // 32).bfloat16()
        z = (8.5 * s.float()).bfloat16()
        byte = lambda x: x[..., 0::2] | (x[..., 1::2] << 4)
        c.v.copy_(torch.cat((byte(nib), byte(16 - nib))))
        c.v_scale.copy_(torch.cat((torch.stack((s, z), -1), torch.stack((s, -z), -1))))
        _, back = c.read(i32([page]), page)
        assert (back > 0).all()
        mean = 8.5 * s.double().mean()
    out = c.attend(torch.zeros((1, 1, G, d), dtype=torch.bfloat16, device=DEV), i32([L]), L)
    assert c.device_status() == 0
    worst = float((out.cpu().double().abs() / mean).max())
    rounded = 2 ** -19.4 if up > 1 else 2 ** -24.4
    if pages == 1:
        rounded = 2 ** -15 if up > 1 else 2 ** -20
    assert worst <= rounded + 2 ** -21.4, math.log2(worst)


@pytest.mark.parametrize("fmt", ["bf16", "int4"])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (192, 128)])
@pytest.mark.parametrize("G,n", [(1, 1), (4, 1), (8, 1), (16, 1), (2, 2), (8, 3), (16, 2), (16, 4), (16, 16)])
@pytest.mark.parametrize("cap,sloped,window", [(20.0, True, 70), (0.7, False, 0), (0.0, True, 0)])
def test_options_in_every_shape(fmt, dk, dv, G, n, cap, sloped, window):
    """Caps, slopes and windows at once and alone, from one row a head (plain decoding) to 256, over short sequences and over
    one that is cut over blocks."""
    h_kv = 2 if G * n < 64 else 1
    lens = [300, 0, 17, 1200, 1] if G * n < 64 else [75, 900]
    h_q = h_kv * G
    slopes = torch.exp2(-8.0 * torch.arange(1, h_q + 1) / h_q) * (1 - 2 * (torch.arange(h_q) % 2)) * 0.05 if sloped else None
    _, q, held, out, lse, slopes = run_attention(fmt, dk, dv, 16, h_kv, G, lens, n, seed=80 + G, softcap=cap, slopes=slopes,
                                                 window=window, max_len=2048, max_seqlen=2048)
    check_attention(out, lse, q, held, lens, softcap=cap, slopes=slopes, window=window)


@pytest.mark.parametrize("size,shows", [(2.0 ** 100, False), (2.0 ** 110, False), (2.0 ** 120, True), (2.0 ** 127, True)])
def test_the_largest_queries_are_right_or_show(size, shows):
    """4 bits: the powers of two that take a row of queries into f16 leave fp32 for queries of 2^118 and more (d = 64).  Such a
    row is NaN, not a finite wrong result, and the other rows stay."""
    g = gen(90)
    lens, d = [40], 64
    k = (torch.randn((40, 1, 2), generator=g).repeat_interleave(32, -1) / size).bfloat16()      # groups without a span: exact
    v = bf((40, 1, d), g)
    c = KVCache(1, 40, 1, d, d, fmt="int4", page_size=16, device=DEV)
    c.append(k.to(DEV), v.to(DEV), i32(lens), cu_seqlens=i32([0, 40]))
    unit = co.quantise(v.unflatten(-1, (-1, 32)))[1].double().repeat_interleave(32, -1) * 8
    held = [(co.through_4_bits(k), co.through_4_bits(v), unit)]
    q = bf((1, 1, 4, d), g)
    q[0, 0, 1] = (q[0, 0, 1].float() * size / 4).bfloat16()
    q[0, 0, 1, 0] = size
    out = c.attend(q.to(DEV), i32(lens), 40)
    rows = [0, 2, 3] if shows else [0, 1, 2, 3]
    assert not shows or torch.isnan(out[0, 0, 1].float()).all()
    check_attention(out[:, :, rows], None, q[:, :, rows], held, lens)


@pytest.mark.parametrize("fmt", ["bf16", "int4"])
@pytest.mark.parametrize("odd", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("dk,dv,G,n,window", [(64, 64, 1, 4, 0), (128, 128, 2, 4, 50), (192, 128, 4, 4, 50), (128, 128, 8, 5, 0),
                                              (64, 64, 16, 4, 20), (128, 128, 16, 16, 100)])
def test_odd_values_reach_the_queries_that_attend_them_alone(fmt, odd, dk, dv, G, n, window):
    """A NaN or an infinity in a draft's value leaves the drafts before it alone, and one that has left a query's window that
    query; all that attend it show it."""
    lens = [700, n, 90]
    h_kv, h_q = 2, 2 * G
    c, q, _, want, want_lse, _ = run_attention(fmt, dk, dv, 16, h_kv, G, lens, n, seed=95, window=window)
    for b, i in ((0, n - 2), (2, 1), (1, n - 1), (0, 0)):           # the position of query i of sequence b
        where = lens[b] - n + i
        places = [where] if not window else [where, where - window + 1]
        for u in places:
            if u < 0:
                continue
            page, off = int(c.page_table[b, u // 16]), u % 16
            pool = c.v if fmt == "bf16" else c.v_scale
            at = (page, off, 1) if fmt == "bf16" else (page, 1, off)
            kept = pool[at].clone()
            pool[at + ((dv - 3,) if fmt == "bf16" else (dv // 32 - 1, 1))] = odd
            lse = torch.full_like(want_lse, 7.0)
            out = c.attend(q, i32(lens), max(lens), window=window, lse=lse)
            pool[at] = kept
            meets = torch.zeros((len(lens), n, h_q), dtype=torch.bool)
            for j in range(n):
                p = lens[b] - n + j
                if u <= p and (not window or u > p - window):
                    meets[b, j, G:] = True
            got = ~torch.isfinite(out.float()).all(-1).cpu()     # an infinity times a weight is one, or NaN with its second term
            assert torch.equal(got, meets), (b, i, u)
            assert torch.equal(out[~meets.to(DEV)], want[~meets.to(DEV)])
            assert torch.equal(lse, want_lse)
    assert c.device_status() == 0
