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
