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
