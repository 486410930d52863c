"""The paged cache on the CPU: its structs match the header, the C entries refuse what they must
before anything is launched, and the oracle is pinned by closed forms and brute force."""
import ctypes
import math
import os
import subprocess
import tempfile

import pytest
import torch

import block_sparse_attention_compress_b200 as nsa
from oracle import cache_oracle as co
from tests.test_abi import ROOT, made_up_pointers


@pytest.fixture(scope="module")
def lib():
    from block_sparse_attention_compress_b200 import build
    build.build()
    return nsa.load_library()


@pytest.mark.parametrize("c_name,mirror", [("nsa_cache", nsa.NsaCache),
                                           ("nsa_cache_append_args", nsa.NsaCacheAppendArgs),
                                           ("nsa_cache_attention_args", nsa.NsaCacheAttentionArgs)])
def test_struct_layouts_match_header(c_name, mirror):
    fields = [n for n, _ in mirror._fields_]
    src = "#include <stddef.h>\n#include <stdio.h>\n#include \"nsa.h\"\nint main(void) {\n" + \
        f'printf("%zu", sizeof({c_name}));\n' + \
        "".join(f'printf(" %zu", offsetof({c_name}, {n}));\n' for n in fields) + "return 0;\n}\n"
    with tempfile.TemporaryDirectory() as d:
        c = os.path.join(d, "l.c")
        open(c, "w").write(src)
        subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), c, "-o", os.path.join(d, "l")], check=True)
        got = subprocess.run([os.path.join(d, "l")], capture_output=True, text=True, check=True).stdout.split()
    assert [int(x) for x in got] == [ctypes.sizeof(mirror)] + [getattr(mirror, n).offset for n in fields]


def _cache(**kw):
    base = dict(format=nsa.NSA_CACHE_INT4, batch=2, h_kv=2, d_k=128, d_v=128, page_size=64, n_pages=8, max_pages=4,
                k=0x10000, v=0x20000, k_scale=0x30000, v_scale=0x40000, page_table=0x50000, status=0x60000)
    base.update(kw)
    return nsa.NsaCache(**base)


def _append(**kw):
    base = dict(k=0x100000, v=0x200000, seqlens=0x300000, k_stride=256, v_stride=256, n_new=1, cos_sin=0x400000,
                n_positions=256, rot_dim=128)
    base.update(kw)
    return nsa.NsaCacheAppendArgs(**base)


def _attn(**kw):
    base = dict(seqlens=0x300000, n_new=1, h_q=8, max_seqlen=256, workspace=0x10000000, workspace_bytes=1 << 30)
    base.update(kw)
    return nsa.NsaCacheAttentionArgs(**base)


BAD_CACHES = [
    (dict(format=2), nsa.NSA_ERR_INVALID_ARG),
    (dict(batch=0), nsa.NSA_ERR_INVALID_ARG),
    (dict(n_pages=0), nsa.NSA_ERR_INVALID_ARG),
    (dict(max_pages=0), nsa.NSA_ERR_INVALID_ARG),
    (dict(page_size=0), nsa.NSA_ERR_INVALID_ARG),
    (dict(k=0), nsa.NSA_ERR_INVALID_ARG),
    (dict(v=0x20008), nsa.NSA_ERR_INVALID_ARG),
    (dict(k_scale=0), nsa.NSA_ERR_INVALID_ARG),
    (dict(v_scale=0x40004), nsa.NSA_ERR_INVALID_ARG),
    (dict(page_table=0), nsa.NSA_ERR_INVALID_ARG),
    (dict(page_table=0x50002), nsa.NSA_ERR_INVALID_ARG),
    (dict(status=0x60001), nsa.NSA_ERR_INVALID_ARG),
    (dict(d_k=96), nsa.NSA_ERR_UNSUPPORTED),
    (dict(d_k=64), nsa.NSA_ERR_UNSUPPORTED),          # (64, 128) is no head layout
    (dict(page_size=40), nsa.NSA_ERR_UNSUPPORTED),    # several pages: multiples of 16
    (dict(page_size=40, max_pages=1), nsa.NSA_ERR_UNSUPPORTED),   # and always in 4 bits
    (dict(batch=65536), nsa.NSA_ERR_UNSUPPORTED),
    (dict(page_size=1 << 20, max_pages=1 << 11), nsa.NSA_ERR_UNSUPPORTED),
]


@made_up_pointers
@pytest.mark.parametrize("kw,status", BAD_CACHES)
def test_bad_caches_are_refused_by_every_entry(lib, kw, status):
    c = _cache(**kw)
    assert nsa.nsa_cache_append(c, _append(), stream=0, check=False) == status
    assert nsa.nsa_cache_read(c, 0x300000, None, 1, 0, 0x700000, 0x800000, stream=0, check=False) == status
    assert nsa.nsa_cache_attention(c, 0x700000, _attn(max_seqlen=1), 0x800000, stream=0, check=False) == status


@made_up_pointers
@pytest.mark.parametrize("kw,status", [
    (dict(k=0), nsa.NSA_ERR_INVALID_ARG), (dict(v=0x200008), nsa.NSA_ERR_INVALID_ARG),
    (dict(seqlens=0), nsa.NSA_ERR_INVALID_ARG), (dict(seqlens=0x300002), nsa.NSA_ERR_INVALID_ARG),
    (dict(n_new=0), nsa.NSA_ERR_INVALID_ARG), (dict(n_new=-1), nsa.NSA_ERR_INVALID_ARG),
    (dict(cu_seqlens=0x310000, total_tokens=0), nsa.NSA_ERR_INVALID_ARG),
    (dict(cu_seqlens=0x310002, total_tokens=1), nsa.NSA_ERR_INVALID_ARG),
    (dict(k_stride=248), nsa.NSA_ERR_INVALID_ARG),     # tokens would overlap
    (dict(v_stride=260), nsa.NSA_ERR_INVALID_ARG),     # rows off the 16-byte grid
    (dict(cos_sin=0x400004), nsa.NSA_ERR_INVALID_ARG), (dict(n_positions=0), nsa.NSA_ERR_INVALID_ARG),
    (dict(rot_dim=8), nsa.NSA_ERR_INVALID_ARG), (dict(rot_dim=40), nsa.NSA_ERR_INVALID_ARG),
    (dict(rot_dim=144), nsa.NSA_ERR_INVALID_ARG), (dict(interleaved=2), nsa.NSA_ERR_INVALID_ARG),
    (dict(q=0x500000), nsa.NSA_ERR_INVALID_ARG),       # queries without a place for them
    (dict(q_out=0x500000), nsa.NSA_ERR_INVALID_ARG),
    (dict(q=0x500000, q_out=0x600000, h_q=0, q_stride=256), nsa.NSA_ERR_INVALID_ARG),
    (dict(q=0x500000, q_out=0x600008, h_q=2, q_stride=256), nsa.NSA_ERR_INVALID_ARG),
    (dict(q=0x500000, q_out=0x600000, h_q=4, q_stride=256), nsa.NSA_ERR_INVALID_ARG),
    (dict(n_new=1 << 30), nsa.NSA_ERR_UNSUPPORTED),    # 2^31 rows
])
def test_bad_appends_are_refused(lib, kw, status):
    assert nsa.nsa_cache_append(_cache(), _append(**kw), stream=0, check=False) == status


@made_up_pointers
@pytest.mark.parametrize("args,status", [
    ((0, None, 1, 0, 0x700000, 0x800000), nsa.NSA_ERR_INVALID_ARG),
    ((0x300000, None, 0, 0, 0x700000, 0x800000), nsa.NSA_ERR_INVALID_ARG),
    ((0x300000, 0x310000, 1, 0, 0x700000, 0x800000), nsa.NSA_ERR_INVALID_ARG),
    ((0x300000, None, 1, 0, 0, 0x800000), nsa.NSA_ERR_INVALID_ARG),
    ((0x300000, None, 1, 0, 0x700000, 0x800004), nsa.NSA_ERR_INVALID_ARG),
    ((0x300000, None, 1 << 30, 0, 0x700000, 0x800000), nsa.NSA_ERR_UNSUPPORTED),
])
def test_bad_reads_are_refused(lib, args, status):
    assert nsa.nsa_cache_read(_cache(), *args, stream=0, check=False) == status


@made_up_pointers
@pytest.mark.parametrize("kw,status", [
    (dict(seqlens=0), nsa.NSA_ERR_INVALID_ARG), (dict(seqlens=0x300001), nsa.NSA_ERR_INVALID_ARG),
    (dict(n_new=0), nsa.NSA_ERR_INVALID_ARG), (dict(h_q=3), nsa.NSA_ERR_INVALID_ARG),
    (dict(max_seqlen=0), nsa.NSA_ERR_INVALID_ARG), (dict(max_seqlen=257), nsa.NSA_ERR_INVALID_ARG),
    (dict(window=-1), nsa.NSA_ERR_INVALID_ARG), (dict(softcap=-1.0), nsa.NSA_ERR_INVALID_ARG),
    (dict(softcap=math.nan), nsa.NSA_ERR_INVALID_ARG), (dict(softcap=math.inf), nsa.NSA_ERR_INVALID_ARG),
    (dict(softmax_scale=-1.0), nsa.NSA_ERR_INVALID_ARG), (dict(softmax_scale=math.inf), nsa.NSA_ERR_INVALID_ARG),
    (dict(slopes=0x900002), nsa.NSA_ERR_INVALID_ARG), (dict(lse=0x900002), nsa.NSA_ERR_INVALID_ARG),
    (dict(n_new=17), nsa.NSA_ERR_UNSUPPORTED), (dict(h_q=34), nsa.NSA_ERR_UNSUPPORTED),
    (dict(workspace=0, max_seqlen=1024), nsa.NSA_ERR_WORKSPACE),
    (dict(workspace=0x10000010, max_seqlen=1024), nsa.NSA_ERR_WORKSPACE),
    (dict(workspace_bytes=16, max_seqlen=1024), nsa.NSA_ERR_WORKSPACE),
])
def test_bad_attention_calls_are_refused(lib, kw, status):
    cache = _cache(max_pages=16 if kw.get("max_seqlen") == 1024 else 4)
    assert nsa.nsa_cache_attention(cache, 0x700000, _attn(**kw), 0x800000, stream=0, check=False) == status
    for q, out in ((0, 0x800000), (0x700008, 0x800000), (0x700000, 0), (0x700000, 0x800008)):
        assert nsa.nsa_cache_attention(_cache(), q, _attn(), out, stream=0, check=False) == nsa.NSA_ERR_INVALID_ARG


def test_attention_workspace_size(lib):
    # short sequences need none; a long one two parts of every row for each block that shares it
    assert nsa.nsa_cache_attention_workspace(_cache(batch=1), _attn(max_seqlen=16)) == 0
    need = nsa.nsa_cache_attention_workspace(_cache(batch=1, max_pages=1024, n_pages=1024), _attn(max_seqlen=65536))
    assert need > 0 and need % 16 == 0
    wider = nsa.nsa_cache_attention_workspace(_cache(batch=64, max_pages=1024, n_pages=1024), _attn(max_seqlen=65536))
    assert need <= wider < 64 * need        # the blocks of a call are bounded
    assert nsa.nsa_cache_attention_workspace(_cache(batch=0), _attn()) == 0
    assert nsa.nsa_cache_attention_workspace(_cache(), _attn(h_q=3)) == 0


def test_kvcache_wants_a_gpu_and_sane_sizes():
    from block_sparse_attention_compress_b200.torch_ops import KVCache
    with pytest.raises(ValueError):
        KVCache(1, 64, 1, 64, 64, fmt="fp8", device="cpu")
    with pytest.raises(ValueError):
        KVCache(0, 64, 1, 64, 64, device="cpu")
    with pytest.raises(ValueError):
        KVCache(1, 64, 1, 64, 64, device="cpu")


def test_memory_for_a_given_stream_is_that_streams(monkeypatch):
    """Outputs and workspaces of a call on a stream are allocated with that stream current, so that their memory
    cannot be a block that work queued on another stream still uses."""
    from block_sparse_attention_compress_b200.torch_ops import KVCache
    current, seen = [], []

    class Current:
        def __init__(self, stream):
            self.stream = stream

        def __enter__(self):
            current.append(self.stream)

        def __exit__(self, *exc):
            current.pop()

    class Like:
        shape, dtype, device = (2, 3), torch.bfloat16, torch.device("cpu")

        def new_empty(self, shape, dtype):
            seen.append(current[-1] if current else None)
            return torch.empty(shape, dtype=dtype)

    monkeypatch.setattr(torch.cuda, "stream", Current)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: ("external", handle))
    cache = KVCache.__new__(KVCache)
    cache.device = torch.device("cpu")
    mine = object()
    for stream, want in ((mine, mine), (77, ("external", 77)), (0, ("external", 0)), (None, None)):
        cache._new(Like(), (4, 5), stream)
        assert seen.pop() == want
    cache._new(Like(), (2, 3), mine)      # of the same shape as well
    assert seen.pop() is mine


def _on_cpu(batch=1, max_pages=4, page_size=16, h_kv=1, d=64):
    """A KVCache over CPU memory: everything up to the library's entries works on it."""
    from block_sparse_attention_compress_b200.torch_ops import KVCache
    c = KVCache.__new__(KVCache)
    c.fmt, c.batch, c.h_kv, c.d_k, c.d_v, c.page_size, c.device = "bf16", batch, h_kv, d, d, page_size, torch.device("cpu")
    c.desc = nsa.NsaCache(format=nsa.NSA_CACHE_BF16, batch=batch, h_kv=h_kv, d_k=d, d_v=d, page_size=page_size,
                          n_pages=batch * max_pages, max_pages=max_pages)
    c._lib, c._ref, c._workspaces = nsa.load_library(), ctypes.byref(c.desc), {}
    return c


@pytest.mark.parametrize("kw", [dict(max_seqlen=2 ** 32 + 5), dict(max_seqlen=2 ** 31), dict(window=2 ** 32 + 100),
                                dict(window=2 ** 31), dict(window=-2 ** 32 + 7)])
def test_integers_beyond_32_bits_are_refused(lib, kw):
    """ctypes would keep their low 32 bits: 2^32 + 5 would pass as 5."""
    c = _on_cpu()
    q, lens = torch.zeros((1, 1, 1, 64), dtype=torch.bfloat16), torch.ones(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="2\\^31"):
        c.attend(q, lens, **kw)
    with pytest.raises(ValueError, match="2\\^31"):
        c.attend_workspace(1, 1, **kw)


def test_row_counts_beyond_32_bits_are_refused(lib):
    c = _on_cpu()
    lens, cu = torch.ones(1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    for n in (2 ** 31, 2 ** 32 + 1):
        with pytest.raises(ValueError, match="2\\^31"):
            c.read(lens, n)
        with pytest.raises(ValueError, match="2\\^31"):
            c.read(lens, cu_seqlens=cu, total=n)
        with pytest.raises(ValueError, match="2\\^31"):
            c.attend_workspace(n, 1)
        with pytest.raises(ValueError, match="2\\^31"):
            c.attend_workspace(1, n)
        with pytest.raises(ValueError, match="2\\^31"):
            nsa.nsa_cache_read(c.desc, 0, None, n, 0, 0, 0, stream=0)
    from block_sparse_attention_compress_b200.torch_ops import KVCache
    with pytest.raises(ValueError, match="2\\^31"):      # 2^32 + 1 pages a sequence, of which ctypes would keep one
        KVCache.__new__(KVCache)._set("bf16", 1, 1, 64, 64, 16, (torch.zeros(1, 16, 1, 64),) * 2 + (None, None),
                                      torch.zeros(1, dtype=torch.int32).expand(1, 2 ** 32 + 1))


@pytest.mark.parametrize("name", ["k", "v", "k_scale", "v_scale", "page_table", "status"])
def test_tensors_of_a_cache_cannot_be_replaced(name):
    """The library keeps their addresses: a new tensor in their place would free the old one under the kernels."""
    from block_sparse_attention_compress_b200.torch_ops import KVCache
    with pytest.raises(AttributeError):
        setattr(KVCache.__new__(KVCache), name, torch.zeros(1))


def test_calls_by_addresses_run_on_the_current_stream(monkeypatch):
    """The structs tell no device and no stream: torch's current stream it is, not the default one."""
    class Library:
        def __getattr__(self, name):
            return lambda *args: streams.append(args[-1]) or nsa.NSA_OK

    class Current:
        cuda_stream = 4711

    streams = []
    monkeypatch.setattr(nsa, "load_library", lambda: Library())
    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: True)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: Current)
    c = _cache()
    for stream, want in ((None, 4711), (0, 0), (12, 12)):
        nsa.nsa_cache_append(c, _append(), stream=stream)
        nsa.nsa_cache_read(c, 0x300000, None, 1, 0, 0x700000, 0x800000, stream=stream)
        nsa.nsa_cache_attention(c, 0x700000, _attn(), 0x800000, stream=stream)
        assert streams[-3:] == [want] * 3


def test_the_default_streams_own_handle_is_the_default_stream(monkeypatch):
    """cudaStreamLegacy is 1, which torch would take for a stream of its own pool."""
    import contextlib

    from block_sparse_attention_compress_b200.torch_ops import KVCache
    handles = []
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: handles.append(handle))
    cache = KVCache.__new__(KVCache)
    cache.device = torch.device("cpu")
    for handle in (1, 0, 2, 0x7f00):
        cache._new(torch.zeros(3), (4,), handle)
    assert handles == [0, 0, 2, 0x7f00]


# ------------------------------------------------------------------ the oracle's pins

def test_rotation_turns_pairs_by_the_angle():
    """A rotation by a then b is one by a + b, lengths stay, and a quarter turn maps (1, 0) to (0, 1)."""
    row = lambda ang: torch.cat((torch.cos(ang), torch.sin(ang)))
    a, b = torch.tensor([0.3, 1.0, -2.0, 0.0]).double(), torch.tensor([0.5, 0.1, 1.0, 3.0]).double()
    x = torch.randn(3, 12, generator=torch.Generator().manual_seed(1)).double()
    for il in (False, True):
        two = co.rotate(co.rotate(x, row(a), il), row(b), il)
        one = co.rotate(x, row(a + b), il)
        assert torch.allclose(two, one, atol=1e-12)
        assert torch.equal(one[:, 8:], x[:, 8:])                       # dims behind the rotation
        assert torch.allclose(one.square().sum(-1), x.square().sum(-1))
    quarter = torch.tensor([0.0, 1.0])
    assert co.rotate(torch.tensor([[1.0, 0.0]]), quarter).tolist() == [[0.0, 1.0]]
    assert co.rotate(torch.tensor([[0.0, 1.0]]), quarter, True).tolist() == [[-1.0, 0.0]]


def test_four_bits_hand_worked():
    x = torch.arange(32).float() * 0.5 - 4.0                            # -4 .. 11.5, span 15.5
    codes, s, z = co.quantise(x)
    s_want = torch.tensor(15.5 / 15).bfloat16().float()                 # 1.03125
    assert float(s) == float(s_want) == 1.03125
    assert float(z) == -4.0 + 8 * 1.03125                               # 4.25, exact in bf16
    assert codes[0] == 0 and codes[-1] == 15
    assert co.quantise(torch.full((32,), 3.0))[0].tolist() == [8] * 32  # no span: the value itself
    assert float(co.through_4_bits(torch.full((32,), 3.0))[5]) == 3.0
    for odd in (math.nan, math.inf, -math.inf):
        y = x.clone()
        y[7] = odd
        assert torch.isnan(co.through_4_bits(y)).all()


def test_four_bits_error_bound():
    """Half a step, plus what rounding s (2^-8 of it, over up to 15 steps) and z (2^-8) can add."""
    g = torch.Generator().manual_seed(2)
    for std, mean in ((1.0, 0.0), (1e-6, 0.0), (1e6, 0.0), (0.1, 2.0)):
        x = (torch.randn((200, 32), generator=g) * std + mean).bfloat16()
        codes, s, z = co.quantise(x)
        err = (co.dequantise(codes, s, z) - x.double()).abs()
        bound = s.double() * (0.5 + 15 * 2.0 ** -8) + z.double().abs() * 2.0 ** -8
        assert (err <= bound[:, None] * (1 + 1e-5)).all()


@pytest.mark.parametrize("d", [64, 128, 192])
def test_nibble_orders_are_permutations_that_keep_runs(d):
    for order, run in ((co.nibble_order_keys(d), 8), (co.nibble_order_values(d), 4)):
        assert sorted(order) == list(range(d))
        for i in range(0, d, run):
            assert order[i:i + run] == list(range(order[i], order[i] + run)) and order[i] % run == 0
    # the first stored words of a key row: word 0 of every group
    assert co.nibble_order_keys(d)[::8][: d // 32] == [32 * g for g in range(d // 32)]


def test_attention_oracle_against_library_and_closed_forms():
    g = torch.Generator().manual_seed(3)
    L, n, h_q, h_kv, d = 23, 4, 4, 2, 8
    q, k, v = (torch.randn(s, generator=g).double() for s in ((n, h_q, d), (L, h_kv, d), (L, h_kv, d)))
    out, lse, mag = co.attend(q, k, v)
    mask = torch.ones(L, L).tril().bool()[-n:]
    ref = torch.nn.functional.scaled_dot_product_attention(
        q.transpose(0, 1), k.repeat_interleave(2, 1).transpose(0, 1), v.repeat_interleave(2, 1).transpose(0, 1), mask)
    assert torch.allclose(out, ref.transpose(0, 1), atol=1e-12)
    assert (mag >= out.abs() - 1e-12).all()
    # a window of one token gives that token's value; a huge slope as well
    assert torch.allclose(co.attend(q, k, v, window=1)[0], v[-n:].repeat_interleave(2, 1))
    steep = co.attend(q, k, v, slopes=torch.full((h_q,), 1e3))[0]
    assert torch.allclose(steep, v[-n:].repeat_interleave(2, 1))
    # a cap far above the scores changes nothing, a tiny one makes them equal
    assert torch.allclose(co.attend(q, k, v, softcap=1e6)[0], out, atol=1e-9)
    flat = co.attend(q[-1:], k, v, softcap=1e-9)
    assert torch.allclose(flat[0], v.mean(0, keepdim=True).repeat_interleave(2, 1), atol=1e-8)
    assert torch.allclose(flat[1], torch.full((1, h_q), math.log(L)).double(), atol=1e-8)
    # fewer tokens than queries: the first ones have nothing
    out, lse, _ = co.attend(q, k[:2], v[:2])
    assert (out[:2] == 0).all() and (lse[:2] == -math.inf).all() and torch.allclose(out[2], v[0].repeat_interleave(2, 0))
    # tokens that do not exist are as if never there
    seen = torch.rand(L, generator=g) > 0.3
    seen[-1] = True
    a = co.attend(q[-1:], k, v, seen=seen)[0]
    assert torch.allclose(a, co.attend(q[-1:], k[seen], v[seen])[0])
