"""Torch-facing convenience calls over the C ABI: they allocate the outputs
and the workspace with torch (device memory is all torch provides) and call
the library's entry points on the current stream."""
from __future__ import annotations

import ctypes

import torch

from . import (NSA_CACHE_BF16, NSA_CACHE_INT4, NSA_MODE_MOBA, NSA_MODE_NSA, NsaCache, NsaCacheAppendArgs,
               NsaCacheAttentionArgs, NsaError, load_library, make_config, nsa_cache_attention_workspace, nsa_compress,
               nsa_decode, nsa_forward, nsa_forward_varlen, nsa_workspace_size)


def n_cmp(T: int, l: int = 32, s: int = 16) -> int:
    return 0 if T < l else (T - l) // s + 1


class NSAForward:
    """Prefill forward with a reusable workspace (one allocation per shape)."""

    def __init__(self, B, T, h_q, h_kv, d_k, d_v, w_k, w_v, *, top_k=16, window=512, sel_block=64,
                 force_first=1, force_local=1, softmax_scale=0.0, keep_idx=True, keep_kc=True, device="cuda",
                 score_map=0, mlp=None):
        """mlp: dict(b_k, w_k2, b_v, w_v2) of device tensors makes phi the two-layer MLP (w_k and
        w_v are then its first layers); None keeps the linear phi."""
        self.shape = (B, T, h_q, h_kv, d_k, d_v)
        nc = n_cmp(T)
        self.idx = torch.empty((B, h_kv, T, top_k), dtype=torch.int32, device=device) if keep_idx else None
        self.kc = torch.empty((B, nc, h_kv, d_k), dtype=torch.bfloat16, device=device) if keep_kc else None
        self.vc = torch.empty((B, nc, h_kv, d_v), dtype=torch.bfloat16, device=device) if keep_kc else None
        self.w_k, self.w_v = w_k, w_v
        self.cfg = make_config(mode=NSA_MODE_NSA, batch=B, seqlen=T, h_q=h_q, h_kv=h_kv, d_k=d_k, d_v=d_v,
                               top_k=top_k, window=window, sel_block=sel_block, force_first=force_first,
                               force_local=force_local, softmax_scale=softmax_scale, w_cmp_k=w_k, w_cmp_v=w_v,
                               sel_idx_out=self.idx, kc_out=self.kc, vc_out=self.vc, score_map=score_map)
        if mlp is not None:
            self.mlp = mlp   # keep the weights alive as long as the config points at them
            for name, val in (("phi_mlp", 1), ("w_cmp_k2", mlp["w_k2"].data_ptr()), ("w_cmp_v2", mlp["w_v2"].data_ptr()),
                              ("b_cmp_k", mlp["b_k"].data_ptr()), ("b_cmp_v", mlp["b_v"].data_ptr())):
                setattr(self.cfg, name, val)
        nbytes = nsa_workspace_size(self.cfg)
        if nbytes == 0:
            raise ValueError("nsa_workspace_size rejected the configuration")
        self.workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
        self.cfg.workspace = self.workspace.data_ptr()
        self.cfg.workspace_bytes = nbytes

    def device_status(self) -> int:
        """The workspace's status word after a synchronised call: 0, or the code of a
        device-side wait that timed out."""
        return int(self.workspace[:4].view(torch.int32).item())

    def __call__(self, q, k, v, gates, out=None):
        B, T, h_q, h_kv, d_k, d_v = self.shape
        if out is None:
            out = torch.empty((B, T, h_q, d_v), dtype=torch.bfloat16, device=q.device)
        nsa_forward(q, k, v, gates, self.cfg, out)
        return out


class NSAForwardVarlen(NSAForward):
    """Prefill forward of a packed batch of sequences of different lengths (at most T
    tokens each): q [total, h_q, d_k], k/v [total, h_kv, d], gates [total, h_q, 3], and
    cu_seqlens int32 [B + 1] on the device.  idx, kc and vc keep the per-sequence layouts of
    NSAForward (B sequences of up to T tokens)."""

    def __call__(self, q, k, v, gates, cu_seqlens, out=None):
        B, T, h_q, h_kv, d_k, d_v = self.shape
        if out is None:
            out = torch.empty((q.shape[0], h_q, d_v), dtype=torch.bfloat16, device=q.device)
        nsa_forward_varlen(q, k, v, gates, cu_seqlens, self.cfg, out)
        return out


def nsa_forward_torch(q, k, v, gates, w_k, w_v, **kw):
    """One-shot forward: returns (out, idx, kc, vc)."""
    B, T, h_q, d_k = q.shape
    h_kv, d_v = k.shape[2], v.shape[3]
    f = NSAForward(B, T, h_q, h_kv, d_k, d_v, w_k, w_v, device=q.device, **kw)
    out = f(q, k, v, gates)
    return out, f.idx, f.kc, f.vc


def compress_torch(x, w, l=32, s=16):
    B, T, H, d = x.shape
    out = torch.empty((B, n_cmp(T, l, s), H, w.shape[1]), dtype=torch.bfloat16, device=x.device)
    if out.shape[1]:
        nsa_compress(x, w, out, l, s)
    return out


# the current stream's handle, without the Stream object around it where torch offers that
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)


def _need(ok, what):
    if not ok:
        raise ValueError(what)


_INT32 = 1 << 31   # the C entries' integers are below it, and ctypes would keep the low bits of a larger one


class KVCache:
    """A paged key/value cache in bf16 or in 4 bits, with the three calls that work on it.

    ``KVCache(batch, max_len, h_kv, d_k, d_v)`` allocates the pool (``fmt`` "bf16" or "int4"),
    a status word and a page table that gives every sequence its own pages in order; a program
    with its own page allocator passes ``n_pages`` and writes into ``page_table`` [batch, max_pages]
    (int32) itself (the tensors of a cache stay: they are written into, not replaced).  ``from_pools`` takes existing bf16 pools, such as
    nsa_decode's caches.  Lengths (``seqlens``, int32 [batch] on the device) always count the new
    tokens.

    A token that cannot be placed (page table entry, position or length out of range) is skipped,
    and ``device_status()`` is then NSA_CODE_CACHE until ``status`` is zeroed.

    The calls run on the current stream, or on ``stream`` (a torch stream or its handle).  Outputs
    and workspaces are then that stream's memory, and as ever with streams the caller makes it wait
    for the inputs, and makes others wait for the outputs (and tells torch of their use there, with
    ``record_stream``)."""

    def __init__(self, batch, max_len, h_kv, d_k, d_v, *, fmt="bf16", page_size=64, n_pages=None, device="cuda"):
        _need(fmt in ("bf16", "int4"), f"fmt is 'bf16' or 'int4', not {fmt!r}")
        _need(min(batch, max_len, h_kv, d_k, d_v, page_size) >= 1, "sizes must be at least 1")
        max_pages = -(-max_len // page_size)
        n_pages = batch * max_pages if n_pages is None else n_pages
        _need(n_pages >= 1, "n_pages must be at least 1")
        bf, u8 = torch.bfloat16, torch.uint8
        if fmt == "bf16":
            pools = (torch.zeros((n_pages, page_size, h_kv, d_k), dtype=bf, device=device),
                     torch.zeros((n_pages, page_size, h_kv, d_v), dtype=bf, device=device), None, None)
        else:
            _need(d_k % 32 == 0 and d_v % 32 == 0, "4 bits: head dims are multiples of 32")
            pools = (torch.zeros((n_pages, h_kv, page_size, d_k // 2), dtype=u8, device=device),
                     torch.zeros((n_pages, h_kv, page_size, d_v // 2), dtype=u8, device=device),
                     torch.zeros((n_pages, h_kv, page_size, d_k // 32, 2), dtype=bf, device=device),
                     torch.zeros((n_pages, h_kv, page_size, d_v // 32, 2), dtype=bf, device=device))
        table = torch.arange(batch * max_pages, dtype=torch.int32, device=device).view(batch, max_pages)
        self._set(fmt, batch, h_kv, d_k, d_v, page_size, pools, table)

    @classmethod
    def from_pools(cls, k, v, page_table):
        """Over existing bf16 pools k [n_pages, page_size, h_kv, d_k], v [.., d_v] and an int32
        page table [batch, max_pages] on the same device."""
        _need(k.dim() == 4 and v.dim() == 4 and k.shape[:3] == v.shape[:3], "k and v: [n_pages, page_size, h_kv, d]")
        _need(k.dtype == v.dtype == torch.bfloat16, "k and v must be bf16")
        _need(page_table.dim() == 2 and page_table.dtype == torch.int32, "page_table: int32 [batch, max_pages]")
        self = cls.__new__(cls)
        self._set("bf16", page_table.shape[0], k.shape[2], k.shape[3], v.shape[3], k.shape[1], (k, v, None, None), page_table)
        return self

    def _set(self, fmt, batch, h_kv, d_k, d_v, page_size, pools, table):
        _need(max(batch, h_kv, d_k, d_v, page_size, pools[0].shape[0], table.shape[1]) < _INT32, "sizes must be below 2^31")
        self.fmt, self.batch, self.h_kv, self.d_k, self.d_v, self.page_size = fmt, batch, h_kv, d_k, d_v, page_size
        self._pools, self._page_table = pools, table
        self.device = self.k.device
        for t in (self.k, self.v, self.page_table):
            _need(t.is_cuda and t.device == self.device and t.is_contiguous(), "pools and page table: contiguous, on one GPU")
        self._status = torch.zeros(1, dtype=torch.int32, device=self.device)
        p = lambda t: t.data_ptr() if t is not None else None
        self.desc = NsaCache(format=NSA_CACHE_INT4 if fmt == "int4" else NSA_CACHE_BF16, batch=batch, h_kv=h_kv, d_k=d_k,
                             d_v=d_v, page_size=page_size, n_pages=self.k.shape[0], max_pages=table.shape[1],
                             k=p(self.k), v=p(self.v), k_scale=p(self.k_scale), v_scale=p(self.v_scale),
                             page_table=p(table), status=p(self.status))
        self._lib, self._ref = load_library(), ctypes.byref(self.desc)
        self._workspaces = {}   # bytes by (n, h_q, max_seqlen, window)

    # The library has these tensors' addresses: their contents may be written, the attributes not be assigned.
    k = property(lambda self: self._pools[0], doc="keys: bf16 [n_pages, page_size, h_kv, d_k], or codes")
    v = property(lambda self: self._pools[1], doc="values, like the keys")
    k_scale = property(lambda self: self._pools[2], doc="4 bits: (s, z) of the keys' groups")
    v_scale = property(lambda self: self._pools[3], doc="4 bits: (s, z) of the values' groups")
    page_table = property(lambda self: self._page_table, doc="int32 [batch, max_pages]")
    status = property(lambda self: self._status, doc="int32 [1]: 0, or NSA_CODE_CACHE")

    @property
    def max_len(self):
        return self.desc.max_pages * self.page_size

    def device_status(self) -> int:
        """The status word after a synchronised call: 0, or NSA_CODE_CACHE."""
        return int(self.status.item())

    # A single token's calls take as long on the host as on the GPU: checks are plain conditions, and
    # their messages are made only when one fails.

    def _call(self, name, stream, *args):
        """The library's entry `name` on this cache, with the cache's device current."""
        index = self.device.index
        if stream is None:
            stream = _current_stream(index)
        elif not isinstance(stream, int):
            stream = stream.cuda_stream
        fn = getattr(self._lib, name)
        if torch.cuda.current_device() == index:
            st = fn(self._ref, *args, stream)
        else:
            with torch.cuda.device(index):
                st = fn(self._ref, *args, stream)
        if st:
            raise NsaError(st, name)

    def _lengths(self, t, n, name):
        if t.dtype is not torch.int32 or t.dim() != 1 or t.shape[0] != n or t.device != self.device or not t.is_contiguous():
            raise ValueError(f"{name}: contiguous int32 [{n}] on {self.device}")
        return t.data_ptr()

    def _rows(self, x, heads, d, packed, name):
        """Checks new rows [batch, n, heads, d] (packed: [total, heads, d]); the elements from one
        token to the next.  Tokens may lie apart (a slice of a wider row), a token's heads not."""
        shape = x.shape
        if len(shape) != (3 if packed else 4) or shape[-2] != heads or shape[-1] != d or not (packed or shape[0] == self.batch):
            raise ValueError(f"{name}: {'[total' if packed else f'[{self.batch}, n'}, {heads}, {d}], not {tuple(shape)}")
        if x.dtype is not torch.bfloat16 or x.device != self.device:
            raise ValueError(f"{name}: bf16 on {self.device}")
        stride = x.stride()
        if stride[-1] != 1 or (heads > 1 and stride[-2] != d):
            raise ValueError(f"{name}: heads and dims must be contiguous")
        tokens = shape[0] if packed else shape[0] * shape[1]
        if tokens <= 1:
            return max(heads * d, 8)
        if packed or shape[0] == 1:
            return stride[-3]
        if shape[1] == 1:
            return stride[0]
        if stride[0] != shape[1] * stride[1]:
            raise ValueError(f"{name}: tokens must lie at one stride")
        return stride[1]

    def _like(self, t, shape, dtype, name):
        """Checks a given output or table."""
        if tuple(t.shape) != tuple(shape) or t.dtype is not dtype or t.device != self.device or not t.is_contiguous():
            raise ValueError(f"{name}: contiguous {dtype} {tuple(shape)} on {self.device}")
        return t.data_ptr()

    def _new(self, like, shape, stream, dtype=torch.bfloat16):
        """Memory for `stream`: from that stream's pool, since a block of another's may still be in use there."""
        if stream is not None:
            if isinstance(stream, int):
                stream = torch.cuda.ExternalStream(stream if stream != 1 else 0, device=self.device)   # 1: the default stream's handle
            with torch.cuda.stream(stream):
                return like.new_empty(shape, dtype=dtype)
        if like.shape == shape and dtype is like.dtype:   # the quickest of torch's ways
            return torch.empty_like(like, memory_format=torch.contiguous_format)
        return like.new_empty(shape, dtype=dtype)

    def append(self, k, v, seqlens, *, cu_seqlens=None, cos_sin=None, interleaved=False, q=None, q_out=None, stream=None):
        """Write new tokens: k [batch, n, h_kv, d_k] and v [batch, n, h_kv, d_v] are the last n of
        each sequence's ``seqlens`` tokens; with cu_seqlens (int32 [batch + 1]) packed [total, ...].
        cos_sin fp32 [positions, rot_dim] (cosines, then sines) rotates the keys by their
        positions, and the queries q [.., h_q, d_k], which are returned (into q_out)."""
        packed = cu_seqlens is not None
        k_stride, v_stride = self._rows(k, self.h_kv, self.d_k, packed, "k"), self._rows(v, self.h_kv, self.d_v, packed, "v")
        lead = k.shape[:-2]
        if v.shape[:-2] != lead:
            raise ValueError("k and v must hold the same tokens")
        a = NsaCacheAppendArgs(k.data_ptr(), v.data_ptr(), None, None, self._lengths(seqlens, self.batch, "seqlens"))
        a.k_stride, a.v_stride = k_stride, v_stride
        if packed:
            a.cu_seqlens, a.total_tokens = self._lengths(cu_seqlens, self.batch + 1, "cu_seqlens"), lead[0]
        else:
            a.n_new = lead[1]
        if cos_sin is not None:
            if cos_sin.dim() != 2:
                raise ValueError("cos_sin: [positions, rot_dim]")
            a.n_positions, a.rot_dim = cos_sin.shape
            a.cos_sin, a.interleaved = self._like(cos_sin, cos_sin.shape, torch.float32, "cos_sin"), int(interleaved)
        if q is not None:
            if q.dim() < 2:
                raise ValueError("q: the new tokens' queries, [.., h_q, d_k]")
            h_q = q.shape[-2]
            a.q_stride = self._rows(q, h_q, self.d_k, packed, "q")
            if q.shape[:-2] != lead:
                raise ValueError("q must hold the same tokens as k")
            if q_out is None:
                q_out = self._new(q, q.shape, stream)
            else:
                self._like(q_out, q.shape, torch.bfloat16, "q_out")
            a.q, a.q_out, a.h_q = q.data_ptr(), q_out.data_ptr(), h_q
        if lead.numel():   # no tokens: nothing to do
            self._call("nsa_cache_append", stream, ctypes.byref(a))
        return q_out if q is not None else None

    def read(self, seqlens, n=None, *, cu_seqlens=None, total=None, k_out=None, v_out=None, stream=None):
        """The last n tokens of each sequence as contiguous bf16 (k [batch, n, h_kv, d_k], v), or,
        with cu_seqlens, the last cu[b+1] - cu[b] of each, packed into ``total`` rows."""
        packed = cu_seqlens is not None
        self._lengths(seqlens, self.batch, "seqlens")
        if packed:
            self._lengths(cu_seqlens, self.batch + 1, "cu_seqlens")
        if (total if packed else n) is None:
            raise ValueError("read takes n, or cu_seqlens and total")
        lead = (int(total),) if packed else (self.batch, int(n))
        if not 0 <= lead[-1] < _INT32:
            raise ValueError("read takes a number of tokens, below 2^31")
        shapes = (*lead, self.h_kv, self.d_k), (*lead, self.h_kv, self.d_v)
        if k_out is None:
            k_out = self._new(seqlens, shapes[0], stream, torch.bfloat16)
        else:
            self._like(k_out, shapes[0], torch.bfloat16, "k_out")
        if v_out is None:
            v_out = self._new(k_out, shapes[1], stream)
        else:
            self._like(v_out, shapes[1], torch.bfloat16, "v_out")
        if lead[-1]:
            self._call("nsa_cache_read", stream, seqlens.data_ptr(), cu_seqlens.data_ptr() if packed else None,
                       0 if packed else lead[1], lead[0] if packed else 0, k_out.data_ptr(), v_out.data_ptr())
        return k_out, v_out

    def attend(self, q, seqlens, max_seqlen=None, *, softmax_scale=0.0, softcap=0.0, slopes=None, window=0, out=None,
               lse=None, workspace=None, stream=None):
        """Attention of the newest tokens q [batch, n, h_q, d_k] (n = 1 .. 16; their keys and values
        are in the cache) over the cache.  max_seqlen bounds seqlens (default: the capacity; the
        nearer the bound, the better the work is split).  softcap caps the scores by tanh, slopes
        (fp32 [h_q]) adds slope * (u - p), window (0: none) keeps the last tokens; lse (fp32
        [batch, n, h_q]) receives the log-sum-exps.  The workspace is torch's unless one of
        attend_workspace() bytes is given."""
        if q.dim() != 4 or q.shape[0] != self.batch or q.shape[1] < 1 or q.shape[3] != self.d_k or \
                q.dtype is not torch.bfloat16 or q.device != self.device or not q.is_contiguous():
            raise ValueError(f"q: contiguous bf16 [{self.batch}, n, h_q, {self.d_k}] on {self.device}")
        B, n, h_q, _ = q.shape
        if out is None:
            out = self._new(q, (B, n, h_q, self.d_v), stream)
        else:
            self._like(out, (B, n, h_q, self.d_v), torch.bfloat16, "out")
        max_seqlen = self.max_len if max_seqlen is None else max_seqlen
        if not (-_INT32 <= max_seqlen < _INT32 and -_INT32 <= window < _INT32):
            raise ValueError("max_seqlen and window: below 2^31")
        a = NsaCacheAttentionArgs(self._lengths(seqlens, self.batch, "seqlens"),
                                  None if slopes is None else self._like(slopes, (h_q,), torch.float32, "slopes"),
                                  None if lse is None else self._like(lse, (B, n, h_q), torch.float32, "lse"),
                                  None, 0, softmax_scale, softcap, n, h_q, max_seqlen, window)
        if workspace is None:
            key = (n, h_q, max_seqlen, window)
            need = self._workspaces.get(key)
            if need is None:
                if len(self._workspaces) >= 64:
                    self._workspaces.clear()
                need = self._workspaces[key] = nsa_cache_attention_workspace(self.desc, a)
            if need:
                workspace = self._new(q, (need,), stream, torch.uint8)
        elif workspace.device != self.device or not workspace.is_contiguous():
            raise ValueError(f"workspace: contiguous on {self.device}")
        if workspace is not None:
            a.workspace, a.workspace_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
        self._call("nsa_cache_attention", stream, q.data_ptr(), ctypes.byref(a), out.data_ptr())
        return out

    def attend_workspace(self, n, h_q, max_seqlen=None, window=0):
        """Bytes of workspace attend() needs for n new tokens and h_q query heads."""
        max_seqlen = self.max_len if max_seqlen is None else max_seqlen
        if not all(-_INT32 <= x < _INT32 for x in (n, h_q, max_seqlen, window)):
            raise ValueError("n, h_q, max_seqlen and window: below 2^31")
        return nsa_cache_attention_workspace(
            self.desc, NsaCacheAttentionArgs(n_new=n, h_q=h_q, window=window, max_seqlen=max_seqlen))
