"""Python face of the serving calls: one new token per sequence through a
decoder layer.

PagedKVCache holds a paged key-value cache (append, attend); W4Experts holds
4-bit expert weights.  As in api.py the work is done by the library's kernels;
here arguments are checked and turned into pointers.  Tensors are on the
current CUDA device, where the library launches.
"""
from __future__ import annotations

import ctypes
import math
import threading

import torch

from . import _lib
from .api import MoEError, _check, _p, _stream, make_desc  # noqa: F401

_DT = {torch.float32: _lib.MOE_F32, torch.bfloat16: _lib.MOE_BF16,
       torch.float8_e4m3fn: _lib.MOE_E4M3}
_PER_THREAD = 2  # cudaStreamPerThread: one handle for a stream of every thread
_I32, _F32, _BF16 = torch.int32, torch.float32, torch.bfloat16
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _want(ok: bool, what: str):
    if not ok:
        raise ValueError(what)


def _ready(device):
    """Refuses what the library cannot run on: it launches on the current
    device, and takes every pointer for that device's memory."""
    if device.type != "cuda":
        raise ValueError(f"tensors on a CUDA device wanted, these are on {device}")
    if device.index != _current_device():
        raise ValueError(f"the tensors are on {device}, which is not the current CUDA device "
                         "(torch.cuda.set_device, or with torch.cuda.device)")


def _index(device):
    """A CUDA device's number, None for other devices."""
    return device.index if device.type == "cuda" else None


def _handle(stream, index):
    """The CUDA stream handle of `stream`, or of device `index`'s current
    stream (without building a Stream object, which costs 2 us a call)."""
    if stream is None:
        return _raw_stream(index)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _empty(shape, dtype, device, stream):
    """Memory for a result that a call on `stream` (None: the current one) writes:
    the allocator's reuse of it is ordered on that stream, and waits for the
    current one, where the result is used."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    current, handle = torch.cuda.current_stream(device), _handle(stream, None)
    own = torch.cuda.ExternalStream(handle, device=device)
    with torch.cuda.stream(own):
        if handle != _PER_THREAD or torch.cuda.is_current_stream_capturing():
            t = torch.empty(shape, dtype=dtype, device=device)
            t.record_stream(current)
            return t
    # the allocator takes threads' streams of one handle for one stream: memory of
    # the current one, which this thread's waits for
    t = torch.empty(shape, dtype=dtype, device=device)
    own.wait_stream(current)
    t.record_stream(own)
    return t


class _Workspaces:
    """A workspace for each stream that an object's calls run on, so that calls
    on several streams may run at the same time.

    make() allocates one on the current stream; `kept` are the object's other
    tensors, filled on the stream that is current now.  Another stream's first
    call waits for that.  A call under stream capture on a stream that has no
    workspace yet uses the first one (memory allocated by a capture belongs to
    its graph).  The per-thread default stream is one of each thread."""

    def __init__(self, device, make, kept):
        self._device, self._make, self._kept = device, make, kept
        self.all = [make()]
        self._made, handle = None, 0
        if device.type == "cuda":
            stream = torch.cuda.current_stream(device)
            self._made, handle = stream.record_event(), stream.cuda_stream
        self._thread = threading.local()  # pointer: of the thread's default stream
        self.pointers = {}  # by stream handle
        if handle == _PER_THREAD:
            self._thread.pointer = self.all[0].data_ptr()
        else:
            self.pointers[handle] = self.all[0].data_ptr()

    def add(self, handle):
        """The workspace of a stream's first call."""
        own = handle == _PER_THREAD
        if own and hasattr(self._thread, "pointer"):
            return self._thread.pointer
        stream = torch.cuda.ExternalStream(handle, device=self._device)
        with torch.cuda.stream(stream):
            if torch.cuda.is_current_stream_capturing():
                return self.all[0].data_ptr()
            stream.wait_event(self._made)
            if not own:
                ws = self._make()
        if own:  # not of the handle's memory, which the allocator takes for one stream's
            home = torch.cuda.default_stream(self._device)
            with torch.cuda.stream(home):
                ws = self._make()
            stream.wait_stream(home)
        for t in self._kept:
            t.record_stream(stream)
        self.all.append(ws)
        if own:
            self._thread.pointer = ws.data_ptr()
            return ws.data_ptr()
        return self.pointers.setdefault(handle, ws.data_ptr())


def rope_table(rows: int, dim: int, base: float = 10000.0, device="cuda"):
    """(rows, dim) float32: for each position the cosines and then the sines of
    its dim/2 angles position * base^(-2i/dim), evaluated in float64."""
    f = base ** (-torch.arange(0, dim, 2, dtype=torch.float64) / dim)
    a = torch.arange(rows, dtype=torch.float64)[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).to(device=device, dtype=_F32)


class PagedKVCache:
    """A paged key-value cache of one layer and the calls on it.

    k_cache, v_cache: (num_pages, kv_heads, page_size, head_dim) float32,
    bfloat16 or float8_e4m3fn; each page contiguous, pages any equal distance
    apart.  page_table: (num_seqs, max_pages) int32.  q_heads: query heads.
    k_scale, v_scale: (kv_heads,) float32, float8 caches only.  rope: a
    rope_table, or None.  All are the caller's and are kept alive here; the
    page table may be changed in place between calls.  Queries, keys, values
    and results are bfloat16 (float32 for a float32 cache).

    Calls run on `stream`, or the current stream; each stream has a workspace
    of its own, and a result allocated by a call is ready for that stream's
    next work.  Calls captured in graphs share the workspace of the stream on
    which the object was made: replays are ordered with each other and with
    that stream's calls by the caller.
    """

    def __init__(self, k_cache, v_cache, page_table, q_heads, k_scale=None, v_scale=None,
                 rope=None, rope_interleaved=False):
        _want(k_cache.dim() == 4 and k_cache.shape == v_cache.shape
              and k_cache.dtype == v_cache.dtype, "k_cache and v_cache: one 4-dimensional shape and type")
        _want(k_cache.dtype in _DT, "cache type: float32, bfloat16 or float8_e4m3fn")
        pages, kv_heads, size, dim = k_cache.shape
        for t in (k_cache, v_cache):
            _want(t.stride()[1:] == (size * dim, dim, 1) and t.stride(0) == k_cache.stride(0),
                  "pages are contiguous, and as far apart in k_cache as in v_cache")
        _want(page_table.dim() == 2 and page_table.dtype == _I32 and page_table.is_contiguous(),
              "page_table: contiguous (num_seqs, max_pages) int32")
        dev = k_cache.device
        for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
            _want(t is None or (t.dtype == _F32 and t.shape == (kv_heads,) and t.is_contiguous()),
                  f"{name}: (kv_heads,) float32")
        _want(rope is None or (rope.dim() == 2 and rope.dtype == _F32 and rope.is_contiguous()),
              "rope: contiguous (rows, dim) float32")
        for t in (v_cache, page_table, k_scale, v_scale, rope):
            _want(t is None or t.device == dev, "all tensors on one device")
        self.k_cache, self.v_cache, self.page_table = k_cache, v_cache, page_table
        self.k_scale, self.v_scale, self.rope = k_scale, v_scale, rope
        self.dtype = _F32 if k_cache.dtype == _F32 else _BF16
        self.device, self._index = dev, _index(dev)
        self._scale = 1.0 / math.sqrt(dim)
        self.num_seqs, self.q_heads, self.kv_heads, self.head_dim = (
            page_table.shape[0], int(q_heads), kv_heads, dim)
        rows, rdim = rope.shape if rope is not None else (0, 0)
        self.desc = _lib.KVCacheDesc(
            self.num_seqs, self.q_heads, kv_heads, dim, size, pages, page_table.shape[1],
            _DT[self.dtype], _DT[k_cache.dtype], rows, rdim, int(bool(rope_interleaved)),
            k_cache.stride(0) if pages > 1 else kv_heads * size * dim, _p(k_cache), _p(v_cache),
            _p(page_table), _p(k_scale), _p(v_scale), _p(rope))
        self._ref = ctypes.byref(self.desc)
        lib = _lib.load()
        self._append, self._attend = lib.moe_kv_append, lib.moe_paged_attention
        nbytes = lib.moe_paged_attention_workspace_size(self._ref)
        if nbytes == 0:  # the library's own reason
            _check(self._attend(self._ref, None, 0, None, 0, 1.0, None, None, None, 0, None, None),
                   "PagedKVCache")
        self.status = torch.zeros(1, dtype=_I32, device=dev)
        self._nbytes, self._status = nbytes, self.status.data_ptr()
        self._streams = _Workspaces(
            dev, lambda: torch.zeros(nbytes, dtype=torch.uint8, device=dev), [self.status])
        self.ws = self._streams.all[0]
        self._pointers = self._streams.pointers

    def _heads(self, t, rows, heads, name):
        """Pointer and token stride of a (rows, heads, head_dim) tensor whose
        heads are contiguous."""
        st = t.stride()
        if (t.dtype is not self.dtype or t.shape != (rows, heads, self.head_dim) or st[2] != 1
                or (st[1] != self.head_dim and heads != 1) or t.device != self.device):
            raise ValueError(f"{name}: ({rows}, {heads}, {self.head_dim}) {self.dtype} on "
                             f"{self.device}, a token's heads contiguous")
        return t.data_ptr(), st[0]

    def _ints(self, t, n, name):
        """Pointer of a contiguous (n,) int32 tensor."""
        if (t.dtype is not _I32 or t.shape != (n,) or not t.is_contiguous()
                or t.device != self.device):
            raise ValueError(f"{name}: contiguous ({n},) int32 on {self.device}")
        return t.data_ptr()

    def _result(self, rows, stream):
        if self._index is None or self._index != _current_device():
            _ready(self.device)
        return _empty((rows, self.q_heads, self.head_dim), self.dtype, self.device, stream)

    def append(self, q, k, v, seq_ids, positions, q_out=None, stream=None):
        """Rotates q and k by position, writes k and v into the cache, returns
        the rotated q (in q_out, allocated when not given; q_out may be q).
        q: (n, q_heads, head_dim) or None (then None is returned); k, v:
        (n, kv_heads, head_dim); seq_ids, positions: (n,) int32, a negative
        sequence marking a padding token."""
        n = k.shape[0]
        kp, ks = self._heads(k, n, self.kv_heads, "k")
        vp, vs = self._heads(v, n, self.kv_heads, "v")
        sp, pp = self._ints(seq_ids, n, "seq_ids"), self._ints(positions, n, "positions")
        qp, qs, op = None, 0, None
        if q is not None:
            qp, qs = self._heads(q, n, self.q_heads, "q")
            if q_out is None:
                q_out = self._result(n, stream)
            op, os = self._heads(q_out, n, self.q_heads, "q_out")
            _want(n < 2 or os == self.q_heads * self.head_dim, "q_out: contiguous")
        else:
            _want(q_out is None, "q_out without q")
        if self._index is None or self._index != _current_device():
            _ready(self.device)
        handle = _handle(stream, self._index)
        if handle not in self._pointers:
            self._streams.add(handle)  # for the status word
        st = self._append(self._ref, n, qp, qs, kp, ks, vp, vs, sp, pp, op, self._status, handle)
        if st:
            raise MoEError(st, "moe_kv_append")
        return q_out

    def attend(self, q, seq_lens, out=None, lse=None, window=0, scale=None, stream=None):
        """Attention of one new token per sequence: q (num_seqs, q_heads,
        head_dim), seq_lens (num_seqs,) int32 with the new token counted.
        Returns out (allocated when not given); lse: (num_seqs, q_heads)
        float32 to fill, or None.  window: only the last tokens (0: all).
        scale: of the scores, 1/sqrt(head_dim) when None."""
        B = self.num_seqs
        qp, qs = self._heads(q, B, self.q_heads, "q")
        lp = self._ints(seq_lens, B, "seq_lens")
        if out is None:
            out = self._result(B, stream)
        op, os = self._heads(out, B, self.q_heads, "out")
        _want(B < 2 or os == self.q_heads * self.head_dim, "out: contiguous")
        if lse is not None and (lse.dtype is not _F32 or lse.shape != (B, self.q_heads)
                                or not lse.is_contiguous() or lse.device != self.device):
            raise ValueError(f"lse: contiguous ({B}, {self.q_heads}) float32 on {self.device}")
        if self._index is None or self._index != _current_device():
            _ready(self.device)
        handle = _handle(stream, self._index)
        st = self._attend(self._ref, qp, qs, lp, window, self._scale if scale is None else scale,
                          op, None if lse is None else lse.data_ptr(),
                          self._pointers.get(handle) or self._streams.add(handle), self._nbytes,
                          self._status, handle)
        if st:
            raise MoEError(st, "moe_paged_attention")
        return out

    def check(self, stream=None):
        """Waits for the stream (the calls' one) and raises MoEError if a call
        met a sequence, position or page out of range."""
        _ready(self.device)
        _check(int(_lib.load().moe_check_status(_p(self.status), _stream(stream))),
               "device status")


def quantize_weights_w4(w13, w2, group=128, stream=None):
    """4-bit codes and group scales of bf16 expert weights w13 (E, H, 2I) and
    w2 (E, I, H): (w13_q, w13_s, w2_q, w2_s) for W4Experts."""
    _want(w13.dim() == 3 and w2.dim() == 3 and w13.dtype == _BF16 and w2.dtype == _BF16
          and w13.is_contiguous() and w2.is_contiguous() and w13.device == w2.device,
          "w13 and w2: contiguous 3-dimensional bfloat16")
    E, H, I2 = w13.shape
    I = I2 // 2
    _want(w2.shape == (E, I, H) and I2 == 2 * I, "w13 (E, H, 2I) and w2 (E, I, H)")
    _want(group > 0, "group: 32, 64 or 128")
    lib, desc = _lib.load(), make_desc(0, H, I, E, 1, _BF16, False)
    refused = lib.moe_w4_tiled_bytes(ctypes.byref(desc), int(group), 0) == 0
    if not refused:
        _ready(w13.device)
    new = lambda shape, dt: _empty(shape, dt, w13.device, None if refused else stream)  # noqa: E731
    out = (new((E, 2 * I, H // 8), _I32), new((E, 2 * I, H // group), _BF16),
           new((E, H, I // 8), _I32), new((E, H, I // group), _BF16))
    _check(lib.moe_quantize_weights_w4(
        ctypes.byref(desc), int(group), _p(w13), _p(w2), *[_p(t) for t in out],
        None if refused else _handle(stream, w13.device.index)), "moe_quantize_weights_w4")
    return out


class W4Experts:
    """The routed experts on 4-bit weights, for up to max_tokens tokens a call.
    Keeps a copy of the weights in the kernels' own order; the tensors passed
    are not needed afterwards.

    w13_q (E, 2I, H/8) and w2_q (E, H, I/8) int32 codes, w13_s (E, 2I,
    H/group) and w2_s (E, H, I/group) bfloat16 scales (quantize_weights_w4, or
    a checkpoint's own codes in the packing that include/moe.h gives).
    K: experts per token.

    Calls run on `stream`, or the current stream; each stream has a workspace
    of its own, and a result allocated by a call is ready for that stream's
    next work.  Calls captured in graphs share the workspace of the stream on
    which the object was made: replays are ordered with each other and with
    that stream's calls by the caller."""

    def __init__(self, w13_q, w13_s, w2_q, w2_s, K, max_tokens):
        _want(all(t.dim() == 3 and t.is_contiguous() for t in (w13_q, w13_s, w2_q, w2_s)),
              "codes and scales: contiguous, 3-dimensional")
        _want(w13_q.dtype == _I32 and w2_q.dtype == _I32 and w13_s.dtype == _BF16
              and w2_s.dtype == _BF16, "codes int32, scales bfloat16")
        E, I2, words = w13_q.shape
        H, I = 8 * words, I2 // 2
        _want(I2 == 2 * I and w2_q.shape == (E, H, I // 8) and I % 8 == 0,
              "w13_q (E, 2I, H/8) and w2_q (E, H, I/8)")
        group = H // w13_s.shape[2] if w13_s.shape[2] else 0
        _want(group > 0 and w13_s.shape == (E, I2, H // group) and H % group == 0
              and w2_s.shape == (E, H, I // group) and I % group == 0,
              "w13_s (E, 2I, H/group) and w2_s (E, H, I/group)")
        dev = w13_q.device
        _want(all(t.device == dev for t in (w13_s, w2_q, w2_s)), "all tensors on one device")
        self.H, self.I, self.E, self.K, self.group = H, I, E, int(K), group
        self.max_tokens, self.device, self._index = int(max_tokens), dev, _index(dev)
        self.desc = make_desc(self.max_tokens, H, I, E, K, _BF16, False)
        self._ref = ctypes.byref(self.desc)
        lib = _lib.load()
        self._call = lib.moe_experts_w4
        sizes = [lib.moe_w4_tiled_bytes(self._ref, group, i) for i in (0, 1)]
        nbytes = lib.moe_experts_w4_workspace_size(self._ref)
        if 0 in sizes or (nbytes == 0 and self.max_tokens > 0):  # the library's own reason
            _check(self._call(self._ref, group, *[None] * 7, 0, None, None), "W4Experts")
        _ready(dev)
        self.w13_t, self.w2_t = (torch.empty(n, dtype=torch.uint8, device=dev) for n in sizes)
        _check(lib.moe_prepare_weights_w4(
            self._ref, group, _p(w13_q), _p(w13_s), _p(w2_q), _p(w2_s), _p(self.w13_t),
            _p(self.w2_t), _handle(None, self._index)), "moe_prepare_weights_w4")
        self.status = torch.zeros(1, dtype=_I32, device=dev)
        self._streams = _Workspaces(
            dev, lambda: torch.empty(max(nbytes, 1), dtype=torch.uint8, device=dev),
            [self.w13_t, self.w2_t, self.status])
        self.ws = self._streams.all[0]
        self._pointers = self._streams.pointers
        self._w = self.w13_t.data_ptr(), self.w2_t.data_ptr()
        self._nbytes, self._status = nbytes, self.status.data_ptr()
        self._refs = {}  # descriptions by token count
        # a call is two or three kernels on one workspace: threads' calls enter the
        # stream one after another
        self._lock = threading.Lock()

    def _ref_for(self, n):
        """The layer's description for n tokens, which no other call changes."""
        ref = self._refs.get(n)
        if ref is None:
            desc = _lib.LayerDesc.from_buffer_copy(self.desc)
            desc.n = n
            ref = self._refs[n] = ctypes.byref(desc)
        return ref

    def __call__(self, x, topk_idx, topk_w, y=None, stream=None):
        """y (n, H) bfloat16 (allocated when not given) for x (n, H) bfloat16
        and its routing topk_idx (n, K) int32, topk_w (n, K) float32."""
        n = x.shape[0]
        if (n > self.max_tokens or x.dtype is not _BF16 or x.shape != (n, self.H)
                or not x.is_contiguous() or x.device != self.device):
            raise ValueError(f"x: contiguous (up to {self.max_tokens}, {self.H}) bfloat16 on "
                             f"{self.device}")
        for t, dt, name in ((topk_idx, _I32, "topk_idx"), (topk_w, _F32, "topk_w")):
            if (t.dtype is not dt or t.shape != (n, self.K) or not t.is_contiguous()
                    or t.device != self.device):
                raise ValueError(f"{name}: contiguous ({n}, {self.K}) {dt} on {self.device}")
        if y is None:
            if self._index is None or self._index != _current_device():
                _ready(self.device)
            y = _empty(x.shape, _BF16, self.device, stream)
        elif (y.dtype is not _BF16 or y.shape != x.shape or not y.is_contiguous()
              or y.device != self.device):
            raise ValueError("y: like x")
        if self._index is None or self._index != _current_device():
            _ready(self.device)
        handle = _handle(stream, self._index)
        ws = self._pointers.get(handle) or self._streams.add(handle)
        with self._lock:
            st = self._call(self._ref_for(n), self.group, x.data_ptr(), topk_idx.data_ptr(),
                            topk_w.data_ptr(), *self._w, y.data_ptr(), ws, self._nbytes,
                            self._status, handle)
        if st:
            raise MoEError(st, "moe_experts_w4")
        return y

    def check(self, stream=None):
        """Waits for the stream (the calls' one) and raises MoEError if a call
        met an expert id out of range."""
        _ready(self.device)
        _check(int(_lib.load().moe_check_status(_p(self.status), _stream(stream))),
               "device status")
