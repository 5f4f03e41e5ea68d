"""Python face of the serving calls: one new token per sequence through a
decoder layer.

PagedKVCache holds a paged key-value cache (append, attend); W4Experts holds
4-bit expert weights.  As in api.py the work is done by the library's kernels;
here arguments are checked and turned into pointers.
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import _lib
from .api import MoEError, _check, _p, _stream, make_desc  # noqa: F401

_DT = {torch.float32: _lib.MOE_F32, torch.bfloat16: _lib.MOE_BF16,
       torch.float8_e4m3fn: _lib.MOE_E4M3}
_I32, _F32, _BF16 = torch.int32, torch.float32, torch.bfloat16
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _want(ok: bool, what: str):
    if not ok:
        raise ValueError(what)


def _handle(stream, device):
    """The CUDA stream handle of `stream`, or of the device's current stream
    (without building a Stream object, which costs 2 us a call)."""
    if stream is None:
        return _raw_stream(device.index or 0)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


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
        self.device = dev
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
        self.ws = torch.zeros(nbytes, dtype=torch.uint8, device=dev)
        self.status = torch.zeros(1, dtype=_I32, device=dev)
        self._ws, self._nbytes, self._status = self.ws.data_ptr(), nbytes, self.status.data_ptr()

    def _heads(self, t, rows, heads, name):
        """Pointer and token stride of a (rows, heads, head_dim) tensor whose
        heads are contiguous."""
        _want(t.dtype == self.dtype and t.device == self.device
              and t.shape == (rows, heads, self.head_dim)
              and (t.stride(2) == 1 and (heads == 1 or t.stride(1) == self.head_dim)),
              f"{name}: ({rows}, {heads}, {self.head_dim}) {self.dtype}, a token's heads contiguous")
        return t.data_ptr(), t.stride(0)

    def append(self, q, k, v, seq_ids, positions, q_out=None, stream=None):
        """Rotates q and k by position, writes k and v into the cache, returns
        the rotated q (in q_out, allocated when not given; q_out may be q).
        q: (n, q_heads, head_dim) or None (then None is returned); k, v:
        (n, kv_heads, head_dim); seq_ids, positions: (n,) int32, a negative
        sequence marking a padding token."""
        n = k.shape[0]
        kp, ks = self._heads(k, n, self.kv_heads, "k")
        vp, vs = self._heads(v, n, self.kv_heads, "v")
        for name, t in (("seq_ids", seq_ids), ("positions", positions)):
            _want(t.dtype == _I32 and t.shape == (n,) and t.device == self.device
                  and t.is_contiguous(), f"{name}: ({n},) int32")
        qp, qs, op = None, 0, None
        if q is not None:
            qp, qs = self._heads(q, n, self.q_heads, "q")
            if q_out is None:
                q_out = torch.empty((n, self.q_heads, self.head_dim), dtype=self.dtype,
                                    device=self.device)
            op = self._heads(q_out, n, self.q_heads, "q_out")[0]
            _want(q_out.is_contiguous(), "q_out: contiguous")
        else:
            _want(q_out is None, "q_out without q")
        st = self._append(self._ref, n, qp, qs, kp, ks, vp, vs, seq_ids.data_ptr(),
                          positions.data_ptr(), op, self._status, _handle(stream, self.device))
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
        _want(seq_lens.dtype == _I32 and seq_lens.shape == (B,) and seq_lens.is_contiguous()
              and seq_lens.device == self.device, f"seq_lens: ({B},) int32")
        if out is None:
            out = torch.empty((B, self.q_heads, self.head_dim), dtype=self.dtype,
                              device=self.device)
        else:
            _want(out.dtype == self.dtype and out.is_contiguous() and out.device == self.device
                  and out.shape == (B, self.q_heads, self.head_dim), "out: like q, contiguous")
        _want(lse is None or (lse.dtype == _F32 and lse.is_contiguous()
                              and lse.device == self.device and lse.shape == (B, self.q_heads)),
              f"lse: ({B}, {self.q_heads}) float32")
        st = self._attend(self._ref, qp, qs, seq_lens.data_ptr(), int(window),
                          1.0 / math.sqrt(self.head_dim) if scale is None else float(scale),
                          out.data_ptr(), None if lse is None else lse.data_ptr(), self._ws,
                          self._nbytes, self._status, _handle(stream, self.device))
        if st:
            raise MoEError(st, "moe_paged_attention")
        return out

    def check(self, stream=None):
        """Waits for the stream and raises MoEError if a call met a sequence,
        position or page out of range."""
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
    new = lambda shape, dt: torch.empty(shape, dtype=dt, device=w13.device)  # noqa: E731
    out = (new((E, 2 * I, H // 8), _I32), new((E, 2 * I, max(H // group, 0)), _BF16),
           new((E, H, I // 8), _I32), new((E, H, max(I // group, 0)), _BF16))
    desc = make_desc(0, H, I, E, 1, _BF16, False)
    _check(_lib.load().moe_quantize_weights_w4(
        ctypes.byref(desc), int(group), _p(w13), _p(w2), *[_p(t) for t in out],
        _handle(stream, w13.device)), "moe_quantize_weights_w4")
    return out


class W4Experts:
    """The routed experts on 4-bit weights, for up to max_tokens tokens a call.
    Keeps a copy of the weights in the kernels' own order; the tensors passed
    are not needed afterwards.

    w13_q (E, 2I, H/8) and w2_q (E, H, I/8) int32 codes, w13_s (E, 2I,
    H/group) and w2_s (E, H, I/group) bfloat16 scales (quantize_weights_w4, or
    a checkpoint's own codes in the packing that include/moe.h gives).
    K: experts per token."""

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
        self.max_tokens, self.device = int(max_tokens), dev
        self.desc = make_desc(self.max_tokens, H, I, E, K, _BF16, False)
        self._ref = ctypes.byref(self.desc)
        lib = _lib.load()
        self._call = lib.moe_experts_w4
        sizes = [lib.moe_w4_tiled_bytes(self._ref, group, i) for i in (0, 1)]
        nbytes = lib.moe_experts_w4_workspace_size(self._ref)
        if 0 in sizes or (nbytes == 0 and self.max_tokens > 0):  # the library's own reason
            _check(self._call(self._ref, group, *[None] * 7, 0, None, None), "W4Experts")
        self.w13_t, self.w2_t = (torch.empty(n, dtype=torch.uint8, device=dev) for n in sizes)
        _check(lib.moe_prepare_weights_w4(
            self._ref, group, _p(w13_q), _p(w13_s), _p(w2_q), _p(w2_s), _p(self.w13_t),
            _p(self.w2_t), _handle(None, dev)), "moe_prepare_weights_w4")
        self.ws = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=dev)
        self.status = torch.zeros(1, dtype=_I32, device=dev)
        self._w = self.w13_t.data_ptr(), self.w2_t.data_ptr()
        self._tail = (self.ws.data_ptr(), nbytes, self.status.data_ptr())

    def __call__(self, x, topk_idx, topk_w, y=None, stream=None):
        """y (n, H) bfloat16 (allocated when not given) for x (n, H) bfloat16
        and its routing topk_idx (n, K) int32, topk_w (n, K) float32."""
        n = x.shape[0]
        _want(n <= self.max_tokens, f"{n} tokens, and {self.max_tokens} at most")
        _want(x.dtype == _BF16 and x.shape == (n, self.H) and x.is_contiguous()
              and x.device == self.device, f"x: contiguous ({n}, {self.H}) bfloat16")
        _want(topk_idx.dtype == _I32 and topk_idx.shape == (n, self.K)
              and topk_idx.is_contiguous() and topk_idx.device == self.device
              and topk_w.dtype == _F32 and topk_w.shape == (n, self.K)
              and topk_w.is_contiguous() and topk_w.device == self.device,
              f"topk_idx and topk_w: contiguous ({n}, {self.K}) int32 and float32")
        if y is None:
            y = torch.empty((n, self.H), dtype=_BF16, device=self.device)
        else:
            _want(y.dtype == _BF16 and y.shape == x.shape and y.is_contiguous()
                  and y.device == self.device, "y: like x")
        self.desc.n = n
        st = self._call(self._ref, self.group, x.data_ptr(), topk_idx.data_ptr(),
                        topk_w.data_ptr(), *self._w, y.data_ptr(), *self._tail,
                        _handle(stream, self.device))
        if st:
            raise MoEError(st, "moe_experts_w4")
        return y

    def check(self, stream=None):
        """Waits for the stream and raises MoEError if a call met an expert id
        out of range."""
        _check(int(_lib.load().moe_check_status(_p(self.status), _stream(stream))),
               "device status")
