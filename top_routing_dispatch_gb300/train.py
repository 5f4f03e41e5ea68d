"""Python face of the training calls around the layer's backward pass.

LayerNorm is the norm before the layer with its gradients, GradNorm the global
norm of all gradients, AdamW the step that takes them.  As in api.py the work
is done by the library's kernels; here arguments are checked and turned into
pointers.  Tensors are on the current CUDA device, where the library launches.
Gradients are computed by explicit calls; torch's automatic differentiation does
not see them.

Calls run on `stream`, or the current stream.  Results that a call allocates
are ready for that stream's next work.  Scratch memory belongs to the stream
(calls on one stream run one after another), or to the graph where a call is
captured, so calls of one LayerNorm or GradNorm may run on several streams, and
in several graphs, at the same time.  Up to 32 MiB are kept for each stream; more
is allocated for the call.  A stream that is given by its handle, and is not
torch's, is to be destroyed only behind the work of its calls.
"""
from __future__ import annotations

import bisect
import ctypes
import itertools
import math
import threading

import torch

from . import _lib, api, decode
from .api import MoEError, _check, _p
from .decode import (_BF16, _DT, _F32, _I32, _PER_THREAD, _Workspaces, _empty, _handle, _index,
                     _want)

_E4M3 = torch.float8_e4m3fn
BLOCK = 256  # values of a tensor that share a scale where states are held in 8 bits


_scratch = {}  # (device, stream handle): the stream's scratch memory
_KEPT = 32 << 20  # bytes of it, at most: a norm's backward of up to 13797 columns
# a call with scratch is two kernels: threads' calls enter a stream one after another
_scratch_lock = threading.Lock()


def _scratch_for(nbytes, device, index, stream, handle):
    """Scratch memory of a call on `stream`, under the lock."""
    if stream is None:
        capturing = torch.cuda.is_current_stream_capturing()
    else:
        with torch.cuda.stream(torch.cuda.ExternalStream(handle, device=device)):
            capturing = torch.cuda.is_current_stream_capturing()
    if capturing:  # memory of the graph
        return _empty(nbytes, torch.uint8, device, stream)
    if handle == _PER_THREAD:  # another stream in every thread: memory of the call
        with torch.cuda.stream(torch.cuda.default_stream(device)):
            return _empty(nbytes, torch.uint8, device, handle)
    if nbytes > _KEPT:  # memory of the call: reused in the stream's order
        return _empty(nbytes, torch.uint8, device, stream)
    t = _scratch.get((index, handle))
    if t is None or t.numel() < nbytes:
        # the old one's memory is reused in the stream's order
        t = _scratch[index, handle] = _empty(max(nbytes, 1 << 20), torch.uint8, device, stream)
    return t


def _here(device, index):
    if index is None or index != decode._current_device():
        decode._ready(device)


class LayerNorm:
    """Layer norm of rows: y = (s - mean) / sqrt(variance + eps) * weight + bias,
    or its root mean square form (rms: the mean taken as 0).

    weight, bias: (H,), float32 or of the rows' type; bias may be None.
    dtype: of the rows, float32 or bfloat16 (weight's type when None).  Both
    tensors are the caller's and are kept alive here; they may be changed in
    place between calls.  Results share no memory with arguments or each other,
    and carry no graph for torch's automatic differentiation: gradients come
    from backward."""

    def __init__(self, weight, bias=None, eps=1e-5, rms=False, dtype=None):
        _want(weight.dim() == 1 and weight.is_contiguous() and weight.dtype in (_F32, _BF16),
              "weight: contiguous (H,) float32 or bfloat16")
        _want(bias is None or (bias.shape == weight.shape and bias.dtype == weight.dtype
                               and bias.is_contiguous() and bias.device == weight.device),
              "bias: like weight")
        dtype = weight.dtype if dtype is None else dtype
        _want(dtype in (_F32, _BF16), "dtype: float32 or bfloat16")
        self.weight, self.bias, self.dtype, self.H = weight, bias, dtype, weight.shape[0]
        self.device, self._index = weight.device, _index(weight.device)
        self._dev = weight.get_device()
        self._form = (self.H, _DT[dtype], _DT[weight.dtype], int(bool(rms)), float(eps))
        self._w, self._b = weight.data_ptr(), None if bias is None else bias.data_ptr()
        self._refs = {}  # descriptions by number of rows
        lib = _lib.load()
        self._forward, self._backward = lib.moe_layer_norm, lib.moe_layer_norm_backward
        self._ws_size = lib.moe_layer_norm_backward_workspace_size
        if self._ws_size(self._ref_for(1)[0]) == 0:  # the library's own reason
            _check(self._forward(self._ref_for(0)[0], None, 0, None, 0, *[None] * 6), "LayerNorm")

    def _ref_for(self, n):
        """The description of n rows, which no other call changes, and the bytes
        of scratch that its backward needs."""
        ref = self._refs.get(n)
        if ref is None:
            if len(self._refs) > 1000:
                self._refs = {}
            ref = ctypes.byref(_lib.NormDesc(n, *self._form))
            ref = self._refs[n] = (ref, self._ws_size(ref))
        return ref

    def _rows(self, t, shape, name):
        """Pointer and row stride of a (n, H) tensor whose rows are contiguous."""
        st = t.stride()
        if (t.dtype is not self.dtype or t.shape != shape or t.get_device() != self._dev
                or (st[1] != 1 and self.H != 1)):
            raise ValueError(f"{name}: {tuple(shape)} {self.dtype} on {self.device}, "
                             "rows contiguous")
        return t.data_ptr(), st[0]

    def _first(self, t, name):
        """Shape, pointer and row stride of the tensor that says how many rows there are."""
        shape = t.shape
        _want(len(shape) == 2 and shape[1] == self.H, f"{name}: (n, {self.H})")
        return shape, *self._rows(t, shape, name)

    def _out(self, t, shape, dtype, name):
        """Pointer of a given contiguous tensor."""
        if (t.dtype is not dtype or t.shape != shape or not t.is_contiguous()
                or t.get_device() != self._dev):
            raise ValueError(f"{name}: contiguous {tuple(shape)} {dtype} on {self.device}")
        return t.data_ptr()

    def __call__(self, x, residual=None, y=None, s=None, stats=None, stream=None):
        """y (n, H) of the rows x (n, H); with residual (n, H), of s = x +
        residual, and (y, s) is returned.  y and s are allocated when not
        given.  stats: (2, n) float32 to fill with means and reciprocal
        deviations for backward, or None."""
        shape, xp, xs = self._first(x, "x")
        n = shape[0]
        rp, rs, sp, tp = None, 0, None, None
        _here(self.device, self._index)
        if residual is not None:
            rp, rs = self._rows(residual, shape, "residual")
            if s is None:
                s = _empty(shape, self.dtype, self.device, stream)
            sp = self._out(s, shape, self.dtype, "s")
        elif s is not None:
            raise ValueError("s without residual")
        if y is None:
            y = _empty(shape, self.dtype, self.device, stream)
        yp = self._out(y, shape, self.dtype, "y")
        if stats is not None:
            tp = self._out(stats, (2, n), _F32, "stats")
        st = self._forward(self._ref_for(n)[0], xp, xs, rp, rs, self._w, self._b, sp, yp, tp,
                           _handle(stream, self._index))
        if st:
            raise MoEError(st, "moe_layer_norm")
        return y if residual is None else (y, s)

    def backward(self, dy, s, stats, ds=None, dx=None, dweight=None, dbias=None, stream=None):
        """(dx, dweight, dbias) for dy (n, H), from the rows s that were
        normalised (x, or the sum with the residual) and their stats.  ds (n,
        H): a gradient that reaches s by other ways, added to dx.  dx is of the
        rows' type, dweight and dbias (H,) float32 (None without a bias); they
        are allocated when not given and overwritten."""
        shape, dp, dst = self._first(dy, "dy")
        n, vec = shape[0], (self.H,)
        sp, sst = self._rows(s, shape, "s")
        ep, est = (None, 0) if ds is None else self._rows(ds, shape, "ds")
        _here(self.device, self._index)
        tp = self._out(stats, (2, n), _F32, "stats")
        if dx is None:
            dx = _empty(shape, self.dtype, self.device, stream)
        if dweight is None:
            dweight = _empty(vec, _F32, self.device, stream)
        bp = None
        if self._b is not None:
            if dbias is None:
                dbias = _empty(vec, _F32, self.device, stream)
            bp = self._out(dbias, vec, _F32, "dbias")
        elif dbias is not None:
            raise ValueError("dbias without a bias")
        ref, nbytes = self._ref_for(n)
        xp, wp = self._out(dx, shape, self.dtype, "dx"), self._out(dweight, vec, _F32, "dweight")
        handle = _handle(stream, self._index)
        with _scratch_lock:
            ws = _scratch_for(nbytes, self.device, self._index, stream, handle)
            st = self._backward(ref, dp, dst, sp, sst, tp, self._w, ep, est, xp, wp, bp,
                                ws.data_ptr(), nbytes, handle)
        if st:
            raise MoEError(st, "moe_layer_norm_backward")
        return dx, dweight, dbias


def _tensors(ts, name, types=(_F32, _BF16)):
    """A list of contiguous tensors of one device."""
    ts = list(ts)
    _want(len(ts) > 0, f"{name}: at least one tensor")
    for t in ts:
        _want(t.dtype in types and t.is_contiguous() and t.device == ts[0].device,
              f"{name}: contiguous {' or '.join(str(d) for d in types)}, all on one device")
    return ts


def _scalar(t, device, name):
    """Pointer of one float32 on the device, None for None."""
    if t is None:
        return None
    if t.dtype is not _F32 or t.numel() != 1 or t.get_device() != (
            -1 if device.type == "cpu" else device.index):
        raise ValueError(f"{name}: one float32 on {device}")
    return t.data_ptr()


def _apart(t, others):
    """Whether a contiguous tensor shares no memory with others (None: not there),
    what lies between their rows counted as theirs."""
    a, b = t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()
    for o in others:
        if o is not None and o.numel() and t.numel():
            size = (sum((n - 1) * st for n, st in zip(o.shape, o.stride())) + 1) * o.element_size()
            if a < o.data_ptr() + size and o.data_ptr() < b:
                return False
    return True


class GradNorm:
    """The global norm of a list of gradients, and the factor that clips it.

    grads: contiguous float32 or bfloat16 tensors of one device.  They are the
    caller's and are kept alive here; a call reads what they hold then."""

    def __init__(self, grads):
        self.grads = _tensors(grads, "grads")
        self.device = self.grads[0].device
        self._index = _index(self.device)
        self._list = (_lib.TensorDesc * len(self.grads))(
            *[_lib.TensorDesc(t.data_ptr(), t.numel(), _DT[t.dtype]) for t in self.grads])
        lib = _lib.load()
        self._call = lib.moe_grad_norm
        self._nbytes = lib.moe_grad_norm_workspace_size(len(self.grads))

    def __call__(self, max_norm=float("inf"), norm=None, factor=None, stream=None):
        """(norm, factor), one float32 each on the device (allocated when not
        given): the root of the sum of all squares, and min(1, max_norm / (norm
        + 1e-6)), the grad_scale of a clipped AdamW step.  The factor of an
        infinite norm is 0, but 1 where max_norm is infinite too."""
        _here(self.device, self._index)
        norm = _empty(1, _F32, self.device, stream) if norm is None else norm
        factor = _empty(1, _F32, self.device, stream) if factor is None else factor
        np_, fp = _scalar(norm, self.device, "norm"), _scalar(factor, self.device, "factor")
        handle = _handle(stream, self._index)
        with _scratch_lock:
            ws = _scratch_for(self._nbytes, self.device, self._index, stream, handle)
            st = self._call(self._list, len(self.grads), max_norm, np_, fp, ws.data_ptr(),
                            self._nbytes, handle)
        if st:
            raise MoEError(st, "moe_grad_norm")
        return norm, factor


class AdamW:
    """AdamW over a list of parameters, one launch a step.

    params, grads: contiguous float32 or bfloat16 tensors of one device, a
    gradient of the same size for every parameter (its type may differ).  They
    are the caller's and are kept alive here: a step reads the gradients that
    the buffers hold then, and writes the parameters in place.
    masters: None; True, for a float32 copy of every bfloat16 parameter, made
    here; or a list of float32 tensors (entries may be None).  Where there is a
    master the step updates it, and the parameter becomes its rounding.
    state: float32, or float8_e4m3fn for 8-bit states with a scale for every
    256 values (the layout is moe_adamw_step's in include/moe.h).
    rounding, of 8-bit states: "random" (unbiased, from the step's number: the
    moments follow their recurrences on average, and steps repeat themselves) or
    "nearest", which loses what moves a moment by less than 3 to 6 % a step: v
    stays too large where betas[1] is near 1, and parameters whose gradient is
    zero keep moving beside others whose is not.  None: random where betas[1] is
    above 31/32, else nearest.
    weight_decay: one number, or one for every parameter.

    m, v: (blocks, 256) of the state type, the parameters' states one behind
    the other, each beginning a block (offsets: their first blocks; what lies
    behind a parameter's end is never read or written); m_scale, v_scale:
    (blocks,) float32 or None.  8-bit v holds the root of the second moment.

    Steps on one object, and steps that are captured in graphs, are ordered by
    the caller.  The number of steps is kept on the device: a captured step
    counts on at each replay.
    """

    def __init__(self, params, grads, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01,
                 state=_F32, masters=None, rounding=None):
        self.params, self.grads = _tensors(params, "params"), _tensors(grads, "grads")
        n, dev = len(self.params), self.params[0].device
        _want(len(self.grads) == n and self.grads[0].device == dev
              and all(g.shape == p.shape for p, g in zip(self.params, self.grads)),
              "grads: one of the same shape for every parameter, on their device")
        _want(state in (_F32, _E4M3), "state: float32 or float8_e4m3fn")
        _want(rounding in (None, "nearest", "random"), "rounding: None, 'nearest' or 'random'")
        _want(rounding is None or state == _E4M3, "rounding: of float8_e4m3fn states")
        decay = [float(weight_decay)] * n if isinstance(weight_decay, (int, float)) else [
            float(d) for d in weight_decay]
        _want(len(decay) == n, "weight_decay: a number, or one for every parameter")
        if masters is None or masters is True:
            masters = [p.detach().float() if masters and p.dtype == _BF16 else None
                       for p in self.params]
        self.masters = list(masters)
        _want(len(self.masters) == n and all(
            w is None or (w.dtype == _F32 and w.shape == p.shape and w.is_contiguous()
                          and w.device == dev) for p, w in zip(self.params, self.masters)),
              "masters: a contiguous float32 tensor of its shape, or None, for every parameter")
        span = lambda t: (t.data_ptr(), t.data_ptr() + t.numel() * t.element_size())  # noqa: E731
        written = sorted(span(t) for t in self.params + [w for w in self.masters if w is not None]
                         if t.numel())
        _want(all(a[1] <= b[0] for a, b in zip(written, written[1:])),
              "params and masters: no two may share memory")
        ends = [b for _, b in written]
        for a, b in (span(g) for g in self.grads if g.numel()):
            i = bisect.bisect_right(ends, a)  # the first that ends behind the gradient's beginning
            _want(i == len(written) or b <= written[i][0],
                  "grads: none may share memory with a parameter or a master")
        self.lr, self.betas, self.eps = float(lr), (float(betas[0]), float(betas[1])), float(eps)
        _want(all(0 <= b < 1 for b in self.betas) and 2.0 ** -126 <= self.eps < math.inf
              and all(0 <= d < math.inf for d in [self.lr] + decay),
              "betas in [0, 1), eps at least 2^-126, lr and weight_decay at least 0, all finite")
        self.state, self.device, self._index = state, dev, _index(dev)
        self.rounding = rounding
        blocks = [-(-p.numel() // BLOCK) for p in self.params]
        *self.offsets, total = itertools.accumulate(blocks, initial=0)
        zeros = lambda *shape: torch.zeros(shape, dtype=_F32 if state == _F32 else torch.uint8,  # noqa: E731
                                           device=dev).view(state)
        self.m, self.v = zeros(total, BLOCK), zeros(total, BLOCK)
        self.m_scale = self.v_scale = None
        if state != _F32:
            self.m_scale, self.v_scale = (torch.zeros(total, device=dev) for _ in range(2))
        size, e = BLOCK * self.m.element_size(), state != _F32
        self._list = (_lib.AdamWTensor * n)(*[
            _lib.AdamWTensor(p.data_ptr(), _p(w), g.data_ptr(), self.m.data_ptr() + b * size,
                             self.v.data_ptr() + b * size,
                             self.m_scale.data_ptr() + 4 * b if e else None,
                             self.v_scale.data_ptr() + 4 * b if e else None, p.numel(),
                             _DT[p.dtype], _DT[g.dtype], d)
            for p, w, g, b, d in zip(self.params, self.masters, self.grads, self.offsets, decay)])
        self._step = _lib.load().moe_adamw_step
        self.step_state = torch.zeros(_lib.ADAMW_STATE_BYTES, dtype=torch.uint8, device=dev)
        self._set_steps(0)

    def _desc(self, lr, lr_device, scale):
        return _lib.AdamWDesc(_DT[self.state], lr, lr_device, scale, *self.betas, self.eps,
                              _lib.ROUNDING[self.rounding])

    def _set_steps(self, steps):
        decode._ready(self.device)
        _check(_lib.load().moe_adamw_set_steps(*self.betas, steps, _p(self.step_state),
                                               _handle(None, self._index)), "moe_adamw_set_steps")
        kept = [t for t in (self.m, self.v, self.m_scale, self.v_scale, self.step_state)
                if t is not None] + [w for w in self.masters if w is not None]
        # a stream's first step waits for what was enqueued here
        self._streams = _Workspaces(self.device, lambda: self.step_state, kept)

    def step(self, lr=None, grad_scale=None, stream=None):
        """One step with the gradients that the buffers hold.  lr: a number, or
        one float32 on the device (read when the step runs, so a captured step
        may be replayed with another), the constructor's when None.
        grad_scale: one float32 on the device that multiplies the gradients
        (GradNorm's factor), or None."""
        lp = None
        if lr is None:
            lr = self.lr
        elif isinstance(lr, torch.Tensor):
            lp, lr = _scalar(lr, self.device, "lr"), 0.0
        gp = _scalar(grad_scale, self.device, "grad_scale")
        _here(self.device, self._index)
        handle = _handle(stream, self._index)
        if handle not in self._streams.pointers:
            self._streams.add(handle)
        st = self._step(ctypes.byref(self._desc(lr, lp, gp)), self._list, len(self.params),
                        self.step_state.data_ptr(), handle)
        if st:
            raise MoEError(st, "moe_adamw_step")

    @property
    def steps(self):
        """Steps taken (waits for the device, whatever stream the steps ran on)."""
        torch.cuda.synchronize(self.device)
        return int(self.step_state[:8].view(torch.int64).item())

    def state_dict(self):
        """The states (the object's own tensors), the number of steps (waits for
        the device) and the masters."""
        return {"steps": self.steps, "m": self.m, "v": self.v, "m_scale": self.m_scale,
                "v_scale": self.v_scale, "masters": self.masters}

    def load_state_dict(self, d):
        """Copies states and the number of steps, and masters where d has them,
        on the current stream."""
        steps = int(d["steps"])
        _want(0 <= steps < 2 ** 63, "steps: a number of steps")
        for name in ("m", "v", "m_scale", "v_scale"):
            to, src = getattr(self, name), d[name]
            _want((to is None) == (src is None) and (to is None or (
                src.dtype == to.dtype and src.shape == to.shape)), f"{name}: another shape or type")
        masters = d.get("masters")
        _want(masters is None or (len(masters) == len(self.masters) and all(
            (a is None) == (b is None) and (a is None or a.shape == b.shape)
            for a, b in zip(masters, self.masters))), "masters: other shapes")
        for name in ("m", "v", "m_scale", "v_scale"):
            if d[name] is not None:  # the bits move
                getattr(self, name).view(torch.uint8).copy_(d[name].contiguous().view(torch.uint8))
        for to, src in zip(self.masters, masters or []):
            if to is not None:
                to.copy_(src)
        self._set_steps(steps)


class MoEBlock:
    """A residual block for training: s = x + residual; out = experts(norm(s)),
    with the layer's own forward and backward calls on buffers kept here.

    desc: a bf16 layer (make_desc; H % 256 == 0, row-major weights); norm: a
    LayerNorm of bf16 rows; w_gate (H, E), w13 (E, H, 2I), w2 (E, I, H)
    bfloat16, bias (E,) float32 or None.
    params and grads: the block's parameters and their float32 gradients, in
    one order, as AdamW and GradNorm take them; backward overwrites the
    gradients.  One forward's intermediates are kept, for the backward that
    follows it; calls of one block are ordered by the caller.  Torch's automatic
    differentiation does not see them.
    """

    def __init__(self, desc, norm, w_gate, bias, w13, w2):
        _want(norm.dtype == _BF16 and norm.H == desc.H, "norm: of bfloat16 rows of the layer's H")
        nbytes = api.moe_backward_workspace_size(desc)
        _want(nbytes > 0 and not desc.weight_layout,
              "desc: a bf16 layer that moe_backward takes, row-major weights")
        self.desc, self.norm = desc, norm
        self.w_gate, self.bias, self.w13, self.w2 = w_gate, bias, w13, w2
        n, H, I, E, K = desc.n, desc.H, desc.I, desc.E, desc.K
        dev = w13.device
        for t, shape, dt, name in ((w_gate, (H, E), _BF16, "w_gate"), (bias, (E,), _F32, "bias"),
                                   (w13, (E, H, 2 * I), _BF16, "w13"), (w2, (E, I, H), _BF16, "w2")):
            _want(t is None and name == "bias" or (
                t.dtype == dt and t.shape == shape and t.is_contiguous() and t.device == dev),
                f"{name}: contiguous {shape} {dt}")
        _want(norm.device == dev, "all tensors on one device")
        decode._ready(dev)
        new = lambda *shape, dtype=_I32: torch.empty(shape, dtype=dtype, device=dev)  # noqa: E731
        self.stats = new(2, n, dtype=_F32)
        self.h_in, self.s = new(n, H, dtype=_BF16), new(n, H, dtype=_BF16)
        self.logits, self.topk_w = new(n, E, dtype=_F32), new(n, K, dtype=_F32)
        self.topk_idx, self.counts, self.offsets = new(n, K), new(E), new(E + 1)
        self.perm, self.inv_perm = new(n * K), new(n * K)
        self.x_perm, self.y_perm = new(n * K, H, dtype=_BF16), new(n * K, H, dtype=_BF16)
        self.h = new(n * K, I, dtype=_BF16)
        self.d_in = new(n, H, dtype=_BF16)
        self.status = torch.zeros(1, dtype=_I32, device=dev)
        self._layout_ws = new(max(api.moe_layout_workspace_size(desc), 1), dtype=torch.uint8)
        self._ws = new(nbytes, dtype=torch.uint8)
        zeros = lambda t: torch.zeros(t.shape, dtype=_F32, device=dev)  # noqa: E731
        self.params = [t for t in (norm.weight, norm.bias, w_gate, bias, w13, w2) if t is not None]
        self._grads = {name: None if t is None else zeros(t) for name, t in (
            ("norm", norm.weight), ("norm_bias", norm.bias), ("w_gate", w_gate), ("bias", bias),
            ("w13", w13), ("w2", w2))}
        self.grads = [g for g in self._grads.values() if g is not None]
        self._rows = None  # what the last forward normalised
        kept = [t for t in vars(self).values() if isinstance(t, torch.Tensor)] + self.grads
        # a stream's first call waits for what was enqueued here
        self._index = _index(dev)
        self._streams = _Workspaces(dev, lambda: self._ws, kept)

    def _enter(self, stream):
        _here(self.status.device, self._index)
        handle = _handle(stream, self._index)
        if handle not in self._streams.pointers:
            self._streams.add(handle)

    def forward(self, x, residual=None, out=None, stream=None):
        """(out, s) for x (n, H) bfloat16 and residual like it, or None (then s
        is x).  out is allocated when not given; s is a buffer of the block
        where there is a residual, and holds until the next forward; backward
        reads it (or x, which then must not change meanwhile).  out shares no
        memory with them."""
        d = self.desc
        _want(out is None or (out.shape == self.h_in.shape and out.dtype == _BF16
                              and out.is_contiguous() and out.device == self.h_in.device),
              "out: like x, contiguous")
        _want(out is None or _apart(out, (x, residual, self.s, self.h_in)),
              "out: shares memory with x, residual or a buffer of the block")
        self._enter(stream)
        if residual is None:
            self.norm(x, y=self.h_in, stats=self.stats, stream=stream)
            rows = x
        else:
            self.norm(x, residual, y=self.h_in, s=self.s, stats=self.stats, stream=stream)
            rows = self.s
        self._rows = None  # until the call's last kernel is enqueued
        if out is None:
            out = _empty(x.shape, _BF16, x.device, stream)
        api.moe_route_topk(d, self.h_in, self.w_gate, self.bias, self.topk_idx, self.topk_w,
                           self.logits, stream)
        api.moe_dispatch_layout(d, self.topk_idx, self.counts, self.offsets, self.perm,
                                self.inv_perm, self.status, self._layout_ws, stream)
        api.moe_permute(d, self.h_in, self.perm, self.x_perm, self.status, stream)
        api.moe_expert_gemm1_swiglu(d, self.x_perm, self.w13, self.offsets, self.h,
                                    status_word=self.status, stream=stream)
        api.moe_expert_gemm2(d, self.h, self.w2, self.offsets, self.y_perm,
                             status_word=self.status, stream=stream)
        api.moe_combine(d, self.y_perm, self.topk_w, self.inv_perm, out, self.status, stream)
        self._rows = rows
        return out, rows

    def backward(self, dout, ds=None, dx=None, stream=None):
        """dx (n, H): the gradient of x, and of residual alike, for dout = dL/dout
        and ds = dL/ds by other ways (None: there are none).  Fills the gradients."""
        g = self._grads
        _want(self._rows is not None, "backward before a forward")
        _want(dout.dtype == _BF16 and dout.shape == self.h_in.shape and dout.is_contiguous()
              and dout.device == self.h_in.device, "dout: like out, contiguous")
        if ds is not None:  # the norm's checks, before the first kernel
            stride = self.norm._rows(ds, self.h_in.shape, "ds")[1]
            _want(self.desc.n < 2 or stride >= self.desc.H, "ds: rows that do not overlap")
        if dx is not None:
            self.norm._out(dx, self.h_in.shape, _BF16, "dx")
            _want(_apart(dx, (self.d_in, self._rows)),
                  "dx: shares memory with the rows of the forward or a buffer of the block")
        self._enter(stream)
        api.moe_backward(self.desc, self.h_in, self.w_gate, self.w13, self.w2, dout, self.logits,
                         self.topk_idx, self.topk_w, self.offsets, self.inv_perm, self.x_perm,
                         self.h, self.y_perm, self.d_in, g["w_gate"], g["bias"], g["w13"], g["w2"],
                         self._ws, self.status, stream)
        return self.norm.backward(self.d_in, self._rows, self.stats, ds=ds, dx=dx,
                                  dweight=g["norm"], dbias=g["norm_bias"], stream=stream)[0]

    def check(self, stream=None):
        """Waits for the stream (the calls' one) and raises MoEError if a call
        flagged bad routing, an inconsistent layout or a timeout."""
        decode._ready(self.status.device)
        _check(api.moe_check_status(self.status, stream), "device status")
