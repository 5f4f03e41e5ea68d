"""Refusals of the serving calls: every bad argument is answered before any
CUDA call, through the C ABI (fake pointers, never dereferenced) and through
the Python classes (CPU tensors).  No GPU needed."""
import contextlib
import ctypes
import math
import os
import shutil
import threading
import types

import pytest
import torch

pytestmark = pytest.mark.skipif(
    not (shutil.which("nvcc") or os.path.exists("/usr/local/cuda/bin/nvcc")),
    reason="CUDA toolkit not installed")

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
P = 1 << 20          # a fake, well aligned pointer
BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def lib():
    from top_routing_dispatch_gb300 import build as B
    B.build()
    from top_routing_dispatch_gb300 import _lib
    return _lib.load()


def cache(**kw):
    from top_routing_dispatch_gb300._lib import KVCacheDesc
    d = dict(num_seqs=4, q_heads=8, kv_heads=2, head_dim=128, page_size=16, num_pages=10,
             max_pages=5, dtype=1, cache_dtype=1, rope_rows=0, rope_dim=0, rope_interleaved=0,
             page_stride=2 * 16 * 128, k_cache=P, v_cache=P, page_table=P, k_scale=None,
             v_scale=None, rope=None)
    d.update(kw)
    return KVCacheDesc(**d)


BAD_CACHES = [
    (dict(num_seqs=-1), INVALID), (dict(q_heads=0), INVALID), (dict(kv_heads=0), INVALID),
    (dict(q_heads=7), INVALID), (dict(head_dim=0), INVALID), (dict(page_size=0), INVALID),
    (dict(max_pages=0), INVALID), (dict(num_pages=-1), INVALID), (dict(dtype=2), INVALID),
    (dict(dtype=5), INVALID), (dict(cache_dtype=0), INVALID),
    (dict(dtype=0, cache_dtype=2), INVALID), (dict(k_scale=P), INVALID),
    (dict(rope_dim=128), INVALID), (dict(rope=P, rope_rows=8), INVALID),
    (dict(rope=P, rope_rows=8, rope_dim=144), INVALID), (dict(rope_rows=-1), INVALID),
    (dict(page_stride=2 * 16 * 128 - 16), INVALID),
    (dict(head_dim=96, page_stride=1 << 20), UNSUPPORTED), (dict(page_size=8), UNSUPPORTED),
    (dict(page_size=24, page_stride=1 << 20), UNSUPPORTED),
    (dict(rope=P, rope_rows=8, rope_dim=24), UNSUPPORTED),
    (dict(page_stride=2 * 16 * 128 + 8), UNSUPPORTED), (dict(num_seqs=65537), UNSUPPORTED),
]
BAD_MEMORY = [dict(k_cache=None), dict(v_cache=None), dict(page_table=None), dict(k_cache=P + 8),
              dict(v_cache=P + 4), dict(page_table=P + 2),
              dict(rope=P + 4, rope_rows=8, rope_dim=64)]


def append(lib, c=None, n=3, q=P, qs=1024, k=P, ks=256, v=P, vs=256, seq=P, pos=P, out=P):
    c = cache() if c is None else c
    return lib.moe_kv_append(ctypes.byref(c), n, q, qs, k, ks, v, vs, seq, pos, out, None, None)


def attend(lib, c=None, q=P, qs=1024, lens=P, window=0, scale=1.0, out=P, lse=None, ws=P,
           nbytes=1 << 40):
    c = cache() if c is None else c
    return lib.moe_paged_attention(ctypes.byref(c), q, qs, lens, window, scale, out, lse, ws,
                                   nbytes, None, None)


@pytest.mark.parametrize("bad,code", BAD_CACHES, ids=lambda v: str(v)[:40])
def test_bad_cache_descriptions(lib, bad, code):
    c = cache(**bad)
    assert append(lib, c) == code and attend(lib, c) == code
    assert append(lib, c, n=0) == code
    assert lib.moe_paged_attention_workspace_size(ctypes.byref(c)) == 0


@pytest.mark.parametrize("bad", BAD_MEMORY, ids=str)
def test_bad_cache_memory(lib, bad):
    assert append(lib, cache(**bad)) == INVALID
    assert attend(lib, cache(**bad)) == INVALID


def test_null_descriptions(lib):
    null = ctypes.POINTER(type(cache()))()
    assert lib.moe_kv_append(null, 1, P, 0, P, 0, P, 0, P, P, P, None, None) == INVALID
    assert lib.moe_paged_attention(null, P, 0, P, 0, 1.0, P, None, P, 1, None, None) == INVALID
    assert lib.moe_paged_attention_workspace_size(null) == 0
    assert lib.moe_experts_w4_workspace_size(None) == 0
    assert lib.moe_w4_tiled_bytes(None, 64, 0) == 0


def test_append_refusals(lib):
    assert append(lib, n=-1) == INVALID
    assert append(lib, n=0, q=None, k=None, v=None, seq=None, pos=None, out=None) == 0
    for kw in (dict(k=None), dict(v=None), dict(seq=None), dict(pos=None), dict(q=None),
               dict(out=None), dict(q=P + 8), dict(k=P + 2), dict(v=P + 8), dict(out=P + 8),
               dict(seq=P + 1), dict(pos=P + 2), dict(qs=1016), dict(qs=1028), dict(ks=128),
               dict(vs=260), dict(q=P, out=P, qs=2048)):
        assert append(lib, **kw) == INVALID, kw


def test_attend_refusals(lib):
    need = lib.moe_paged_attention_workspace_size(ctypes.byref(cache()))
    assert need > 0 and need % 256 == 0
    assert attend(lib, nbytes=need - 1) == WORKSPACE
    assert attend(lib, cache(num_seqs=0), q=None, lens=None, out=None, ws=None) == 0
    for kw in (dict(q=None), dict(lens=None), dict(out=None), dict(ws=None), dict(q=P + 8),
               dict(out=P + 4), dict(lse=P + 2), dict(lens=P + 2), dict(ws=P + 128),
               dict(window=-1), dict(scale=0.0), dict(scale=-1.0), dict(scale=math.nan),
               dict(scale=math.inf), dict(qs=1000), dict(qs=1025)):
        assert attend(lib, **kw) == INVALID, kw


def desc(**kw):
    import top_routing_dispatch_gb300 as M
    d = dict(n=4, H=256, I=128, E=8, K=2, dtype="bf16", norm_topk_prob=False)
    d.update(kw)
    return M.make_desc(**d)


def experts(lib, d=None, group=64, ptrs=(P,) * 6, ws=P, nbytes=1 << 40):
    d = desc() if d is None else d
    return lib.moe_experts_w4(ctypes.byref(d), group, *ptrs, ws, nbytes, None, None)


def test_experts_refusals(lib):
    d = desc()
    need = lib.moe_experts_w4_workspace_size(ctypes.byref(d))
    assert need > 0 and need % 256 == 0
    assert experts(lib, nbytes=need - 1) == WORKSPACE
    for g in (0, 16, 48, 256, -64):
        assert experts(lib, group=g) == UNSUPPORTED
        assert lib.moe_w4_tiled_bytes(ctypes.byref(d), g, 0) == 0
        assert lib.moe_prepare_weights_w4(ctypes.byref(d), g, *[P] * 6, None) == UNSUPPORTED
        assert lib.moe_quantize_weights_w4(ctypes.byref(d), g, *[P] * 6, None) == UNSUPPORTED
    for kw in (dict(dtype="f32"), dict(H=192), dict(I=192), dict(n=2049), dict(E=300)):
        assert experts(lib, desc(**kw)) == UNSUPPORTED, kw
    for kw in (dict(n=-1), dict(K=9), dict(E=0)):
        assert experts(lib, desc(**kw)) == INVALID, kw
    for i in range(6):
        for bad in (None, P + 2):
            assert experts(lib, ptrs=[bad if j == i else P for j in range(6)]) == INVALID
            if bad is None or i < 6:
                args = [None if j == i else P for j in range(6)]
                assert lib.moe_prepare_weights_w4(ctypes.byref(d), 64, *args, None) == INVALID
                assert lib.moe_quantize_weights_w4(ctypes.byref(d), 64, *args, None) == INVALID
    assert experts(lib, ws=None) == INVALID and experts(lib, ws=P + 16) == INVALID
    assert experts(lib, desc(n=0), ptrs=(None,) * 6, ws=None) == 0
    # 16 rows x 128 codes and their scales
    assert lib.moe_w4_tiled_bytes(ctypes.byref(d), 64, 0) == 8 * 16 * 2 * (1024 + 64)
    assert lib.moe_w4_tiled_bytes(ctypes.byref(d), 32, 1) == 8 * 16 * 1 * (1024 + 128)
    assert lib.moe_w4_tiled_bytes(ctypes.byref(d), 64, 2) == 0


def test_status_string(lib):
    assert lib.moe_status_string(8) != b"unknown status"
    assert lib.moe_status_string(9) == b"unknown status"


# ------------------------------------------------------------ Python classes
def kv(pages=6, heads=2, page=16, dim=64, dt=BF16):
    return torch.zeros((pages, heads, page, dim)).to(dt)


def make(**kw):
    import top_routing_dispatch_gb300 as M
    a = dict(k_cache=kv(), v_cache=kv(), page_table=torch.zeros((3, 2), dtype=torch.int32), q_heads=4)
    a.update(kw)
    return M.PagedKVCache(**a)


def test_cache_constructor_refusals(lib):
    import top_routing_dispatch_gb300 as M
    make()
    for kw in (dict(v_cache=kv(pages=7)), dict(v_cache=kv(dt=F32)), dict(k_cache=kv()[0]),
               dict(k_cache=kv(dt=torch.float16), v_cache=kv(dt=torch.float16)),
               dict(k_cache=kv(heads=4)[:, ::2], v_cache=kv(heads=4)[:, ::2]),
               dict(k_cache=kv(heads=3)[:, :2]),  # further apart than v_cache's
               dict(page_table=torch.zeros((3, 2))), dict(page_table=torch.zeros(3, dtype=torch.int32)),
               dict(page_table=torch.zeros((3, 4), dtype=torch.int32)[:, ::2]),
               dict(k_scale=torch.ones(3)), dict(rope=torch.zeros((8, 64), dtype=torch.float64)),
               dict(rope=torch.zeros((8, 128))[:, ::2])):
        with pytest.raises(ValueError):
            make(**kw)
    for kw in (dict(q_heads=3), dict(k_cache=kv(dim=96), v_cache=kv(dim=96)),
               dict(k_cache=kv(page=8), v_cache=kv(page=8)), dict(k_scale=torch.ones(2)),
               dict(rope=torch.zeros((8, 24)))):
        with pytest.raises(M.MoEError):
            make(**kw)


def test_cache_call_refusals(lib):
    c = make()
    n = 3
    good = dict(q=torch.zeros((n, 4, 64), dtype=BF16), k=torch.zeros((n, 2, 64), dtype=BF16),
                v=torch.zeros((n, 2, 64), dtype=BF16), seq_ids=torch.zeros(n, dtype=torch.int32),
                positions=torch.zeros(n, dtype=torch.int32))
    wide = torch.zeros((n, 2, 128), dtype=BF16)
    for kw in (dict(q=good["k"]), dict(k=good["q"]), dict(v=good["v"][:2]), dict(q=good["q"].float()),
               dict(k=wide[:, :, ::2]), dict(v=torch.zeros((n, 4, 64), dtype=BF16)[:, ::2]),
               dict(seq_ids=torch.zeros(n)), dict(positions=torch.zeros(n + 1, dtype=torch.int32)),
               dict(positions=torch.zeros(2 * n, dtype=torch.int32)[::2]),
               dict(q_out=good["q"].float()), dict(q=None, q_out=good["q"]),
               dict(q_out=torch.zeros((n, 5, 64), dtype=BF16)[:, :4])):
        with pytest.raises(ValueError):
            c.append(**{**good, **kw})
    q, lens = good["q"], torch.ones(3, dtype=torch.int32)
    for kw in (dict(q=q[:2]), dict(q=q.float()), dict(seq_lens=lens.long()), dict(seq_lens=lens[:2]),
               dict(out=q.float()), dict(out=torch.zeros((n, 5, 64), dtype=BF16)[:, :4]),
               dict(lse=torch.zeros((3, 2))), dict(lse=torch.zeros((3, 4), dtype=BF16))):
        with pytest.raises(ValueError):
            c.attend(**{**dict(q=q, seq_lens=lens), **kw})


def w4(E=2, H=128, I=128, g=64):
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    b = lambda *s: torch.zeros(s, dtype=BF16)  # noqa: E731
    return [i(E, 2 * I, H // 8), b(E, 2 * I, H // g), i(E, H, I // 8), b(E, H, I // g)]


def test_experts_constructor_refusals(lib):
    import top_routing_dispatch_gb300 as M
    for change in ({0: w4()[0].float()}, {1: w4()[1].float()}, {2: w4(I=256)[2]}, {3: w4(g=32)[3]},
                   {0: w4()[0][0]}, {1: w4()[1][:, :, :0]}, {0: w4(H=256)[0][:, :, ::2]}):
        t = w4()
        for k, v in change.items():
            t[k] = v
        with pytest.raises(ValueError):
            M.W4Experts(*t, K=1, max_tokens=4)
    for t, kw in ((w4(g=16), {}), (w4(), dict(K=3)), (w4(H=64), {}), (w4(), dict(max_tokens=5000))):
        with pytest.raises(M.MoEError):
            M.W4Experts(*t, **{**dict(K=1, max_tokens=4), **kw})
    with pytest.raises(ValueError):
        M.quantize_weights_w4(torch.zeros((2, 128, 256)), torch.zeros((2, 128, 128)))
    with pytest.raises(ValueError):
        M.quantize_weights_w4(torch.zeros((2, 128, 256), dtype=BF16), torch.zeros((2, 64, 128), dtype=BF16))
    with pytest.raises(M.MoEError):
        M.quantize_weights_w4(torch.zeros((2, 128, 256), dtype=BF16),
                              torch.zeros((2, 128, 128), dtype=BF16), group=48)


def test_rope_table():
    import top_routing_dispatch_gb300 as M
    t = M.rope_table(50, 16, base=100.0, device="cpu")
    assert t.shape == (50, 16) and t.dtype is F32
    for p in (0, 1, 49):
        for i in range(8):
            a = p * 100.0 ** (-2 * i / 16)
            assert abs(float(t[p, i]) - math.cos(a)) < 1e-6
            assert abs(float(t[p, 8 + i]) - math.sin(a)) < 1e-6


def test_experts_refuse_sizes_past_32_bits(lib):
    """2 I columns are counted in 32 bits."""
    d = desc(H=128, I=1 << 30, E=1, K=1, n=1)
    for which in (0, 1):
        assert lib.moe_w4_tiled_bytes(ctypes.byref(d), 128, which) == 0
    assert lib.moe_experts_w4_workspace_size(ctypes.byref(d)) == 0
    assert experts(lib, d, group=128) == UNSUPPORTED
    assert lib.moe_prepare_weights_w4(ctypes.byref(d), 128, *[P] * 6, None) == UNSUPPORTED
    assert lib.moe_quantize_weights_w4(ctypes.byref(d), 128, *[P] * 6, None) == UNSUPPORTED
    d = desc(H=128, I=(1 << 30) - 128, E=1, K=1, n=1)
    assert lib.moe_w4_tiled_bytes(ctypes.byref(d), 128, 0) == ((1 << 31) - 256) // 16 * 1056


# ------------------------------------------------------------------ devices
def calls():
    """Every Python call that launches, on CPU tensors that are right otherwise."""
    import top_routing_dispatch_gb300 as M
    n, c = 3, make()
    q, kv3 = torch.zeros((n, 4, 64), dtype=BF16), torch.zeros((n, 2, 64), dtype=BF16)
    ints = torch.zeros(n, dtype=torch.int32)
    return {
        "append": lambda: c.append(q, kv3, kv3, ints, ints, q_out=q.clone()),
        "attend": lambda: c.attend(q, ints, out=q.clone()),
        "check": lambda: c.check(),
        "experts": lambda: M.W4Experts(*w4(), K=1, max_tokens=4),
        "quantize": lambda: M.quantize_weights_w4(torch.zeros((2, 128, 256), dtype=BF16),
                                                  torch.zeros((2, 128, 128), dtype=BF16), group=64),
    }


@pytest.mark.parametrize("name", ["append", "attend", "check", "experts", "quantize"])
def test_calls_refuse_tensors_that_are_not_on_a_gpu(lib, name):
    with pytest.raises(ValueError, match="CUDA"):
        calls()[name]()


def test_calls_refuse_a_device_that_is_not_current(lib, monkeypatch):
    """The library launches on the current device."""
    from top_routing_dispatch_gb300 import decode
    monkeypatch.setattr(decode, "_current_device", lambda: 0)
    decode._ready(torch.device("cuda", 0))
    with pytest.raises(ValueError, match="current"):
        decode._ready(torch.device("cuda", 1))
    seen = []

    class Reached(Exception):
        pass

    def ready(device):
        seen.append(device)
        raise Reached
    monkeypatch.setattr(decode, "_ready", ready)
    for call in calls().values():
        with pytest.raises(Reached):
            call()
    assert len(seen) == 5


def test_an_experts_call_asks_for_its_device(lib, monkeypatch):
    from top_routing_dispatch_gb300 import decode
    ex = object.__new__(decode.W4Experts)
    ex.H, ex.K, ex.max_tokens, ex.device, ex._index = 128, 1, 4, torch.device("cpu"), None
    x = torch.zeros((2, 128), dtype=BF16)
    idx, tw = torch.zeros((2, 1), dtype=torch.int32), torch.zeros((2, 1))
    for call in (lambda: ex(x, idx, tw, y=torch.zeros_like(x)), ex.check):
        with pytest.raises(ValueError, match="CUDA"):
            call()


# ------------------------------------------------------- threads and streams
def host_experts(monkeypatch, call):
    """A W4Experts whose launches go to `call`, for up to 8 tokens."""
    from top_routing_dispatch_gb300 import decode
    lib = types.SimpleNamespace(
        moe_w4_tiled_bytes=lambda *a: 64, moe_experts_w4_workspace_size=lambda *a: 256,
        moe_prepare_weights_w4=lambda *a: 0, moe_experts_w4=call)
    monkeypatch.setattr(decode._lib, "load", lambda: lib)
    monkeypatch.setattr(decode, "_ready", lambda device: None)
    monkeypatch.setattr(decode, "_handle", lambda stream, index: stream or 0)
    return decode.W4Experts(*w4(), K=1, max_tokens=8)


def expert_inputs(n):
    x = torch.zeros((n, 128), dtype=BF16)
    return dict(x=x, topk_idx=torch.zeros((n, 1), dtype=torch.int32), topk_w=torch.zeros((n, 1)),
                y=torch.zeros_like(x))


def test_two_threads_keep_their_token_counts(lib, monkeypatch):
    """A call's token count is its own, whatever other calls of the object do
    between its start and the library's reading of it."""
    seen, other, threads = {}, expert_inputs(7), []

    def call(ref, group, x, *rest):
        first = not seen
        seen.setdefault(x, None)
        if first:  # another call has begun meanwhile, as far as it gets
            threads.append(threading.Thread(target=lambda: ex(**other)))
            threads[0].start()
            threads[0].join(0.3)
        seen[x] = ref._obj.n
        return 0
    ex = host_experts(monkeypatch, call)
    mine = expert_inputs(2)
    ex(**mine)
    threads[0].join()
    assert seen[mine["x"].data_ptr()] == 2 and seen[other["x"].data_ptr()] == 7


def test_expert_calls_of_two_threads_do_not_interleave(lib, monkeypatch):
    """A call is two or three kernels on one workspace: another thread's must not
    come between them."""
    inside, most, gate = [0], [0], threading.Event()

    def call(*a):
        inside[0] += 1
        most[0] = max(most[0], inside[0])
        gate.wait(0.1)
        inside[0] -= 1
        return 0
    ex = host_experts(monkeypatch, call)
    threads = [threading.Thread(target=lambda: ex(**expert_inputs(3))) for _ in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert most[0] == 1


class FakeStream:
    """Stands for torch's stream objects where there is no GPU."""
    waits, recorded, capturing, inside = [], [], False, []

    def __init__(self, handle, device=None):
        self.cuda_stream = handle

    def wait_event(self, event):
        FakeStream.waits.append((self.cuda_stream, event))


@pytest.fixture
def fake_streams(monkeypatch):
    from top_routing_dispatch_gb300 import decode
    FakeStream.waits, FakeStream.recorded, FakeStream.capturing = [], [], False

    @contextlib.contextmanager
    def use(stream):
        FakeStream.inside.append(stream.cuda_stream)
        yield
        FakeStream.inside.pop()
    monkeypatch.setattr(torch.cuda, "ExternalStream", FakeStream)
    monkeypatch.setattr(torch.cuda, "stream", use)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: FakeStream(0))
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: FakeStream.capturing)
    monkeypatch.setattr(torch.Tensor, "record_stream",
                        lambda t, s: FakeStream.recorded.append((t.data_ptr(), s.cuda_stream)))
    monkeypatch.setattr(decode, "_ready", lambda device: None)
    monkeypatch.setattr(decode, "_handle", lambda stream, index: stream or 0)


def test_each_stream_has_a_workspace_of_its_own(lib, monkeypatch, fake_streams):
    """Two calls on two streams may run at the same time, and a stream's first
    call waits for what the constructor enqueued."""
    c = make()
    q, lens = torch.zeros((3, 4, 64), dtype=BF16), torch.ones(3, dtype=torch.int32)
    used = []
    c._attend = lambda *a: used.append((a[-1], a[8])) or 0
    for s in (None, 5, 6, 5, None, 6):
        c.attend(q, lens, out=q.clone(), stream=s)
    by = dict(used)
    assert len(set(by.values())) == 3 and used == [(s, by[s]) for s in (0, 5, 6, 5, 0, 6)]
    assert [s for s, _ in FakeStream.waits] == [5, 6]
    ints, kv3 = torch.zeros(3, dtype=torch.int32), torch.zeros((3, 2, 64), dtype=BF16)
    c._append = lambda *a: 0
    c.append(None, kv3, kv3, ints, ints, stream=7)  # its status word is the constructor's
    assert [s for s, _ in FakeStream.waits] == [5, 6, 7]
    assert (c.status.data_ptr(), 7) in FakeStream.recorded

    used.clear()
    ex = host_experts(monkeypatch, lambda *a: used.append((a[-1], a[8])) or 0)
    for s in (None, 5, 6, 5, None, 6):
        ex(**expert_inputs(3), stream=s)
    by = dict(used)
    assert len(set(by.values())) == 3 and used == [(s, by[s]) for s in (0, 5, 6, 5, 0, 6)]
    assert (ex.w13_t.data_ptr(), 5) in FakeStream.recorded


def test_a_capture_uses_the_first_workspace(lib, fake_streams):
    c = make()
    q, lens = torch.zeros((3, 4, 64), dtype=BF16), torch.ones(3, dtype=torch.int32)
    used = []
    c._attend = lambda *a: used.append(a[8]) or 0
    FakeStream.capturing = True
    c.attend(q, lens, out=q.clone(), stream=9)
    assert used == [c.ws.data_ptr()] and FakeStream.waits == []
    FakeStream.capturing = False
    c.attend(q, lens, out=q.clone(), stream=9)
    assert used[1] != used[0]


def test_results_are_allocated_on_the_calls_stream(lib, monkeypatch, fake_streams):
    made = []
    empty = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, **k: made.append(list(FakeStream.inside)) or empty(*a, **k))
    c = make()
    q, lens = torch.zeros((3, 4, 64), dtype=BF16), torch.ones(3, dtype=torch.int32)
    ints, kv3 = torch.zeros(3, dtype=torch.int32), torch.zeros((3, 2, 64), dtype=BF16)
    c._attend = c._append = lambda *a: 0
    for call in (lambda: c.attend(q, lens, stream=5),
                 lambda: c.append(q, kv3, kv3, ints, ints, stream=5)):
        made.clear()
        t = call()
        assert made == [[5]] and (t.data_ptr(), 0) in FakeStream.recorded


@pytest.mark.parametrize("bad", [None, P + 2, P + 8])
@pytest.mark.parametrize("i", range(6))
def test_weight_preparation_refuses_null_and_misaligned_pointers(lib, i, bad):
    d, args = desc(), [bad if j == i else P for j in range(6)]
    assert lib.moe_prepare_weights_w4(ctypes.byref(d), 64, *args, None) == INVALID
    assert lib.moe_quantize_weights_w4(ctypes.byref(d), 64, *args, None) == INVALID
