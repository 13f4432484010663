"""Which scratch a decode call without `workspace` takes, on the host: streams, captures and the library are stand-ins, the
tensors lie in host memory."""
import contextlib
import ctypes
import weakref

import pytest
import torch

import paged_kv_cache_252_gb300 as pkv
from paged_kv_cache_252_gb300 import api


class Stream:
    def __init__(self, handle, capture=0):
        self.cuda_stream, self.capture = handle, capture


class Library:
    """Notes the workspace of every decode call, and which captures have ended."""

    def __init__(self, world):
        self.world = world

    def pkv_decode_workspace_bytes(self, S, Hq, n, desc):
        return 4096 * S

    def pkv_decode_counter_bytes(self, S, Hq, n, desc, code):
        return 256 * S

    def pkv_decode_chunked_workspace_bytes(self, ql, S, Hq, mbs, desc):
        return 8192 * S

    def pkv_capture_watch(self, stream, ident, watch):
        ctypes.cast(ident, ctypes.POINTER(ctypes.c_uint64))[0] = self.world.current.capture
        if watch is not None:
            ctypes.cast(watch, ctypes.POINTER(ctypes.c_void_p))[0] = self.world.current.capture
        return 0

    def pkv_capture_gone(self, watch):
        return int(watch in self.world.gone)

    def __getattr__(self, name):
        assert name.startswith("pkv_paged_attention_decode"), name

        def call(*args):
            at = [getattr(a, "value", a) for a in args]
            found = [(p, t(), stream) for p, (t, stream) in self.world.made if p in at and t() is not None]
            assert len(found) == 1, "no scratch, or two"
            p, ws, stream = found[0]
            counters = 256 * self.world.S
            self.world.calls.append((p, stream, not ws[:counters].any()))
            ws[counters:] = 0x77          # (the call's sums)
            return 0
        return call


class World:
    def __init__(self, monkeypatch):
        self.default = self.current = Stream(1)
        self.made, self.calls, self.gone = [], [], set()
        self.S = 0

        @contextlib.contextmanager
        def on(stream):
            was, self.current = self.current, stream
            try:
                yield
            finally:
                self.current = was

        def make(fn):
            def made(n, dtype=None, device=None):
                t = fn(n, dtype=dtype)
                self.made.append((t.data_ptr(), (weakref.ref(t), self.current)))
                return t
            return made
        self.on = on
        fake = type("torch_", (), {})()
        fake.__dict__.update(torch.__dict__)
        fake.empty, fake.zeros = make(torch.empty), make(torch.zeros)
        cuda = type("cuda_", (), {})()
        cuda.__dict__.update(torch.cuda.__dict__)
        cuda.stream = on
        cuda.current_stream = lambda device=None: self.current
        cuda.current_device = lambda: 0
        cuda.is_current_stream_capturing = lambda: self.current.capture != 0
        fake.cuda = cuda
        monkeypatch.setattr(api, "torch", fake)
        monkeypatch.setattr(api, "_lib", Library(self))
        monkeypatch.setattr(api, "_raw_stream", lambda dev: self.current.cuda_stream)
        monkeypatch.setattr(api, "_need_cuda_contig", lambda name, t: None)
        monkeypatch.setattr(api, "_on_device", lambda device: contextlib.nullcontext())
        monkeypatch.setattr(api, "_placed", lambda names, tensors: 0)
        monkeypatch.setattr(api, "_at", lambda dev: contextlib.nullcontext())
        for name in ("_scratches", "_captures", "_decode_sizes", "_workspaces", "_ws_bytes_cache", "_int4_workspaces", "_int4_ws_bytes"):
            if hasattr(api, name):
                monkeypatch.setattr(api, name, {})


@pytest.fixture
def world(monkeypatch):
    return World(monkeypatch)


def _call(world, form, kv, S=2, stream=None):
    world.S = S
    n, hq, hkv, d = 2, 4, 2, 64
    q = torch.zeros((S * n, hq, d), dtype=torch.float16)
    k, v = pkv.alloc_kv_cache(4, hkv, d, kv, "cpu") if kv != "fp16" else (torch.zeros((4, hkv, 16, d), dtype=torch.float16),) * 2
    sc = None if kv == "fp16" else torch.zeros((4, hkv, 2, 16) if kv == "int8" else (4, hkv, 2, 16, 1, 2),
                                               dtype=torch.float32 if kv == "int8" else torch.float16)
    bt, cl = torch.zeros((S, 2), dtype=torch.int32), torch.full((S,), 5, dtype=torch.int32)
    if form == "chunked":
        return pkv.paged_attention_decode_chunked(q, q, [n] * S, [5] * S, k, v, bt, 0.1, kv, scales=sc, stream=stream)
    if form == "varlen":
        cu = torch.arange(0, S * n + 1, n, dtype=torch.int32)
        return pkv.paged_attention_decode_varlen(q, q, cu, k, v, bt, cl, n, 0.1, kv, scales=sc, stream=stream)
    if form == "tree":
        masks = torch.ones(S * n, dtype=torch.int64)
        return pkv.paged_attention_decode_tree(q, q, masks, k, v, bt, cl, n, 0.1, kv, scales=sc, stream=stream)
    if kv == "fp16":
        return pkv.paged_attention_decode(q, q, k, v, bt, cl, n, 0.1, stream=stream)
    fn = pkv.paged_attention_decode_int8 if kv == "int8" else pkv.paged_attention_decode_int4
    return fn(q, q, k, v, sc, bt, cl, n, 0.1, stream=stream)


ALL = [(form, kv) for form in ("decode", "varlen", "tree", "chunked") for kv in ("fp16", "int8", "int4")]


@pytest.mark.parametrize("form,kv", ALL)
def test_scratch_goes_by_the_stream_the_call_runs_on(world, form, kv):
    s1, s2 = Stream(11), Stream(12)
    for s in (None, s1, s2, s1, None):
        _call(world, form, kv, stream=s)
    with world.on(s2):
        _call(world, form, kv)
    ptrs = [c[0] for c in world.calls]
    assert len({ptrs[0], ptrs[1], ptrs[2]}) == 3
    assert ptrs[3] == ptrs[1] and ptrs[4] == ptrs[0] and ptrs[5] == ptrs[2]
    assert [c[1].cuda_stream for c in world.calls] == [1, 11, 12, 11, 1, 12]   # made on that stream


@pytest.mark.parametrize("form,kv", ALL)
def test_a_captured_call_shares_its_scratch_with_its_graph_alone(world, form, kv):
    live = lambda p: next(t for q, (t, _) in reversed(world.made) if q == p)()
    eager = Stream(21)
    _call(world, form, kv, stream=eager)
    for capture in (7, 8):
        with world.on(Stream(21, capture)):
            _call(world, form, kv)
            _call(world, form, kv)
            _call(world, form, kv, S=3)      # one that needs more
    _call(world, form, kv, S=3, stream=eager)
    p = [c[0] for c in world.calls]
    assert p[1] == p[2] and p[4] == p[5]
    groups = [{p[0], p[7]}, {p[1], p[3]}, {p[4], p[6]}]
    assert all(not a & b for i, a in enumerate(groups) for b in groups[:i])
    assert all(live(x) is not None for x in (p[1], p[3], p[4], p[6]))    # held: nobody else gets that memory
    held = [weakref.ref(live(x)) for x in (p[1], p[3])]
    world.gone.add(7)                                                   # the first graph is destroyed
    with world.on(Stream(21, 9)):
        _call(world, form, kv)
    assert all(t() is None for t in held) and live(p[4]) is not None
    held = [weakref.ref(live(x)) for x in (p[4], p[6])]
    world.gone.add(8)
    _call(world, form, kv, S=3, stream=eager)                           # (nothing to make: not looked at)
    assert all(t() is not None for t in held)
    _call(world, form, kv, S=30, stream=eager)
    assert all(t() is None for t in held)


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("form,kv", [x for x in ALL if x[0] != "chunked"])   # (which clears its counters itself)
def test_counters_are_clear_before_every_call(world, form, kv, captured):
    """The sums of a call with fewer counters, and of a chunked one, lie where a later call's counters are."""
    with world.on(Stream(31, 5 if captured else 0)):
        for S in (8, 2, 5, 8, 1, 8):
            _call(world, form, kv, S=S)
        _call(world, "chunked", kv, S=3)
        _call(world, form, kv, S=4)
        calls = [c for i, c in enumerate(world.calls) if i != 6]
        assert len({c[0] for c in calls}) == 1 and all(c[2] for c in calls)


@pytest.mark.parametrize("form,kv", [x for x in ALL if x[0] != "chunked"])
def test_a_size_that_could_not_be_told_is_asked_for_again(world, form, kv, monkeypatch):
    with monkeypatch.context() as m:
        m.setattr(Library, "pkv_decode_workspace_bytes", lambda self, S, Hq, n, desc: 0)   # (a device error, say)
        _call(world, form, kv)
    _call(world, form, kv)
    ws = next(t for p, (t, _) in reversed(world.made) if p == world.calls[-1][0])()
    assert ws.shape[0] >= 2 * 4096


@pytest.mark.parametrize("form,kv", [x for x in ALL if x[0] != "chunked"])
def test_a_shape_that_the_library_refuses_gets_as_far_as_its_refusal(world, form, kv, monkeypatch):
    for name in ("pkv_decode_workspace_bytes", "pkv_decode_counter_bytes"):
        monkeypatch.setattr(Library, name, lambda self, *a: 0)
    world.S = 0
    _call(world, form, kv)
    assert len(world.calls) == 1


def test_counter_bytes_and_captures_on_the_host():
    from paged_kv_cache_252_gb300 import build
    lib = ctypes.CDLL(build.build())
    lib.pkv_decode_counter_bytes.restype = ctypes.c_size_t
    desc = lambda nb=8, bs=16, h=2, d=64: ctypes.byref(api._CacheDesc(nb, bs, h, d))
    for kv in range(4):
        assert lib.pkv_decode_counter_bytes(5, 8, 1, desc(), kv) == 256 and lib.pkv_decode_counter_bytes(33, 8, 4, desc(), kv) == 768
        assert lib.pkv_decode_counter_bytes(0, 8, 1, desc(), kv) == 0
    for bad in ((-1, 8, 1, desc(), 0), (5, 0, 1, desc(), 0), (5, 7, 1, desc(), 0), (5, 8, 0, desc(), 0), (5, 8, 17, desc(), 0),
                (5, 8, 1, None, 0), (5, 8, 1, desc(d=96), 0), (5, 8, 1, desc(bs=8), 0), (5, 8, 1, desc(nb=0), 0), (5, 8, 1, desc(), 5)):
        assert lib.pkv_decode_counter_bytes(*bad) == 0
    assert lib.pkv_capture_watch(None, None, None) == -1
    assert lib.pkv_capture_gone(None) == 0
