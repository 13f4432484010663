"""The scratch that a decode call without `workspace` takes: one buffer for each stream that calls run on, a graph's
own for captured calls, kept from everything else until the graph is gone."""
import gc
import math

import pytest
import torch

import paged_kv_cache_252_gb300 as pkv
import _int4 as i4
import _operators as op

pytestmark = pytest.mark.gpu
DEV = "cuda"
FORMS = ["decode", "varlen", "tree", "chunked"]


class Call:
    """A form of decode attention over a cache type; every call into an output of its own."""

    def __init__(self, form, kv, lens, n=3, hq=8, hkv=2, d=128, seed=0):
        g = torch.Generator(device=DEV)
        g.manual_seed(seed)
        self.form, self.kv, self.lens, self.n, S = form, kv, lens, n, len(lens)
        self.tables, blocks = i4.tables_for(lens, g, DEV)
        self.tables = self.tables.clamp(max=blocks - 1)
        make = i4.make_cache if kv == "int4" else lambda *a: op.make_cache(kv, *a)
        self.k, self.v, self.sc = make(blocks, hkv, d, g, DEV)
        self.q = torch.randn((S * n, hq, d), generator=g, device=DEV).to(op.src_dtype(kv))
        self.ctx = torch.tensor(lens, device=DEV, dtype=torch.int32)
        self.cu = torch.arange(0, S * n + 1, n, device=DEV, dtype=torch.int32)
        self.masks = i4.chain(n, DEV).repeat(S)
        self.scale = d ** -0.5

    def out(self):
        return torch.full_like(self.q, math.nan)

    def __call__(self, out=None, **kw):
        out = self.out() if out is None else out
        a = (self.k, self.v)
        if self.form == "chunked":
            return pkv.paged_attention_decode_chunked(out, self.q, [self.n] * len(self.lens), self.lens, *a, self.tables,
                                                      self.scale, self.kv, scales=self.sc, **kw)
        rest = (self.tables, self.ctx, self.n, self.scale)
        if self.form == "varlen":
            return pkv.paged_attention_decode_varlen(out, self.q, self.cu, *a, *rest, self.kv, scales=self.sc, **kw)
        if self.form == "tree":
            return pkv.paged_attention_decode_tree(out, self.q, self.masks, *a, *rest, self.kv, scales=self.sc, **kw)
        if self.kv == "int8":
            return pkv.paged_attention_decode_int8(out, self.q, *a, self.sc, *rest, **kw)
        if self.kv == "int4":
            return pkv.paged_attention_decode_int4(out, self.q, *a, self.sc, *rest, **kw)
        return pkv.paged_attention_decode(out, self.q, *a, *rest, self.kv, **kw)


def _pair(form, kv):
    return (Call(form, kv, [9000, 40, 700, 3], seed=1), Call(form, kv, [64, 12000, 5, 900, 333, 17], seed=2))


@pytest.mark.parametrize("kv", ["fp16", "int8", "int4"])
@pytest.mark.parametrize("form", FORMS)
def test_two_streams_given_by_name(form, kv):
    calls = _pair(form, kv)
    want = [c() for c in calls]
    streams = [torch.cuda.Stream() for _ in calls]
    outs = [[c.out() for _ in range(60)] for c in calls]
    torch.cuda.synchronize()
    for i in range(60):
        for c, o, s in zip(calls, outs, streams):
            c(o[i], stream=s)
    torch.cuda.synchronize()
    for w, o in zip(want, outs):
        assert all(torch.equal(x, w) for x in o)


@pytest.mark.parametrize("kv", ["fp16", "int8", "int4"])
@pytest.mark.parametrize("form", FORMS)
def test_a_stream_given_by_name_while_the_current_one_is_busy(form, kv):
    """A call's buffer is made (or grown) on the stream that the call runs on: nothing that waits on the current one
    touches it."""
    c = _pair(form, kv)[1]
    want = c()
    cur, s = torch.cuda.Stream(), torch.cuda.Stream()
    outs = [c.out() for _ in range(300)]
    torch.cuda.synchronize()
    with torch.cuda.stream(cur):
        torch.cuda._sleep(4_000_000)      # about 2 ms, while the calls on the other stream go on
        for o in outs:
            c(o, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)


@pytest.mark.parametrize("kv", ["fp16", "int8", "int4"])
@pytest.mark.parametrize("form", FORMS)
def test_a_captured_call_keeps_its_scratch(form, kv):
    """A larger call on the same stream, and tensors that take whatever memory is free then: the replayed call writes
    to none of them and none of them changes its result."""
    small = Call(form, kv, [4000, 30], seed=3)
    large = Call(form, kv, [5000] * 60, n=4, hq=32, hkv=4, seed=4)
    want, big = small(), large()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        small()
    torch.cuda.synchronize()
    g, out = torch.cuda.CUDAGraph(), small.out()
    with torch.cuda.graph(g, stream=s):
        small(out)
    with torch.cuda.stream(s):
        grown = large()
        free = [torch.full((n,), 0x5A, dtype=torch.uint8, device=DEV) for n in [1 << 10] * 40 + [1 << 18] * 20 + [3 << 20] * 20]
    torch.cuda.synchronize()
    for _ in range(3):
        out.fill_(math.nan)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    assert torch.equal(grown, big)
    assert all(bool((x == 0x5A).all()) for x in free)


@pytest.mark.parametrize("kv", ["fp16", "int8", "int4"])
@pytest.mark.parametrize("form", FORMS)
def test_two_graphs_of_one_stream_replayed_side_by_side(form, kv):
    calls = _pair(form, kv)
    want = [c() for c in calls]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graphs, outs = [], []
    for c in calls:
        g, out = torch.cuda.CUDAGraph(), [c.out() for _ in range(20)]
        with torch.cuda.graph(g, stream=s):
            for o in out:
                c(o)
        graphs.append(g)
        outs.append(out)
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    for _ in range(3):
        for o in sum(outs, []):
            o.fill_(math.nan)
        torch.cuda.synchronize()
        for g, r in zip(graphs, streams):
            with torch.cuda.stream(r):
                g.replay()
        torch.cuda.synchronize()
        for w, o in zip(want, outs):
            assert all(torch.equal(x, w) for x in o)


def test_a_graph_that_is_gone_gives_its_scratch_back():
    from paged_kv_cache_252_gb300 import api
    c = Call("decode", "fp16", [3000, 30], seed=5)
    s = torch.cuda.Stream()

    def capture():
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            c()
        return g
    def captured():
        before = set(api._captures)
        g = capture()
        g.replay()
        torch.cuda.synchronize()
        return g, set(api._captures) - before
    (g, held), (kept, live) = captured(), captured()
    assert len(held) == len(live) == 1 and held <= set(api._captures)
    del g
    gc.collect()
    for _ in range(50):      # (CUDA reports it some time later)
        torch.cuda.synchronize()
        g = capture()
        if not held & set(api._captures):
            break
        torch.cuda._sleep(10_000_000)
    assert not held & set(api._captures) and live <= set(api._captures)
    kept.replay()


def _epoch(n):
    """The tag of the process's n-th call with piece counters."""
    m = 0xFFFFFFFF
    n ^= n >> 16
    n = n * 0x7FEB352D & m
    n ^= n >> 15
    n = n * 0x846CA68B & m
    return n ^ n >> 16


def test_nodes_behind_a_captured_call_do_not_reach_its_counters():
    """The graph's own later tensors take the memory that the captured call gave back, if any, and fill it with words that
    are that call's counters to the letter, half counted."""
    c = Call("decode", "int4", [9000, 40, 700, 3], seed=6)
    want = c()
    need = pkv.api.load_library().pkv_decode_workspace_bytes(4, 8, 3, pkv.api._desc_of(c.k, c.v, True)[0])
    ws = torch.zeros(need, dtype=torch.uint8, device=DEV)
    c(workspace=ws)
    tag = {w >> 32 & 0xFFFFFFFF for w in ws[:256].view(torch.int64).tolist()} - {0}   # (a counter keeps its call's tag)
    n = next(n for n in range(1, 1 << 20) if {_epoch(n)} == tag)
    g, out = torch.cuda.CUDAGraph(), c.out()
    s = torch.cuda.Stream()
    with torch.cuda.graph(g, stream=s):
        c(out)
        later = [torch.empty(need // 8, dtype=torch.int64, device=DEV) for _ in range(4)]
        word = _epoch(n + 1) << 32 | 1
        for x in later:
            x.fill_(word - (1 << 64) if word >> 63 else word)
    for _ in range(4):
        out.fill_(math.nan)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
