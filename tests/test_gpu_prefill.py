"""Attention of chunks of new tokens over the paged cache, against 64 bits."""
import numpy as np
import pytest
import torch

import _operators as op

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    return torch.device("cuda:0")


class Batch:
    def __init__(self, dev, kv, D, hq, hkv, ns, lens, seed=1, q_gain=1.0, extra_rows=0):
        g = torch.Generator(device=dev)
        g.manual_seed(seed)
        self.lens, self.ns = lens, ns
        self.cu_host = [int(x) for x in np.concatenate([[0], np.cumsum(ns)])]
        self.bt, total = op.tables(lens, g, dev)
        self.kc, self.vc, self.sc = op.make_cache(kv, total, hkv, D, g, dev)
        R = self.cu_host[-1] + extra_rows
        self.q = (torch.randn((R, hq, D), generator=g, device=dev) * q_gain).to(op.src_dtype(kv))
        self.cu = torch.tensor(self.cu_host, dtype=torch.int32, device=dev)
        self.cl = torch.tensor(lens, dtype=torch.int32, device=dev)
        self.scale = D ** -0.5
        self.out = torch.full_like(self.q, 7.5)
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)

    def run(self, **kw):
        import paged_kv_cache_252_gb300 as pkv
        return pkv.paged_attention_prefill(self.out, self.q, self.cu, self.kc, self.vc, self.bt, self.cl, self.scale,
                                           scales=self.sc, device_status=self.status, **kw)

    def check(self, what=""):
        want, tol = op.attention_bound(self.q[:self.cu_host[-1]], self.kc, self.vc, self.sc, self.bt, self.cu_host,
                                       self.lens, self.scale)
        r = op.assert_within(self.out[:self.cu_host[-1]], want, tol, what)
        assert (self.out[self.cu_host[-1]:] == 7.5).all(), "rows behind the last sequence were written"
        print(f"{what}: at most {r:.2f} of the bound")


CASES = {
    # name: (D, hq, hkv, new tokens, context lengths)
    "one-token": (128, 32, 8, [1], [1]),
    "edges": (128, 8, 2, [1, 15, 16, 17, 31, 0, 33], [1, 15, 16, 17, 47, 20, 64]),
    "tile-edges": (64, 4, 4, [127, 128, 129, 255, 256, 257], [127, 128, 129, 256, 384, 300]),
    "mha": (128, 3, 3, [300], [300]),
    "mqa": (64, 16, 1, [70, 2], [190, 130]),
    "group3": (128, 6, 2, [200, 5], [333, 1000]),
    "group5": (64, 5, 1, [130], [131]),
    "group7": (128, 7, 1, [77, 41], [500, 41]),
    "group12": (64, 24, 2, [50, 22], [50, 600]),
    "group48": (128, 48, 1, [13], [260]),
    "group64": (64, 64, 1, [9, 3], [400, 3]),
    "decode-rows": (128, 32, 8, [1] * 20, [700 + 31 * i for i in range(20)]),
    "mixed": (128, 16, 4, [1, 500, 4, 1, 0, 33, 1], [900, 1300, 64, 1, 0, 33, 2050]),
    "few-rows-long": (128, 8, 2, [3], [20011]),
    "rows-long": (128, 8, 2, [40], [20011]),          # joined in groups; a row tile of few rows
    "units-long": (64, 8, 2, [150, 1], [30005, 7]),    # units that share a long context
    "chunk-long": (128, 8, 2, [260], [9000]),
    "many": (64, 2, 1, [(7 * i) % 40 for i in range(150)], [(7 * i) % 40 + (13 * i) % 90 for i in range(150)]),
    "prompt": (128, 8, 2, [1100], [1100]),
}


@pytest.mark.parametrize("kv", ["fp16", "bf16", "e5m2", "int8"])
@pytest.mark.parametrize("name", list(CASES))
def test_prefill_matches_64_bits(dev, name, kv):
    D, hq, hkv, ns, lens = CASES[name]
    b = Batch(dev, kv, D, hq, hkv, ns, lens, seed=len(name), extra_rows=3)
    b.run()
    torch.cuda.synchronize()
    assert b.status.item() == 0
    b.check(f"{name} {kv}")


@pytest.mark.parametrize("kv", ["fp16", "bf16", "e5m2", "int8"])
@pytest.mark.parametrize("gain", [0.0, 8.0, 40.0])
def test_flat_and_peaked_scores(dev, kv, gain):
    """Queries scaled so that the weights are equal, or one position takes nearly all."""
    b = Batch(dev, kv, 128, 8, 2, [150, 1, 40], [700, 1500, 40], q_gain=gain)
    b.run()
    b.check(f"gain {gain} {kv}")


@pytest.mark.parametrize("kv", ["fp16", "bf16", "e5m2"])
@pytest.mark.parametrize("D", [64, 128])
def test_rising_scores_move_the_running_maximum(dev, kv, D):
    """Keys that grow along the context: the maximum moves in every tile."""
    b = Batch(dev, kv, D, 4, 2, [200], [1500])
    pos = torch.empty(1500, device=dev)
    ids = b.bt[0].long()
    ramp = torch.linspace(0.05, 3.0, ids.numel() * 16, device=dev).view(-1, 1, 16, 1)
    base = torch.ones((ids.numel(), 2, 16, D), device=dev) * ramp
    k = base.half() if kv != "bf16" else base.bfloat16()
    b.kc[ids] = k.to(torch.float8_e5m2).view(torch.uint8) if kv == "e5m2" else k
    b.q.copy_(torch.where(torch.arange(200, device=dev)[:, None, None] % 2 == 0, 2.0, -2.0).expand_as(b.q))
    b.run()
    b.check(f"ramp {kv}")
    del pos


def _plant(b, s, positions, kval, vval):
    for p in positions:
        blk = int(b.bt[s, p // 16])
        for c, val in ((b.kc, kval), (b.vc, vval)):
            if val is None:
                continue
            if c.dtype == torch.uint8:
                c[blk, :, p % 16] = {"nan": 0x7E, "inf": 0x7C, "-inf": 0xFC}[val]
            else:
                c[blk, :, p % 16] = float(val)


@pytest.mark.parametrize("kv", ["fp16", "bf16", "e5m2"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("val", ["nan", "inf", "-inf"])
def test_what_a_row_does_not_see_does_not_reach_it(dev, kv, D, val):
    """Infinities and NaN in the last block behind the context, in unused blocks and in later
    tokens of the chunk; the rows that see the later tokens are not finite, the rest as ever."""
    ns, lens = [150, 9], [310, 75]
    b = Batch(dev, kv, D, 8, 2, ns, lens)
    clean = Batch(dev, kv, D, 8, 2, ns, lens)
    clean.run()
    _plant(b, 0, range(310, 320), val, val)       # behind the context, in its last block
    _plant(b, 1, range(75, 80), val, val)
    used = b.bt[b.bt < b.kc.shape[0]].long()
    spare = torch.ones(b.kc.shape[0], dtype=torch.bool, device=dev)
    spare[used] = False
    for c in (b.kc, b.vc):
        c[spare] = 0x7E if c.dtype == torch.uint8 else float("nan")
    b.run()
    torch.cuda.synchronize()
    assert b.status.item() == 0
    assert torch.equal(b.out, clean.out)
    # token 100 of the first chunk and token 5 of the second, values only
    hit = {0: 160 + 100, 1: 66 + 5}
    for s, p in hit.items():
        _plant(b, s, [p], None, val)
    b.run()
    torch.cuda.synchronize()
    sees = torch.zeros(b.q.shape[0], dtype=torch.bool, device=dev)
    sees[100:150] = True
    sees[150 + 5:] = True
    assert not torch.isfinite(b.out[sees]).any()
    want, tol = op.attention_bound(clean.q, clean.kc, clean.vc, None, clean.bt, clean.cu_host, lens, clean.scale)
    op.assert_within(b.out[~sees], want[~sees], tol[~sees], "rows before the planted token")


@pytest.mark.parametrize("kv", ["fp16", "bf16"])
def test_minus_infinite_scores_weigh_nothing(dev, kv):
    """A key of -inf where every query is positive scores -inf: weight zero, its value unread
    by the sum; a row that sees nothing else is 0/0."""
    b = Batch(dev, kv, 64, 2, 1, [40], [140])
    b.q.abs_()
    _plant(b, 0, [0, 3, 50, 120], "-inf", None)
    b.run()
    want, tol = op.attention_bound(b.q, b.kc, b.vc, None, b.bt, b.cu_host, b.lens, b.scale)
    op.assert_within(b.out, want, tol, "-inf keys")
    c = Batch(dev, kv, 64, 2, 1, [3], [3])
    c.q.abs_()
    _plant(c, 0, [0], "-inf", None)
    c.run()
    assert torch.isnan(c.out[0]).all() and torch.isfinite(c.out[1:]).all()


def test_rows_that_see_nothing_are_zero_and_flagged(dev):
    """A context shorter than its new tokens: the first rows see no position."""
    for kv in ("fp16", "bf16", "e5m2", "int8"):
        b = Batch(dev, kv, 128, 8, 2, [20, 30, 5], [40, 30, 16])
        b.cl[1] = 11
        b.cl[2] = 0
        b.run()
        torch.cuda.synchronize()
        assert b.status.item() == 4
        out = b.out.clone()
        assert (out[20:39] == 0).all() and (out[50:55] == 0).all()
        # its last 11 tokens see positions 0..10 as the first 11 tokens of a context of 11 would
        c = Batch(dev, kv, 128, 8, 2, [20, 30, 5], [40, 30, 16])
        c.cu = torch.tensor([0, 20, 31, 36], dtype=torch.int32, device=dev)
        c.cu_host, c.lens = [0, 20, 31, 36], [40, 11, 16]
        c.cl[1] = 11
        c.q[20:31] = b.q[39:50]
        c.run()
        want, tol = op.attention_bound(c.q[:36], c.kc, c.vc, c.sc, c.bt, c.cu_host, c.lens, c.scale)
        op.assert_within(out[39:50], want[20:31], tol[20:31], "clipped")


def test_bad_ranges_lengths_and_blocks_are_flagged_and_harmless(dev):
    b = Batch(dev, "fp16", 64, 4, 2, [10, 10, 10], [64, 64, 64])
    b.cu.copy_(torch.tensor([0, 10, 5, 31], dtype=torch.int32))   # decreasing, then past the end of q
    b.run()
    torch.cuda.synchronize()
    assert b.status.item() == 4
    assert (b.out[10:] == 7.5).all() and (b.out[:10] != 7.5).any()
    c = Batch(dev, "fp16", 64, 4, 2, [10, 10], [64, 64])
    c.cl[0] = 100000                                              # clamped to the table's 64 positions
    c.run()
    torch.cuda.synchronize()
    assert c.status.item() == 4
    want, tol = op.attention_bound(c.q, c.kc, c.vc, None, c.bt, c.cu_host, [64, 64], c.scale)
    op.assert_within(c.out, want, tol, "clamped")
    for kv in ("fp16", "bf16", "e5m2", "int8"):
        d = Batch(dev, kv, 128, 4, 2, [10, 10], [64, 200])
        d.bt[1, 3] = -5
        d.run()
        torch.cuda.synchronize()
        assert d.status.item() == 2
        # a block out of range reads as zeros
        e = Batch(dev, kv, 128, 4, 2, [10, 10], [64, 200])
        blk = int(e.bt[1, 3])
        zero = -128 if kv == "int8" else 0
        e.kc[blk], e.vc[blk] = zero, zero
        want, tol = op.attention_bound(e.q, e.kc, e.vc, e.sc, e.bt, e.cu_host, e.lens, e.scale)
        op.assert_within(d.out, want, tol, "bad block")


def test_int8_extreme_scales(dev):
    """The largest row scale an fp16 row gives (516) and a subnormal one."""
    b = Batch(dev, "int8", 128, 4, 2, [70], [500])
    b.sc[:, :, 1] = 516.0
    b.sc[:, :, 0] = 2.0 ** -24
    want, tol = op.attention_bound(b.q, b.kc, b.vc, b.sc, b.bt, b.cu_host, b.lens, b.scale)
    b.run()
    # |out| up to 65532 rounds to fp16 within 2^-11 of itself, or to infinity past 65520
    fin = want.abs() < 65000
    g = b.out.double()
    assert ((g - want).abs()[fin] <= tol[fin] * 1.0 + 0.0).all()


def test_same_bits_every_time_and_whatever_the_workspace_held(dev):
    import paged_kv_cache_252_gb300 as pkv
    b = Batch(dev, "bf16", 128, 8, 2, [300, 7, 1], [4000, 9000, 3000])
    need = pkv.prefill_workspace_bytes(b.q.shape[0], 3, 8, b.kc)
    ref = b.run().clone()
    for fill in (0, 1, 255):
        ws = torch.full((need,), fill, dtype=torch.uint8, device=dev)
        b.out.fill_(7.5)
        b.run(workspace=ws)
        b.run(workspace=ws)
        assert torch.equal(b.out, ref)


@pytest.mark.parametrize("kv,D", [("fp16", 128), ("int8", 64)])
def test_more_sequences_than_threads(dev, kv, D):
    """The plan gives a thread several sequences; runs of empty ones at the start, inside and at the end."""
    ns = [0] * 700 + [(5 * i) % 7 for i in range(900)] + [200] + [0] * 600 + [1, 3] + [0] * 40
    lens = [n + (11 * i) % 50 for i, n in enumerate(ns)]
    b = Batch(dev, kv, D, 4, 2, ns, lens, extra_rows=2)
    b.run()
    b.check("many sequences")
    assert b.status.item() == 0


@pytest.mark.parametrize("kv,D,ns,lens", [("bf16", 128, [300, 5], [300, 900]), ("fp16", 64, [40, 1], [20011, 9000]),
                                          ("e5m2", 128, [90, 40], [3000, 20011])])
def test_output_and_workspace_on_16_byte_boundaries(dev, kv, D, ns, lens):
    """What the header asks for and no more: whole units, cut ones, joined groups, few rows."""
    import paged_kv_cache_252_gb300 as pkv
    b = Batch(dev, kv, D, 8, 2, ns, lens)
    ref = b.run().clone()
    need = pkv.prefill_workspace_bytes(b.q.shape[0], len(ns), 8, b.kc)
    ws = torch.zeros(need + 16, dtype=torch.uint8, device=dev)[16:]
    flat = torch.full((b.q.numel() + 16,), 7.5, dtype=b.q.dtype, device=dev)
    out = flat[8:8 + b.q.numel()].view(b.q.shape)
    assert ws.data_ptr() % 32 == 16 and out.data_ptr() % 32 == 16
    pkv.paged_attention_prefill(out, b.q, b.cu, b.kc, b.vc, b.bt, b.cl, b.scale, workspace=ws)
    assert torch.equal(out, ref)
    assert (flat[:8] == 7.5).all() and (flat[-8:] == 7.5).all()


def test_same_bits_where_pieces_are_joined_in_groups(dev):
    b = Batch(dev, "fp16", 128, 8, 2, [40, 90], [20011, 15000])
    ref = b.run().clone()
    b.check()
    for _ in range(20):
        b.out.fill_(7.5)
        assert torch.equal(b.run(), ref)


def test_graphs_replay_and_do_not_share_scratch(dev):
    """Two captured calls and eager calls, replayed on two streams at once."""
    a = Batch(dev, "fp16", 128, 8, 2, [130, 4], [6000, 9001], seed=1)
    b = Batch(dev, "fp16", 128, 8, 2, [5, 260], [8000, 700], seed=2)
    want_a, want_b = a.run().clone(), b.run().clone()
    graphs = []
    for x in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            x.run()
        graphs.append(g)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        a.out.fill_(0)
        b.out.fill_(0)
        torch.cuda.synchronize()
        with torch.cuda.stream(s1):
            graphs[0].replay()
        with torch.cuda.stream(s2):
            graphs[1].replay()
        torch.cuda.synchronize()
        assert torch.equal(a.out, want_a) and torch.equal(b.out, want_b)
    # other lengths in the same buffers
    a.cl.copy_(torch.tensor([200, 33], dtype=torch.int32))
    a.lens = [200, 33]
    graphs[0].replay()
    a.check("replayed with new lengths")


def test_calls_on_two_streams_at_once(dev):
    a = Batch(dev, "bf16", 64, 8, 2, [130, 4], [6000, 9001], seed=1)
    b = Batch(dev, "bf16", 64, 8, 2, [5, 260], [8000, 700], seed=2)
    want_a, want_b = a.run().clone(), b.run().clone()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(10):
        a.run(stream=s1)
        b.run(stream=s2)
    torch.cuda.synchronize()
    assert torch.equal(a.out, want_a) and torch.equal(b.out, want_b)


def test_agrees_with_the_chunked_call(dev):
    """The same batch through the decode kernels' row tiles: both within the bound."""
    import paged_kv_cache_252_gb300 as pkv
    b = Batch(dev, "e5m2", 128, 64, 8, [100, 1, 9], [180, 200, 50])
    b.run()
    b.check("prefill")
    other = torch.empty_like(b.out)
    pkv.paged_attention_decode_chunked(other, b.q, b.ns, b.lens, b.kc, b.vc, b.bt, b.scale)
    assert (other.double() - b.out.double()).abs().max() <= 4e-3


def test_more_than_2_31_elements_of_cache(dev):
    """A pool of over 2^31 elements a cache: blocks at its far end."""
    import paged_kv_cache_252_gb300 as pkv
    nb, hkv, D = 140_000, 8, 128                     # 2.3e9 elements
    kc = torch.zeros((nb, hkv, 16, D), dtype=torch.uint8, device=dev)
    vc = torch.zeros_like(kc)
    small = Batch(dev, "e5m2", D, 16, hkv, [70], [200])
    far = torch.arange(nb - small.bt.shape[1], nb, device=dev)
    kc[far], vc[far] = small.kc[small.bt[0].long()], small.vc[small.bt[0].long()]
    want = small.run().clone()
    out = torch.empty_like(small.out)
    pkv.paged_attention_prefill(out, small.q, small.cu, kc, vc, far.to(torch.int32)[None], small.cl, small.scale)
    assert torch.equal(out, want)


def test_no_rows_and_no_sequences(dev):
    b = Batch(dev, "fp16", 64, 4, 2, [0, 0], [16, 30])
    b.run()
    c = Batch(dev, "fp16", 64, 4, 2, [3], [3])
    import paged_kv_cache_252_gb300 as pkv
    pkv.paged_attention_prefill(c.out, c.q, torch.zeros(1, dtype=torch.int32, device=dev), c.kc, c.vc, c.bt[:0],
                                c.cl[:0], 1.0)
    assert (c.out == 7.5).all()
