"""Decode attention over an INT4 cache against the 64-bit form: row counts of every shape of the kernel, lengths from one
token on, chains, ragged batches, trees, chunks; what masked places may hold; graphs and streams."""
import math
import random

import pytest
import torch

import paged_kv_cache_252_gb300 as pkv
import _int4 as i4

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


class Case:
    def __init__(self, lens, hq, hkv, d, dtype, n=1, counts=None, seed=0, **cache):
        self.g = _gen(seed)
        self.lens, self.n = lens, n
        counts = counts or [n] * len(lens)
        cu = [0]
        for c in counts:
            cu.append(cu[-1] + c)
        self.cu = cu
        self.tables, blocks = i4.tables_for(lens, self.g, DEV)
        self.k, self.v, self.sc = i4.make_cache(blocks, hkv, d, self.g, DEV, **cache)
        self.q = torch.randn((cu[-1], hq, d), generator=self.g, device=DEV).to(dtype)
        self.ctx = torch.tensor(lens, device=DEV, dtype=torch.int32)
        self.scale = d ** -0.5

    def cu_t(self):
        return torch.tensor(self.cu, device=DEV, dtype=torch.int32)

    def want(self, masks=None):
        return i4.attention(self.q, self.k, self.v, self.sc, self.tables, self.lens, self.cu, self.scale, masks)

    def fixed(self, **kw):
        out = torch.full_like(self.q, math.nan)
        return pkv.paged_attention_decode_int4(out, self.q, self.k, self.v, self.sc, self.tables, self.ctx, self.n, self.scale, **kw)

    def varlen(self, **kw):
        out = torch.full_like(self.q, math.nan)
        return pkv.paged_attention_decode_varlen(out, self.q, self.cu_t(), self.k, self.v, self.tables, self.ctx, self.n,
                                                 self.scale, "int4", scales=self.sc, **kw)

    def tree(self, masks, ragged=True, **kw):
        out = torch.full_like(self.q, math.nan)
        return pkv.paged_attention_decode_tree(out, self.q, masks, self.k, self.v, self.tables, self.ctx, self.n, self.scale,
                                               "int4", cu_q_lens=self.cu_t() if ragged else None, scales=self.sc, **kw)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("g,n", [(1, 1), (4, 1), (8, 1), (3, 3), (4, 4), (6, 4), (8, 4), (8, 8), (64, 1), (1, 64), (5, 12)])
def test_rows_of_every_shape(dtype, d, g, n):
    hkv = 2
    c = Case([max(n, x) for x in (1, 2, 15, 16, 17, 33, 250, 1000)], g * hkv, hkv, d, dtype, n=n, seed=g * 100 + n, bias=2.0)
    r = i4.assert_within(c.fixed(), *c.want(), f"G {g} n {n}")
    print(f"{dtype} D {d} G {g} n {n}: {r:.2f} of the bound")


@pytest.mark.parametrize("lens", [[1], [16], [100000], [131072, 1], [5000] * 3, [20] * 700, [1] * 1300, [17, 40000, 3, 900, 16, 1]])
def test_lengths(lens):
    c = Case(lens, 8, 2, 128, torch.float16, seed=len(lens))
    i4.assert_within(c.fixed(), *c.want())


@pytest.mark.parametrize("d", [64, 128])
def test_ragged_counts_and_rows_behind_the_last_sequence(d):
    r = random.Random(d)
    counts = [r.randint(1, 6) for _ in range(19)]
    lens = [max(c, r.randint(1, 700)) for c in counts]
    c = Case(lens, 16, 4, d, torch.bfloat16, n=6, counts=counts, seed=d)
    want = c.want()
    i4.assert_within(c.varlen(), *want)
    extra = torch.cat((c.q, c.q[:3]))
    out = torch.full_like(extra, 5.0)
    pkv.paged_attention_decode_varlen(out, extra, c.cu_t(), c.k, c.v, c.tables, c.ctx, 6, c.scale, "int4", scales=c.sc)
    i4.assert_within(out[:-3], *want)
    assert bool((out[-3:] == 5).all())


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("g,n", [(4, 5), (1, 64), (4, 16), (2, 8)])
def test_trees(dtype, g, n):
    r = random.Random(n)
    counts = [r.randint(1, n) for _ in range(9)] + [n]
    lens = [max(c, r.randint(1, 400)) for c in counts] + []
    c = Case(lens, 2 * g, 2, 64, dtype, n=n, counts=counts, seed=n)
    masks = torch.tensor([r.getrandbits(63) | 1 << min(62, j) for k in counts for j in range(k)], device=DEV, dtype=torch.int64)
    i4.assert_within(c.tree(masks), *c.want(masks))
    full = Case([100, 64, 70], 2 * g, 2, 128, dtype, n=n, seed=n)
    masks = i4.chain(n, DEV).repeat(3)
    got = full.tree(masks, ragged=False)
    i4.assert_within(got, *full.want(masks))
    assert torch.equal(got, full.fixed())


def test_rows_that_see_nothing_are_zero():
    c = Case([4, 20], 8, 2, 64, torch.float16, n=4)
    masks = torch.tensor([1, 0, 4, 0, 1, 2, 4, 8], device=DEV, dtype=torch.int64)
    out = c.tree(masks, ragged=False)
    assert not out[[1, 3]].any()
    i4.assert_within(out, *c.want(masks))


@pytest.mark.parametrize("d", [64, 128])
def test_what_masked_places_hold_does_not_matter(d):
    """Rows behind the context and hidden drafts hold NaN scales and infinite least values; unused table entries are out of range."""
    c = Case([5, 18, 31, 100], 8, 2, d, torch.float16, n=3, seed=3)
    masks = torch.tensor([1, 2, 4] * 4, device=DEV, dtype=torch.int64)   # each draft sees the context and itself
    clean = c.tree(masks, ragged=False)
    i4.assert_within(clean, *c.want(masks))
    for s, ctx in enumerate(c.lens):
        last = int(c.tables[s, (ctx - 1) // 16])
        if ctx % 16:
            c.sc[last, :, :, ctx % 16:, :, 0] = math.nan
            c.sc[last, :, :, ctx % 16:, :, 1] = -math.inf
    assert torch.equal(c.tree(masks, ragged=False), clean)
    # draft 1 of every sequence is spoilt: only its own row shows it
    for s, ctx in enumerate(c.lens):
        p = ctx - 2
        c.sc[int(c.tables[s, p // 16]), :, :, p % 16, :, 0] = math.nan
    out = c.tree(masks, ragged=False)
    own = torch.arange(len(c.lens), device=DEV) * 3 + 1
    assert out[own].isnan().all()
    rest = torch.ones(out.shape[0], dtype=torch.bool, device=DEV)
    rest[own] = False
    assert torch.equal(out[rest], clean[rest])


@pytest.mark.parametrize("spread", [10.0, 16.0])
def test_values_of_very_different_sizes(spread):
    """V rows of 2^-spread to 2^spread; and all tiny, where an fp16 weight beside them must keep its bits."""
    c = Case([700, 1, 3000], 8, 2, 128, torch.float16, seed=int(spread), spread=spread if spread < 12 else 12.0)
    i4.assert_within(c.fixed(), *c.want())
    c.sc[:, :, 1] *= 2.0 ** -6
    i4.assert_within(c.fixed(), *c.want())


def test_constant_values_have_scale_zero():
    c = Case([50, 16, 1], 4, 2, 128, torch.float16)
    c.sc[:, :, 1, :, :, 0] = 0
    i4.assert_within(c.fixed(), *c.want())
    c.sc[::2, :, 1, :, 0, 0] = 1.0     # ... beside scales that are not
    i4.assert_within(c.fixed(), *c.want())
    c.sc[:, :, 0, :, :, 0] = 0         # constant keys
    i4.assert_within(c.fixed(), *c.want())


@pytest.mark.parametrize("dtype,size", [(torch.float16, 2.0 ** -12), (torch.float16, 2000.0), (torch.bfloat16, 2.0 ** -60),
                                        (torch.bfloat16, 2.0 ** 30), (torch.bfloat16, 40.0)])
def test_queries_of_every_size(dtype, size):
    c = Case([300, 40], 8, 2, 128, dtype, seed=2)
    c.q *= size
    c.scale = c.scale / size if size > 1e4 or size < 1e-4 else c.scale
    i4.assert_within(c.fixed(), *c.want())


def test_sharp_scores_move_the_reference():
    """Scores that grow by hundreds along the context, and that fall."""
    for sign in (1, -1):
        c = Case([2000], 4, 1, 128, torch.float16, seed=6)
        c.q.fill_(1.0)
        blk = c.tables[0].long()
        ramp = torch.arange(blk.numel() * 16, device=DEV, dtype=torch.float32).view(-1, 16) * (sign * 0.01)
        c.sc[blk, :, 0, :, :, 1] = ramp[:, None, :, None].expand(-1, 1, -1, 2).half()
        c.sc[:, :, 0, :, :, 0] = 0.01
        i4.assert_within(c.fixed(), *c.want())


def test_bad_blocks_lengths_and_counts_are_flagged():
    c = Case([40, 40, 40], 8, 2, 128, torch.float16, n=2)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    good = c.fixed(device_status=st)
    assert int(st) == 0
    c.tables[1, 1] = -5
    out = c.fixed(device_status=st)
    assert int(st) == 2 and torch.equal(out[[0, 1, 4, 5]], good[[0, 1, 4, 5]]) and bool(out.isfinite().all())
    st.zero_()
    c.tables[1, 1] = 0
    c.ctx[2] = 1000
    out = c.fixed(device_status=st)
    assert int(st) & 4 and torch.equal(out[:2], good[:2])
    st.zero_()
    c.ctx[2] = 40
    cu = torch.tensor([0, 2, 9, 6], device=DEV, dtype=torch.int32)
    out = torch.full_like(c.q, 5.0)
    pkv.paged_attention_decode_varlen(out, c.q, cu, c.k, c.v, c.tables, c.ctx, 2, c.scale, "int4", scales=c.sc, device_status=st)
    assert int(st) == 4 and torch.equal(out[:2], good[:2]) and bool((out[2:] == 5).all())
    for ctx in (0, -3):
        st.zero_()
        c.ctx[1] = ctx
        out = c.fixed(device_status=st)
        assert int(st) == 4 and not out[2:4].any()


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_chunked(dtype):
    counts = [70, 1, 33, 4, 1]
    lens = [200, 900, 33, 64, 1]
    c = Case(lens, 8, 2, 128, dtype, n=70, counts=counts, seed=4)
    out = torch.full_like(c.q, math.nan)
    pkv.paged_attention_decode_chunked(out, c.q, counts, lens, c.k, c.v, c.tables, c.scale, "int4", scales=c.sc)
    i4.assert_within(out, *c.want())


def test_graphs_streams_and_repeats():
    """Two captured graphs and eager calls on streams of their own, over and over: the bits stay."""
    cases = [Case([3000, 17, 800, 1], 32, 8, 128, torch.float16, seed=1), Case([64] * 9, 16, 4, 64, torch.bfloat16, n=4, seed=2)]
    want = [c.fixed() for c in cases]
    graphs, outs = [], []
    for c in cases:
        g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(g, stream=s):
            outs.append(c.fixed())
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(4)]
    torch.cuda.synchronize()
    eager = []
    for _ in range(20):
        for k, (g, c) in enumerate(zip(graphs, cases)):
            with torch.cuda.stream(streams[k]):
                g.replay()
            eager.append((k, c.fixed(stream=None)))
            with torch.cuda.stream(streams[2 + k]):
                eager.append((k, c.fixed()))
    torch.cuda.synchronize()
    for k in range(2):
        i4.assert_within(want[k], *cases[k].want())
        assert torch.equal(outs[k], want[k])
    for k, o in eager:
        assert torch.equal(o, want[k])


def test_a_stream_given_by_name():
    c = Case([500, 20], 8, 2, 128, torch.float16)
    want = c.fixed()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = c.fixed(stream=s)
    s.synchronize()
    assert torch.equal(out, want)


def test_a_workspace_full_of_small_numbers():
    c = Case([4000, 300], 8, 2, 128, torch.float16)
    need = pkv.api.load_library().pkv_decode_workspace_bytes(2, 8, 1, pkv.api._desc_of(c.k, c.v, True)[0])
    want = c.fixed()
    for fill in (0, 1, 7, -1):
        ws = torch.full((need // 4 + 64,), fill, dtype=torch.int32, device=DEV)
        assert torch.equal(c.fixed(workspace=ws), want)


@pytest.mark.parametrize("hq", [2, 8, 16, 32, 64])
def test_one_unit_over_the_whole_device(hq):
    """Every CTA has a piece of one unit: a join of several levels, and again from a replayed graph."""
    c = Case([262144 - 5], hq, 1, 128, torch.bfloat16, seed=hq)
    i4.assert_within(c.fixed(), *c.want())
    want = c.fixed()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = c.fixed()
    for _ in range(5):
        out.zero_()
        g.replay()
        assert torch.equal(out, want)


@pytest.mark.parametrize("hq", [4, 32])
def test_long_contexts_keep_the_results_bits(hq):
    """Over n similar weights the result is some sqrt(n) times smaller than the sums of codes times weights. A rounding to fp16 of
    a number with mantissa m in [1, 2) has the relative variance (2^-20 / 12) / m^2. The outputs' mantissas take all values (evenly
    in log m: the mean of 1 / m^2 is 3 / (8 ln 2) = 0.541); the weights P may all lie near m = 1. Both roundings together have at most
    1 + 1 / 0.541 = 2.85 times the variance of the output's alone, 3.1 = 1.76^2 times with all else half an output's rounding."""
    c = Case([131072], hq, 1, 128, torch.float16, seed=hq)
    c.q *= 0.25
    want, _ = c.want()
    alone = (want.half().double() - want).norm()
    assert (c.fixed().double() - want).norm() <= 1.76 * alone


@pytest.mark.parametrize("g,n", [(2, 1), (4, 1), (8, 1), (4, 4), (8, 4), (8, 8)])
def test_a_spoilt_group_spoils_its_own_dimensions(g, n):
    """A value group that read back as NaN makes NaN of its 64 dimensions in the rows that see it; the other 64 stay within the bound."""
    c = Case([40, 700], 2 * g, 2, 128, torch.float16, n=n, seed=g)
    for s, at in ((0, 3), (1, 500)):
        c.sc[int(c.tables[s, at // 16]), :, 1, at % 16, s, 0] = math.nan
    out, (want, tol) = c.fixed(), c.want()
    rows = c.cu[1]
    for part, bad, good in ((slice(0, rows), slice(0, 64), slice(64, 128)), (slice(rows, None), slice(64, 128), slice(0, 64))):
        assert out[part, :, bad].isnan().all()
        i4.assert_within(out[part, :, good], want[part, :, good], tol[part, :, good])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("g,n", [(1, 3), (1, 4), (2, 2), (3, 1), (2, 4), (5, 3), (7, 4), (9, 7)])
def test_ragged_counts_of_every_shape(g, n, d):
    """Sequences of fewer rows than the shape holds, behind sequences of more, one of them with queries that are not finite: what
    earlier rows leave behind does not show."""
    r = random.Random(g * 10 + n)
    counts = [n, 1, max(1, n - 1), 1] * 6
    lens = [max(c, r.randint(1, 600)) for c in counts]
    c = Case(lens, 2 * g, 2, d, torch.float16, n=n, counts=counts, seed=g)
    want = c.want()
    i4.assert_within(c.varlen(), *want)
    clean = c.varlen()
    bad = [s for s in range(len(counts)) if s % 4 == 0]
    for k, s in enumerate(bad):
        c.q[c.cu[s]:c.cu[s + 1]] = (math.nan, math.inf, -math.inf)[k % 3]
    out = c.varlen()
    for s in range(len(counts)):
        rows = slice(c.cu[s], c.cu[s + 1])
        if s in bad:
            assert not out[rows].isfinite().all()
        else:
            assert torch.equal(out[rows], clean[rows])
