"""INT4 cache: quantising writes against the codec's definition in 64 bits (codes and scales equal),
reading back from every cache type, block copies and accepted drafts."""
import math

import pytest
import torch

import paged_kv_cache_252_gb300 as pkv
import _int4 as i4
from _operators import make_cache as make_other, cache_rows

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _alloc(blocks, hkv, d):
    return (*pkv.alloc_kv_cache(blocks, hkv, d, "int4", DEV), pkv.alloc_kv_scales(blocks, hkv, DEV, kv_dtype="int4", head_size=d))


def _written(x, slots, cache, scales, which):
    """Codes and scales of the slots against the definition."""
    codes, s, z = i4.quantised(x)
    blk, off = slots.long() // 16, slots.long() % 16
    assert torch.equal(i4.unpack(cache[blk, :, off]), codes)
    got = scales[blk, :, which, off]
    bad = s.isnan()
    assert torch.equal(got[..., 0].isnan(), bad)
    assert torch.equal(torch.where(bad, 0.0, got[..., 0].double()), torch.where(bad, 0.0, s))
    assert torch.equal(torch.where(bad, 0.0, got[..., 1].double()), torch.where(bad, 0.0, z))


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("d,hkv,T", [(128, 8, 1), (128, 8, 64), (128, 1, 3), (64, 4, 2001), (64, 1, 1), (128, 3, 517), (64, 5, 77)])
def test_write_is_the_definition(dtype, d, hkv, T):
    g = _gen(T + d)
    blocks = -(-T // 16) + 2
    kc, vc, sc = _alloc(blocks, hkv, d)
    key = (torch.randn((T, hkv, d), generator=g, device=DEV) + 3 * torch.randn((hkv, d), generator=g, device=DEV)).to(dtype)
    value = torch.randn((T, hkv, d), generator=g, device=DEV).to(dtype)
    slots = torch.randperm(blocks * 16, generator=g, device=DEV)[:T].to(torch.int32)
    pkv.kv_cache_write_int4(key, value, slots, kc, vc, sc)
    _written(key, slots, kc, sc, 0)
    _written(value, slots, vc, sc, 1)
    rest = torch.ones(blocks * 16, dtype=torch.bool, device=DEV)
    rest[slots.long()] = False
    free = rest.nonzero()[:, 0]
    assert not kc[free // 16, :, free % 16].any() and not vc[free // 16, :, free % 16].any()
    assert not sc[free // 16, :, :, free % 16].any()


def _hard_rows(dtype, d):
    """Rows beside the borders: lattices on which many quotients fall exactly halfway, constants, zeros of both
    signs, subnormals, the largest numbers, far apart sizes, all positive and all negative groups."""
    g = torch.Generator().manual_seed(5)
    rows = []
    for step in (1.0, 0.5, 2.0 ** -10, 2.0 ** -24 if dtype == torch.float16 else 2.0 ** -30, 2.0 ** 7, 3.0):
        rows.append(torch.randint(0, 31, (40, d), generator=g).double() * step)          # s of one or two steps
        rows.append(torch.randint(-15, 16, (40, d), generator=g).double() * step)
        rows.append((torch.randint(0, 31, (40, d), generator=g).double() - 100) * step)
    x = torch.randn((200, d), generator=g).double()
    rows += [x * 2.0 ** -14, x * 2.0 ** -20, x * 2.0 ** 12, x.abs() + 4, -x.abs() - 4, x.sign() * torch.exp2(20 * torch.rand((200, d), generator=g) - 14)]
    edge = torch.zeros((6, d), dtype=torch.float64)
    edge[1] = -0.0
    edge[2] = 7.25
    edge[3, ::2], edge[3, 1::2] = 65504.0, -65504.0
    edge[4, 0], edge[4, 1:] = 65504.0, 2.0 ** -24
    edge[5, 3] = -2.0 ** -24
    rows.append(edge)
    # a difference that fp32 rounds: a large number beside a tiny least value
    far = torch.full((64, d), 1.0, dtype=torch.float64)
    far[:, 0] = 2.0 ** -24 * torch.arange(1, 65)
    far[:, 1] = 15.0 * torch.arange(1, 65) / 4
    rows.append(far)
    out = torch.cat(rows).to(dtype)
    if dtype == torch.bfloat16:
        wide = torch.randn((50, d), generator=g) * torch.exp2(torch.randint(-120, 120, (50, 1), generator=g).float())
        out = torch.cat((out, wide.to(dtype)))
    return out


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("d", [64, 128])
def test_write_beside_borders(dtype, d):
    rows = _hard_rows(dtype, d).to(DEV)
    T = rows.shape[0]
    kc, vc, sc = _alloc(-(-T // 16), 1, d)
    slots = torch.arange(T, device=DEV, dtype=torch.int32)
    pkv.kv_cache_write_int4(rows[:, None].contiguous(), rows.flip(0)[:, None].contiguous(), slots, kc, vc, sc)
    _written(rows[:, None], slots, kc, sc, 0)
    _written(rows.flip(0)[:, None], slots, vc, sc, 1)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_write_of_what_is_not_finite(dtype):
    g = _gen(3)
    x = torch.randn((6, 2, 128), generator=g, device=DEV).to(dtype)
    x[0, 0, 5], x[1, 1, 70], x[2, 0, 127], x[3, 1, 0] = math.nan, math.inf, -math.inf, math.nan
    kc, vc, sc = _alloc(1, 2, 128)
    slots = torch.arange(6, device=DEV, dtype=torch.int32)
    pkv.kv_cache_write_int4(x, x, slots, kc, vc, sc)
    _written(x, slots, kc, sc, 0)
    k, v = torch.empty_like(x), torch.empty_like(x)
    pkv.kv_cache_read(k, v, slots, kc, vc, "int4", scales=sc)
    bad = ~x.reshape(6, 2, 2, 64).isfinite().all(-1, keepdim=True).expand(6, 2, 2, 64).reshape(6, 2, 128)
    assert torch.equal(k.isnan(), bad) and torch.equal(v.isnan(), bad)


def test_slots_skipped_and_out_of_range():
    g = _gen(9)
    kc, vc, sc = _alloc(2, 2, 64)
    x = torch.randn((5, 2, 64), generator=g, device=DEV).half()
    slots = torch.tensor([3, -1, 32, -7, 30], device=DEV, dtype=torch.int32)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    pkv.kv_cache_write_int4(x, x, slots, kc, vc, sc, device_status=st)
    assert int(st) == 1
    keep = torch.tensor([0, 4], device=DEV)
    _written(x[keep], slots[keep], kc, sc, 0)
    assert int((kc != 0).any(-1).any(1).sum()) == 2
    k, v = torch.full_like(x, 7.0), torch.full_like(x, 7.0)
    st.zero_()
    pkv.kv_cache_read(k, v, slots, kc, vc, "int4", scales=sc, device_status=st)
    assert int(st) == 1 and bool((k[1:4] == 7).all()) and bool((v[1:4] == 7).all()) and not bool((k[0] == 7).any())
    st.zero_()
    pkv.kv_cache_read(k, v, torch.full_like(slots, -1), kc, vc, "int4", scales=sc, device_status=st)
    assert int(st) == 0


@pytest.mark.parametrize("out", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("kv", ["fp16", "bf16", "e5m2", "int8", "int4"])
@pytest.mark.parametrize("d,hkv,T", [(128, 8, 333), (64, 3, 1), (64, 1, 130), (128, 2, 4097)])
def test_read_is_the_value_rounded_once(out, kv, d, hkv, T):
    g = _gen(T)
    blocks = 40
    if kv == "int4":
        kc, vc, sc = i4.make_cache(blocks, hkv, d, g, DEV, bias=3.0)
    else:
        kc, vc, sc = make_other(kv, blocks, hkv, d, g, DEV)
    slots = torch.randint(0, blocks * 16, (T,), generator=g, device=DEV, dtype=torch.int32)   # some of them repeatedly
    k, v = (torch.full((T, hkv, d), math.nan, dtype=out, device=DEV) for _ in range(2))
    pkv.kv_cache_read(k, v, slots, kc, vc, kv, scales=sc)
    blk, off = slots.long() // 16, slots.long() % 16
    for which, (got, cache) in enumerate(((k, kc), (v, vc))):
        want = (i4.rows_of(cache, sc, which, blk, off)[0] if kv == "int4" else cache_rows(cache, sc, which)[blk, :, off])
        # rounded once; where the value's fp32 form was rounded before, by at most 2^-24 more
        tol = (i4.U[out] + 2.0 ** -24) * want.abs() + (2.0 ** -25 if out == torch.float16 else 0.0)
        assert ((got.double() - want).abs() <= tol).all()
        if kv in ("fp16", "e5m2") and out == torch.float16 or kv == "bf16" and out == torch.bfloat16:
            assert torch.equal(got.double(), want)


def test_written_then_read_is_within_half_a_scale():
    g = _gen(1)
    x = torch.randn((64, 8, 128), generator=g, device=DEV).half()
    kc, vc, sc = _alloc(5, 8, 128)
    slots = torch.randperm(80, generator=g, device=DEV)[:64].to(torch.int32)
    pkv.kv_cache_write_int4(x, x, slots, kc, vc, sc)
    k, v = torch.empty_like(x), torch.empty_like(x)
    pkv.kv_cache_read(k, v, slots, kc, vc, "int4", scales=sc)
    s = sc[slots.long() // 16, :, 0, slots.long() % 16][..., 0].double().repeat_interleave(64, -1)
    # half a scale, and the fp16 rounding of values below 8
    assert ((k.double() - x.double()).abs() <= s / 2 + 8 * 2.0 ** -11).all() and torch.equal(k, v)


def test_copy_blocks_and_accept():
    g = _gen(4)
    for d in (64, 128):
        hkv = 3
        kc, vc, sc = i4.make_cache(12, hkv, d, g, DEV)
        k0, v0, s0 = kc.clone(), vc.clone(), sc.clone()
        src, dst = (torch.tensor(x, device=DEV, dtype=torch.int32) for x in ([1, 5, 2], [0, 7, 11]))
        pkv.copy_blocks(kc, vc, src, dst, "int4", scales=sc)
        for x, x0 in ((kc, k0), (vc, v0), (sc, s0)):
            assert torch.equal(x[dst.long()], x0[src.long()])
            assert torch.equal(x[[1, 2, 3, 4, 5, 6, 8, 9, 10]], x0[[1, 2, 3, 4, 5, 6, 8, 9, 10]])
        # two sequences of 64 drafts: a path is moved together behind the context
        kc, vc, sc = k0.clone(), v0.clone(), s0.clone()
        tables = torch.tensor([[3, 8, 1, 9, 4], [0, 2, 5, 6, 7]], device=DEV, dtype=torch.int32)
        lens = torch.tensor([69, 80], device=DEV, dtype=torch.int32)
        paths = [[0, 3, 4, 17, 40, 63], list(range(0, 64))]
        acc = torch.tensor([p + [0] * (64 - len(p)) for p in paths], device=DEV, dtype=torch.int32)
        num = torch.tensor([len(p) for p in paths], device=DEV, dtype=torch.int32)
        new = torch.zeros(2, device=DEV, dtype=torch.int32)
        pkv.kv_cache_accept(kc, vc, tables, lens, acc, num, new, 64, "int4", scales=sc)
        assert new.tolist() == [69 - 64 + 6, 80]
        want = [k0.clone(), v0.clone(), s0.transpose(2, 3).contiguous()]
        for s, p in enumerate(paths):
            base = int(lens[s]) - 64
            at = [(int(tables[s, (base + i) // 16]), (base + i) % 16) for i in range(64)]
            for w, x0 in zip(want, (k0, v0, s0.transpose(2, 3).contiguous())):
                for i, j in enumerate(p):
                    w[at[i][0], :, at[i][1]] = x0[at[j][0], :, at[j][1]]
        assert torch.equal(kc, want[0]) and torch.equal(vc, want[1]) and torch.equal(sc.transpose(2, 3), want[2])


def test_offsets_beyond_32_bits():
    """Caches of more than 4 GB: the highest blocks."""
    hkv, d = 8, 128
    blocks = (1 << 32) // (hkv * 16 * 64) + 4096
    kc, vc, sc = _alloc(blocks, hkv, d)
    g = _gen(8)
    x = torch.randn((40, hkv, d), generator=g, device=DEV).half()
    slots = (blocks * 16 - 1 - torch.arange(40, device=DEV) * 37).to(torch.int32)
    pkv.kv_cache_write_int4(x, x, slots, kc, vc, sc)
    _written(x, slots, kc, sc, 0)
    _written(x, slots, vc, sc, 1)
    k, v = torch.empty_like(x), torch.empty_like(x)
    pkv.kv_cache_read(k, v, slots, kc, vc, "int4", scales=sc)
    want = i4.rows_of(kc, sc, 0, slots.long() // 16, slots.long() % 16)[0]
    assert ((k.double() - want).abs() <= 2.0 ** -11 * want.abs() + 2.0 ** -25).all() and torch.equal(k, v)
    tables = torch.arange(blocks - 8, blocks, device=DEV, dtype=torch.int32)[None]
    kc[blocks - 8:], vc[blocks - 8:], sc[blocks - 8:] = i4.make_cache(8, hkv, d, g, DEV)
    q = torch.randn((1, 32, d), generator=g, device=DEV).half()
    out = torch.empty_like(q)
    pkv.paged_attention_decode_int4(out, q, kc, vc, sc, tables, torch.tensor([120], device=DEV, dtype=torch.int32), 1, d ** -0.5)
    i4.assert_within(out, *i4.attention(q, kc, vc, sc, tables, [120], [0, 1], d ** -0.5))
