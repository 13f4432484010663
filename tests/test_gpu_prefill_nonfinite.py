"""Infinities and NaN in value rows: which outputs they reach, and that the rest cost what they did."""
import pytest
import torch

import _bounds
import _operators as op
from test_gpu_prefill import Batch, dev  # noqa: F401

pytestmark = pytest.mark.gpu


def _plant(b, s, p, dims, val):
    blk = int(b.bt[s, p // 16])
    if b.vc.dtype == torch.uint8:
        b.vc[blk, :, p % 16, dims] = {"nan": 0x7E, "inf": 0x7C, "-inf": 0xFC}[val]
    else:
        b.vc[blk, :, p % 16, dims] = float(val)


@pytest.mark.parametrize("kv", ["fp16", "bf16", "e5m2"])
@pytest.mark.parametrize("val", ["nan", "inf", "-inf"])
@pytest.mark.parametrize("ns,lens,s,p", [([300], [300], 0, 10), ([90, 40], [3000, 20011], 1, 19990),
                                         ([1, 3], [20011, 9000], 0, 700), ([40], [20011], 0, 5)])
def test_only_the_dimensions_that_hold_one(dev, kv, val, ns, lens, s, p):  # noqa: F811
    """Three dimensions of one value row: rows that see it are not finite there, all else as without it;
    whole units, cut ones, joined groups, few rows."""
    clean = Batch(dev, kv, 128, 8, 2, ns, lens)
    clean.run()
    b = Batch(dev, kv, 128, 8, 2, ns, lens)
    dims = [0, 77, 127]
    _plant(b, s, p, dims, val)
    b.run()
    torch.cuda.synchronize()
    assert b.status.item() == 0
    hit = torch.zeros_like(b.out, dtype=torch.bool)
    first = max(p - (lens[s] - ns[s]), 0)
    hit[b.cu_host[s] + first:b.cu_host[s + 1], :, dims] = True
    assert not torch.isfinite(b.out[hit]).any()
    # (no weight here is below fp16's least number, so an infinity stays one)
    assert torch.isnan(b.out[hit]).all() if val == "nan" else (b.out[hit] == float(val)).all()
    at, want, tol = _bounds.attention_rows(clean, s)
    away = ~hit[at]
    op.assert_within(b.out[at][away], want[away], tol[away], "elements it does not reach")
    other = ~torch.isin(torch.arange(b.q.shape[0], device=dev), torch.arange(at.start, at.stop, device=dev))
    assert torch.equal(b.out[other], clean.out[other])


@pytest.mark.parametrize("kv", ["fp16", "bf16", "e5m2"])
def test_an_unseen_nan_beside_a_seen_infinity(dev, kv):  # noqa: F811
    """Later tokens of the chunk hold NaN in a dimension where an early token holds an infinity, and where
    two hold infinities of both signs."""
    b = Batch(dev, kv, 64, 4, 2, [120], [200])
    _plant(b, 0, 7, [5], "inf")
    _plant(b, 0, 8, [5], "inf")
    _plant(b, 0, 20, [9], "inf")
    _plant(b, 0, 21, [9], "-inf")
    _plant(b, 0, 180, [5, 9, 11], "nan")
    b.run()
    torch.cuda.synchronize()
    before, after = b.out[:100], b.out[100:]
    assert (before[..., 5] == float("inf")).all() and torch.isnan(before[..., 9]).all()
    assert torch.isfinite(before[..., 11]).all() and torch.isnan(after[..., [5, 9, 11]]).all()
    rest = [i for i in range(64) if i not in (5, 9, 11)]
    assert torch.isfinite(b.out[..., rest]).all()


@pytest.mark.parametrize("kv", ["fp16", "bf16", "e5m2", "int8"])
@pytest.mark.parametrize("ns,lens", [([300], [300]), ([3], [20011])])
def test_a_key_that_is_not_a_number(dev, kv, ns, lens):  # noqa: F811
    """Rows that see it are NaN throughout, the rest as without it; the same for a NaN K scale."""
    b, clean = (Batch(dev, kv, 64, 4, 2, ns, lens) for _ in range(2))
    clean.run()
    p = lens[0] - ns[0] + ns[0] // 2
    blk = int(b.bt[0, p // 16])
    if kv == "int8":
        b.sc[blk, :, 0, p % 16] = float("nan")
    elif kv == "e5m2":
        b.kc[blk, :, p % 16, 3] = 0x7E
    else:
        b.kc[blk, :, p % 16, 3] = float("nan")
    b.run()
    torch.cuda.synchronize()
    k = ns[0] // 2
    assert torch.isnan(b.out[k:]).all()
    at, want, tol = _bounds.attention_rows(clean, 0)
    op.assert_within(b.out[:k], want[:k], tol[:k], "rows before it")


@pytest.mark.parametrize("kv", ["fp16", "bf16", "e5m2", "int8"])
@pytest.mark.parametrize("n,ctx", [(30, 11), (4, 3), (300, 290)])
def test_rows_that_see_nothing_stay_zero(dev, kv, n, ctx):  # noqa: F811
    """A context shorter than its new tokens, whose last token holds NaN: only the last row sees that."""
    b = Batch(dev, kv, 64, 4, 2, [n], [n])
    b.cl[0] = ctx
    p = ctx - 1
    if kv == "int8":
        b.sc[int(b.bt[0, p // 16]), :, 1, p % 16] = float("nan")
    else:
        _plant(b, 0, p, [3, 40], "nan")
    b.run()
    torch.cuda.synchronize()
    assert b.status.item() == 4
    assert (b.out[:n - ctx] == 0).all() and torch.isfinite(b.out[:n - 1]).all() and torch.isnan(b.out[n - 1, :, 3]).all()


def _time(b):
    for _ in range(2):
        b.run()
    best = 1e9
    for _ in range(5):
        t = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
        t[0].record()
        b.run()
        t[1].record()
        torch.cuda.synchronize()
        best = min(best, t[0].elapsed_time(t[1]))
    return best


@pytest.mark.parametrize("kv", ["bf16", "e5m2", "int8"])
@pytest.mark.parametrize("ns,lens", [([4096], [4096]), ([1] * 16, [6000] * 16), ([64], [40000])])
@pytest.mark.parametrize("val", ["nan", "inf", "key"])
def test_rows_behind_one_are_not_computed_again(dev, kv, ns, lens, val):  # noqa: F811
    """One value row (or key) that is not finite, early in every context. Rows that see it stand as the products
    left them: all of them again on the CUDA cores took 130 to 7000 times as long."""
    b = Batch(dev, kv, 128, 8, 2, ns, lens)
    plain = _time(b)
    for s in range(len(ns)):
        if kv == "int8":
            b.sc[int(b.bt[s, 6]), :, 0 if val == "key" else 1, 4] = float("nan" if val == "key" else val)
        elif val == "key":
            b.kc[int(b.bt[s, 6]), :, 4, 3] = 0x7E if kv == "e5m2" else float("nan")
        else:
            _plant(b, s, 100, [3, 64], val)
    t = _time(b)
    # Rows before it in its unit do not see it and are computed again: at most 32 a warp, four steps of 32
    # positions each (of 4096 tokens; else none), a step of at most 8 us: two passes over K and V rows
    # from memory, some 1 us each, and 15 shuffles, three times over.
    again = 32 * 4 * 0.008 if ns[0] > 100 else 0.0
    print(f"{kv} {val} {ns[0]} over {lens[0]}: {plain * 1e3:.0f} us, {t * 1e3:.0f} us with it")
    assert t < 10 * plain + 0.05 + again
