"""The prefill tests' long contexts and bound, with mistakes planted in the 64-bit outputs: each must show.
No GPU needed."""
import pytest
import torch

import _bounds
import _exposing as ex
from test_gpu_prefill import Batch

CPU = torch.device("cpu")


def _row(kv, shape, how):
    """(weights, values, out, bound, positions seen) of the last new token, first head."""
    D, hq, hkv, ns, lens, s = ex.SHAPES[shape]
    b = Batch(CPU, kv, D, hq, hkv, ns, lens)
    ex.fill(b, s, how)
    k, v, vs = _bounds.seen_rows(b, s)
    q = b.q[b.cu_host[s + 1] - 1, :1]
    out, tol = _bounds.row_bound(q, k[0], v[0], b.scale, None if vs is None else vs[0])
    p = torch.softmax(q.double() @ k[0].T * b.scale, -1)[0]
    return p, v[0], out[0], tol[0], lens[s]


def _shows(p, v, out, tol, factors):
    """Outputs with the weights times each of the factors [cases][positions]: in which does one leave the bound."""
    w = p * factors
    got = (w @ v) / w.sum(-1, keepdim=True)
    return ((got - out).abs() > tol).any(-1)


@pytest.mark.parametrize("kv", ["fp16", "bf16", "e5m2", "int8"])
@pytest.mark.parametrize("shape", list(ex.SHAPES))
def test_lost_blocks_and_tiles_show(kv, shape):
    p, v, out, tol, n = _row(kv, shape, "blocks")
    at = torch.arange(n)
    for size in (16, 128):
        count = -(-n // size)
        for first in range(0, count, 128):
            c = torch.arange(first, min(first + 128, count))
            lost = (at // size != c[:, None]).double()
            whole = c < n // size                    # (a last block of a few positions weighs less)
            assert _shows(p, v, out, tol, lost)[whole].all(), f"{size} positions lost"
            assert _shows(p, v, out, tol, 2.0 - lost)[whole].all(), f"{size} positions twice"


@pytest.mark.parametrize("kv", ["fp16", "bf16", "e5m2", "int8"])
@pytest.mark.parametrize("shape", list(ex.SHAPES))
def test_pieces_of_a_wrong_weight_show(kv, shape):
    """Three to thirteen tiles weighted 5 % too much or too little."""
    p, v, out, tol, n = _row(kv, shape, "blocks")
    at = torch.arange(n)
    for tiles in (3, 6, 13):
        first = torch.arange(0, n // 128 - tiles, tiles)[:, None]
        inside = ((at // 128 >= first) & (at // 128 < first + tiles)).double()
        wide = tiles * 128 >= 2 * n // (v.shape[1] // 2)     # covers at least one place dimension whole
        for by in (0.05, -0.05, 0.5):
            if wide or by == 0.5:
                assert _shows(p, v, out, tol, 1.0 + by * inside).all(), f"{tiles} tiles, {by}"


@pytest.mark.parametrize("kv", ["fp16", "bf16", "e5m2", "int8"])
@pytest.mark.parametrize("shape", list(ex.SHAPES))
def test_single_positions_show(kv, shape):
    p, v, out, tol, n = _row(kv, shape, "peaks")
    at = torch.tensor(ex.peaks_of(n, ex.SHAPES[shape][3][0]))
    lost = torch.ones((len(at), n), dtype=torch.float64)
    lost[torch.arange(len(at)), at] = 0.0
    assert _shows(p, v, out, tol, lost).all()
    assert _shows(p, v, out, tol, torch.where(lost == 0.0, 1.02, 1.0)).all(), "2 % of one weight"
