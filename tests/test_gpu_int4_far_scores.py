"""INT4 decode with scores far from zero, up to what fp16 queries and keys can make."""
import pytest
import torch

import _int4 as i4
from test_gpu_int4_attention import Case

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("size", [2.0 ** 18, 2.0 ** 25, 2.0 ** 27, 2.0 ** 30, 2.0 ** 36])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("g,n", [(1, 1), (4, 1), (8, 1), (4, 4), (8, 4), (8, 8), (5, 3)])
def test_one_token_stands_out(g, n, d, size):
    """Every row's best token lies half its score (at least 2^7) above all others, so the row is that token's values, whatever fp32 loses of
    the scores: off by the output's rounding and by P's, 2^-11 s |c - 8|, with s |c - 8| <= 8 s; all else (sums of zeros, one
    product, one division) by less than 2^-20 of the two."""
    hkv = 2
    c = Case([max(n, x) for x in (1, 2, 17, 40, 333, 1200)], g * hkv, hkv, d, torch.float16, n=n, seed=g * n)
    c.q = (torch.rand(c.q.shape, generator=c.g, device=DEV) * 0.25 + 1).half() * 32768 if size > 2.0 ** 30 else \
        (torch.rand(c.q.shape, generator=c.g, device=DEV) * 0.25 + 1).half()
    level = torch.exp2(-torch.randint(1, 10, c.sc.shape[:2] + (16,), generator=c.g, device=DEV).double())
    # (the last n positions, which not every row sees, are the lowest; of the others one stands out, else the own token does)
    for s, ctx in enumerate(c.lens):
        p = torch.arange(ctx, device=DEV)
        blk, off = c.tables[s, p // 16].long(), p % 16
        level[blk, :, off] = level[blk, :, off].clamp(max=0.25)
        level[blk[ctx - n:], :, off[ctx - n:]] = torch.exp2(torch.arange(n, device=DEV).double() - n - 1)[:, None]
        if ctx > n:
            best = int(torch.randint(0, ctx - n, (1,), generator=c.g, device=DEV))
            level[blk[best], :, off[best]] = 1.0
    top = 60000.0 if size > 2.0 ** 30 else 1024.0
    c.sc[:, :, 0, :, :, 1] = (level * top).half()[..., None]
    c.sc[:, :, 0, :, :, 0] = (level * top * 2.0 ** -9).half()[..., None]
    c.scale = size / (float(c.q.double().mean()) * top * d)
    want, _ = c.want()
    smax = float(c.sc[:, :, 1, :, :, 0].double().max())
    tol = (i4.U[torch.float16] * want.abs() + 2.0 ** -11 * 8 * smax) * (1 + 2.0 ** -10)
    i4.assert_within(c.fixed(), want, tol)
    i4.assert_within(c.varlen(), want, tol)
