"""Long contexts whose every tile, block and planted position shows in the outputs.

Values are 0 or 1, so a dimension of the output is the weight of the positions that have a 1 there, and the
error bound is relative to it. "blocks": the first half of the dimensions by the block's index (a lost or doubled
block changes one by more than the bound), the second half by the place in the context (a piece joined with a
wrong weight does). "peaks": single positions at the edges of blocks, tiles and the context that all rows weigh
highly, a dimension each."""
from __future__ import annotations

import torch

import _operators as op

SHAPES = {  # name: (D, hq, hkv, new tokens, context lengths, the sequence that is long)
    "few": (128, 8, 2, [3], [20011], 0),
    "joined-in-groups": (128, 8, 2, [40], [20011], 0),
    "shared-context": (64, 8, 2, [150, 1], [30005, 7], 0),
    "chunk": (128, 8, 2, [260], [9000], 0),
    "narrow-few": (64, 4, 1, [5], [17000], 0),
}


def peaks_of(ctx, n):
    past = ctx - n
    return sorted({0, 15, 16, 127, 128, 255, 256, 383, 384, 2047, 2048, 4095, 4096, ctx // 2, past // 128 * 128 - 1,
                   past // 128 * 128 - 128, past // 16 * 16 - 1, past - 1})


def _write(b, s, k, v):
    """k and v [kv head][position][dimension] into the batch's caches, as their type holds them."""
    ctx = b.lens[s]
    p = torch.arange(ctx, device=k.device)
    blk, off = b.bt[s].long()[p // op.BLOCK], p % op.BLOCK
    for which, (x, cache) in enumerate(((k, b.kc), (v, b.vc))):
        x = x.transpose(0, 1)
        if b.sc is not None:
            scale = torch.tensor((0.01, 1 / 127)[which]).half().float()
            b.sc[blk, :, which, off] = scale.to(k.device)
            x = ((x / scale).round().clamp(-127, 127) - 128).to(torch.int8)
        elif cache.dtype == torch.uint8:
            x = x.to(torch.float8_e5m2).view(torch.uint8)
        cache[blk, :, off] = x.to(cache.dtype)


def fill(b, s, how, seed=3):
    """Keys, values and queries of the batch's sequence s."""
    g = torch.Generator(device=b.q.device)
    g.manual_seed(seed)
    hq, d = b.q.shape[1:]
    hkv, ctx, n = b.kc.shape[1], b.lens[s], b.ns[s]

    def randn(*shape):
        return torch.randn(shape, generator=g, device=b.q.device)
    k, v = 0.3 * randn(hkv, ctx, d), torch.zeros((hkv, ctx, d), device=b.q.device)
    at = slice(b.cu_host[s], b.cu_host[s + 1])
    p = torch.arange(ctx, device=b.q.device)
    if how == "blocks":
        v[:, p, p // op.BLOCK % (d // 2)] = 1.0
        v[:, p, d // 2 + p * (d // 2) // ctx] = 1.0
        b.q[at] = randn(n, hq, d).to(b.q.dtype)
    else:
        w = torch.where(randn(d) > 0, 1.0, -1.0)
        for i, q in enumerate(peaks_of(ctx, n)):
            k[:, q] = (8.5 / d ** 0.5) * w           # scores of 8.5 beside 0.3
            v[:, q, i] = 1.0
        b.q[at] = (w + 0.3 * randn(n, hq, d)).to(b.q.dtype)
    _write(b, s, k, v)


def tokens_of(n):
    """New tokens to compare: the ends, and both sides of row tiles and units."""
    return sorted({j for j in (0, 1, 7, 8, 31, 32, 39, 63, 64, 65, 127, 128, n // 2, n - 2, n - 1) if 0 <= j < n})
