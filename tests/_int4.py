"""The INT4 cache in 64 bits: its codec, its layout and attention over it with an error bound.
Dimensions are taken one at a time, by the layout's definition."""
from __future__ import annotations

import math

import torch

BLOCK, GROUP = 16, 64
U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}   # half a step, relative


def _fp16(x, up):
    """The nearest fp16 number not below (up) or not above x, |x| <= 65504, in 64 bits."""
    step = torch.exp2((torch.frexp(x)[1].double() - 11).clamp(min=-24))
    return (torch.ceil if up else torch.floor)(x / step) * step


def quantised(x):
    """(codes [.., D] int64, s, z [.., D/64]) of fp16 or bf16 rows; a group that is not finite has
    codes 0, s = NaN, z = 0."""
    x = x.double().reshape(*x.shape[:-1], -1, GROUP)
    good = x.isfinite().all(-1)
    x = torch.where(good[..., None], x, 0.0).clamp(-65504, 65504)
    z = _fp16(x.min(-1)[0], False)
    s = _fp16((x.max(-1)[0] - z) / 15, True)
    best, codes = (x - z[..., None]).abs(), torch.zeros_like(x, dtype=torch.int64)
    for c in list(range(2, 16, 2)) + list(range(1, 16, 2)):   # halfway: the even code stays
        y = (x - (z + c * s)[..., None]).abs()
        codes = torch.where(y < best, c, codes)
        best = torch.minimum(best, y)
    s = torch.where(good, s, math.nan)
    return codes.flatten(-2), s, torch.where(good, z, 0.0)


def _place(d, dim):
    """(byte of the row, shift in the byte) of a dimension."""
    g, unit, e = dim // GROUP, dim % GROUP // 8, dim % 8
    bit = 2 * e if e % 2 == 0 else 16 + 2 * (e - 1)
    return 4 * (unit * (d // GROUP) + g) + bit // 8, bit % 8


def pack(codes):
    d = codes.shape[-1]
    out = torch.zeros((*codes.shape[:-1], d // 2), dtype=torch.int64, device=codes.device)
    for i in range(d):
        byte, shift = _place(d, i)
        out[..., byte] += codes[..., i] << shift
    return out.to(torch.uint8)


def unpack(rows):
    d = 2 * rows.shape[-1]
    rows = rows.to(torch.int64)
    return torch.stack([(rows[..., b] >> s) & 15 for b, s in (_place(d, i) for i in range(d))], -1)


def stand_for(codes, s, z):
    """Values of rows in 64 bits, and their parts s |c - 8| + |z + 8 s|."""
    c = codes.double().reshape(*codes.shape[:-1], -1, GROUP)
    s, z = s.double()[..., None], z.double()[..., None]
    return (z + s * c).flatten(-2), (s.abs() * (c - 8).abs()).flatten(-2), ((z + 8 * s).abs() + 0 * c).flatten(-2)


def make_cache(blocks, hkv, d, gen, dev, spread=1.0, bias=0.0):
    """(k_cache, v_cache, scales) that hold unit-variance rows; spread: V rows differ in size by up
    to 2^spread either way; bias: keys' means by dimension."""
    out = []
    scales = torch.zeros((blocks, hkv, 2, BLOCK, d // GROUP, 2), dtype=torch.float16, device=dev)
    for w in range(2):
        x = torch.randn((blocks, hkv, BLOCK, d), generator=gen, device=dev)
        if w == 0:
            x += bias * torch.randn((hkv, 1, d), generator=gen, device=dev)
        else:
            x *= torch.exp2((torch.rand((blocks, hkv, BLOCK, 1), generator=gen, device=dev) * 2 - 1) * (spread - 1.0))
        codes, s, z = quantised(x.half())
        out.append(pack(codes))
        scales[:, :, w, :, :, 0], scales[:, :, w, :, :, 1] = s.half(), z.half()
    return out[0], out[1], scales


def rows_of(cache, scales, which, blk, off):
    """Rows (values, |s (c - 8)|, |z + 8 s|) [n, head, D] of the named slots."""
    sc = scales[blk, :, which, off]
    return stand_for(unpack(cache[blk, :, off]), sc[..., 0], sc[..., 1])


def chain(n, dev):
    return torch.tensor([(2 << j) - 1 - (1 << 64 if j == 63 else 0) for j in range(n)], dtype=torch.int64, device=dev)


def attention(q, k_cache, v_cache, scales, tables, lens, cu, scale, masks=None):
    """(out, bound) in 64 bits. masks: per query row, int64 (None: a chain, of any length). With
    p the weights and u the output's half step, an element may be off by
      u |o|                                  the output's rounding,
      2^-11 sum p s |c - 8|                  P = p s rounded to fp16,
      2 (e + ctx 2^-23 + 2^-20) sum p (s |c - 8| + |z + 8 s|)   fp32 scores (e = (D + 16) 2^-24 scale
                                             sum |q| (s c + |z|)), exponentials, sums, numerator and denominator,
      ctx 2^-30 max s                        a P below fp16's normal range: 2^-25 of a unit in which
                                             the largest lies between 2^10 and 2^15, times at most 8."""
    R, hq, d = q.shape
    hkv = k_cache.shape[1]
    g = hq // hkv
    out = torch.full((R, hq, d), math.nan, dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(out)
    for s, ctx in enumerate(lens):
        a, b = int(cu[s]), int(cu[s + 1])
        n = b - a
        if n == 0:
            continue
        p = torch.arange(ctx, device=q.device)
        blk, off = tables[s, p // BLOCK].long(), p % BLOCK
        k, kc, kz = (x.transpose(0, 1).repeat_interleave(g, 0) for x in rows_of(k_cache, scales, 0, blk, off))
        v, vc, vz = (x.transpose(0, 1).repeat_interleave(g, 0) for x in rows_of(v_cache, scales, 1, blk, off))
        x = q[a:b].double().transpose(0, 1)
        i = p - (ctx - n)
        if masks is None:
            seen = i <= torch.arange(n, device=q.device)[:, None]
        else:
            seen = (i < 0) | ((i < 64) & (((masks[a:b, None] >> i.clamp(0, 63)) & 1) != 0))
        # (an unseen key or value may be NaN)
        score = ((x @ torch.where(k.isfinite(), k, 0.0).transpose(1, 2)) * scale).masked_fill(~seen, -math.inf)
        w = torch.softmax(score, -1)
        w = torch.where(seen.any(-1)[:, None], w, 0.0)
        v, vc, vz = (torch.where(t.isfinite(), t, 0.0) for t in (v, vc, vz))
        o = w @ v
        e = (d + 16) * 2.0 ** -24 * abs(scale) * (x.abs() @ (kc + kz).nan_to_num(0.0).transpose(1, 2) * 2).amax(-1, keepdim=True)
        smax = scales[blk, :, 1, off][..., 0].double().abs().nan_to_num(0.0).max()
        out[a:b] = o.transpose(0, 1)
        tol[a:b] = (U[q.dtype] * o.abs() + 2.0 ** -11 * (w @ vc) + 2 * (e + ctx * 2.0 ** -23 + 2.0 ** -20) * (w @ (vc + vz)) +
                    ctx * 2.0 ** -30 * smax).transpose(0, 1)
    return out, tol


def assert_within(got, want, tol, what=""):
    g = got.double()
    assert torch.isfinite(g).all(), f"{what}: non-finite output"
    ratio = ((g - want).abs() / tol.clamp(min=1e-300))
    assert ratio.max().item() <= 1, f"{what}: {int((ratio > 1).sum())} of {ratio.numel()} past the bound, at most {ratio.max().item():.2f} times it"
    return ratio.max().item()


def tables_for(lens, gen, dev, spare=3):
    need = [-(-max(c, 1) // BLOCK) for c in lens]
    total = sum(need) + spare
    order = torch.randperm(total, generator=gen, device=dev).to(torch.int32)
    bt = torch.full((len(lens), max(need)), 1 << 30, dtype=torch.int32, device=dev)
    at = 0
    for s, n in enumerate(need):
        bt[s, :n] = order[at:at + n]
        at += n
    return bt, total
