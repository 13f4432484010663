"""INT4 decode over values of small and of very unequal scales: weights p s, held in fp16, must keep the bits of small scales."""
import math

import pytest
import torch

import _int4 as i4
from test_gpu_int4_attention import Case

pytestmark = pytest.mark.gpu
DEV = "cuda"
ROWS = [(1, 1), (4, 1), (8, 1), (4, 4), (8, 4), (8, 8)]


def _parts(c):
    """w @ |s (c - 8)| and w @ |z + 8 s| of every output, and the scores' error e, as i4.attention takes them."""
    part, both, err = [], [], []
    for s, ctx in enumerate(c.lens):
        p = torch.arange(ctx, device=DEV)
        blk, off = c.tables[s, p // 16].long(), p % 16
        g = c.q.shape[1] // c.k.shape[1]
        k, kc, kz = (x.transpose(0, 1).repeat_interleave(g, 0) for x in i4.rows_of(c.k, c.sc, 0, blk, off))
        _, vc, vz = (x.transpose(0, 1).repeat_interleave(g, 0) for x in i4.rows_of(c.v, c.sc, 1, blk, off))
        x = c.q[c.cu[s]:c.cu[s + 1]].double().transpose(0, 1)
        n = x.shape[1]
        seen = p - (ctx - n) <= torch.arange(n, device=DEV)[:, None]
        w = torch.softmax(((x @ k.transpose(1, 2)) * c.scale).masked_fill(~seen, -math.inf), -1)
        e = (x.shape[-1] + 16) * 2.0 ** -24 * c.scale * (x.abs() @ (kc + kz).transpose(1, 2) * 2).amax(-1, keepdim=True) + ctx * 2.0 ** -23 + 2.0 ** -20
        part.append((w @ vc).transpose(0, 1))
        both.append((2 * e * (w @ (vc + vz))).transpose(0, 1))
    return torch.cat(part), torch.cat(both)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("g,n", ROWS)
@pytest.mark.parametrize("low,high", [(-24, -18), (-24, -23), (-24, -6), (-15, -13)])
def test_all_scales_small(g, n, d, low, high):
    """V scales of 2^low to 2^high, down to fp16's least number: p reaches some 2^35 beside them. bf16 outputs (fp16 ones would be
    subnormal); the bound is that of i4.attention without its last term but for scales 2^-8 and further below the largest: a P
    that is 2^-25 of a unit off, where the largest lies above 2^10 / 2^3 (scores within 2^3 of one another)."""
    c = Case([max(n, x) for x in (1, 2, 40, 700)], 2 * g, 2, d, torch.bfloat16, n=n, seed=g * n + d)
    c.q *= 0.25
    shape = c.sc.shape[:2] + c.sc.shape[3:5]
    s = torch.exp2(torch.rand(shape, generator=c.g, device=DEV) * (high - low) + low).clamp(min=2.0 ** -24)
    c.sc[:, :, 1, :, :, 0] = s.half()
    c.sc[:, :, 1, :, :, 1] = (-s * torch.rand(shape, generator=c.g, device=DEV) * 15).half()
    want, _ = c.want()
    part, both = _parts(c)
    tol = 2.0 ** -8 * want.abs() + 2.0 ** -11 * part + both + 8 * 2.0 ** (3 - 35) * float(c.sc[:, :, 1, ..., 0].double().max())
    i4.assert_within(c.fixed(), want, tol)


@pytest.mark.parametrize("g,n", ROWS)
@pytest.mark.parametrize("apart", [6, 12, 20, 28])
@pytest.mark.parametrize("small", [0, 1])
def test_groups_of_unequal_scales(g, n, apart, small):
    """One group of every value row has scales 2^-apart of the other's. Both groups' weights go by the larger one: their largest
    lies above 2^10, the others' (scores within 2^3) above 2^7, so that a smaller group's are normal fp16 numbers, off by 2^-11,
    down to 2^-20 of it, and beyond that off by 2^-25 of a unit, 2^-32 of the larger group's scale a code."""
    c = Case([max(n, x) for x in (1, 2, 40, 700)], 2 * g, 2, 128, torch.bfloat16, n=n, seed=g * n + apart)
    c.q *= 0.25
    shape = c.sc.shape[:2] + (16,)
    s = 4096 * (1 + torch.rand(shape, generator=c.g, device=DEV))
    for group in range(2):
        x = s * (2.0 ** -apart if group == small else 1.0)
        c.sc[:, :, 1, :, group, 0] = x.half()
        c.sc[:, :, 1, :, group, 1] = (-8 * x).half().clamp(min=-65504)
    want, _ = c.want()
    part, both = _parts(c)
    tol = 2.0 ** -8 * want.abs() + 2.0 ** -11 * part + both
    if apart > 20:
        tol = tol + 8 * 2.0 ** -32 * float(c.sc[:, :, 1, ..., 0].double().max())
    i4.assert_within(c.fixed(), want, tol)
