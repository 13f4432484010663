"""Plain 64-bit forms of the rotary, prefill and accept operators and the inputs their GPU
tests share. Everything works on the caches the library reads, through block tables."""
from __future__ import annotations

import math

import torch

BLOCK = 16
HALF_STEP = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float8_e5m2: 2.0 ** -3}


def src_dtype(kv):
    return torch.bfloat16 if kv == "bf16" else torch.float16


def make_cache(kv, blocks, hkv, d, gen, dev):
    """(k_cache, v_cache, scales or None) holding unit-variance values."""
    shape = (blocks, hkv, BLOCK, d)

    def randn():
        return torch.randn(shape, generator=gen, device=dev)
    if kv == "int8":
        codes = [torch.randint(-127, 128, shape, generator=gen, device=dev, dtype=torch.int16) for _ in range(2)]
        k, v = ((c - 128).to(torch.int8) for c in codes)
        sc = (torch.rand((blocks, hkv, 2, BLOCK), generator=gen, device=dev) * 0.02 + 0.005).half().float()
        return k, v, sc
    if kv == "e5m2":
        return tuple(randn().to(torch.float8_e5m2).view(torch.uint8) for _ in range(2)) + (None,)
    return randn().to(src_dtype(kv)), randn().to(src_dtype(kv)), None


def cache_rows(cache, scales=None, which=0):
    """The cache's numbers in 64 bits, [block][kv head][offset][dimension]."""
    if cache.dtype == torch.int8:
        code = cache.view(torch.uint8).double() - 128.0
        return code * scales[:, :, which, :, None].double()
    if cache.dtype == torch.uint8:
        return cache.view(torch.float8_e5m2).double()
    return cache.double()


def tables(lens, gen, dev, spare=3):
    """Block tables over a shuffled pool, and its block count; unused entries are out of range."""
    need = [-(-c // BLOCK) for c in lens]
    total = sum(need) + spare
    order = torch.randperm(total, generator=gen, device=dev).to(torch.int32)
    bt = torch.full((len(lens), max(1, max(need, default=1))), 1 << 30, dtype=torch.int32, device=dev)
    at = 0
    for s, n in enumerate(need):
        bt[s, :n] = order[at:at + n]
        at += n
    return bt, total


def attention_bound(q, k_cache, v_cache, scales, bt, cu, lens, scale):
    """(out, bound) in 64 bits: the attention of every sequence's rows and how far an output
    may be from it. Per element, with u the half step of q's type, p the weights, A = sum p |v|:
      u |o|                      the output's rounding,
      u A                        the probabilities' rounding to q's type,
      2 (e + ctx 2^-24) A        fp32 scores (e = D 2^-24 scale sum |q||k|, an exponent's absolute
                                 error), exponentials (2^-21) and sums, numerator and denominator,
      ctx 2^-24                  probabilities below fp16's normal range (steps of 2^-24 of a
                                 scaled probability, times |v| or an INT8 code)."""
    R, hq, d = q.shape
    hkv = k_cache.shape[1]
    g = hq // hkv
    u = HALF_STEP[q.dtype]
    k_all, v_all = cache_rows(k_cache, scales, 0), cache_rows(v_cache, scales, 1)
    out = torch.full((R, hq, d), float("nan"), dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(out)
    for s, ctx in enumerate(lens):
        a, b = cu[s], cu[s + 1]
        n = b - a
        if n == 0:
            continue
        ids = bt[s, :-(-ctx // BLOCK)].long()
        k = k_all[ids].transpose(0, 1).reshape(hkv, -1, d)[:, :ctx].repeat_interleave(g, 0)
        v = v_all[ids].transpose(0, 1).reshape(hkv, -1, d)[:, :ctx].repeat_interleave(g, 0)
        x = q[a:b].double().transpose(0, 1)
        score = x @ k.transpose(1, 2) * scale
        seen = torch.arange(ctx, device=q.device) <= torch.arange(ctx - n, ctx, device=q.device)[:, None]
        score = score.masked_fill(~seen, -math.inf)
        p = torch.softmax(score, -1)
        empty = ~seen.any(-1)
        p = torch.where(empty[:, None], torch.zeros_like(p), p)
        v0 = torch.where(v.isfinite(), v, torch.zeros_like(v)) if not v.isfinite().all() else v
        o = p @ v0
        big = p @ v0.abs()
        e = d * 2.0 ** -24 * scale * (x.abs() @ k.abs().nan_to_num(0.0, 0.0, 0.0).transpose(1, 2)).amax(-1, keepdim=True) + 2.0 ** -21
        out[a:b] = o.transpose(0, 1)
        tol[a:b] = (u * o.abs() + u * big + 2 * (e + ctx * 2.0 ** -24) * big + ctx * 2.0 ** -24).transpose(0, 1)
    return out, tol


def assert_within(got, want, tol, what=""):
    g = got.double()
    assert torch.isfinite(g).all(), f"{what}: non-finite output"
    over = (g - want).abs() - tol
    worst = over.max().item()
    ratio = ((g - want).abs() / tol.clamp(min=1e-300)).max().item()
    assert worst <= 0, f"{what}: {int((over > 0).sum())} of {over.numel()} past the bound, at most {ratio:.2f} times it"
    return ratio


def turn(x, positions, inv_freq, interleaved, factor=1.0, inverse=False):
    """Rotary embedding in 64 bits, on complex pairs."""
    half = inv_freq.shape[0]
    ang = positions.double()[:, None] * inv_freq * (-1 if inverse else 1)
    z = torch.polar(torch.full_like(ang, 1.0), ang) * factor
    j = torch.arange(half, device=x.device)
    re, im = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
    y = x.double().clone()
    w = torch.complex(y[..., re], y[..., im]) * z[:, None]
    y[..., re], y[..., im] = w.real, w.imag
    return y
