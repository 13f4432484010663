"""How far a prefill output may be from the 64-bit one, term by term from the kernel's arithmetic.

With p a row's weights, v the values, o = sum p v, A = sum p |v|, u the half step of the query's
type, n the row's visible positions:

* the output's rounding: u |o|, and half of the type's least step;
* the weights' rounding to the type: u A. Below fp16's normal range a weight (over INT8 its product
  with the V scale) is off by at most 2^-25 in units of the row's sums. The largest weight is 2^7
  or more of such units, so n positions add at most n 2^-32 max p max |v|. Over INT8 the largest
  product is 2^4 or more and a code at most 127: n 2^-29 max (p 127 scale), where a V scale below 2^-32
  counts as that;
* the fp32 scores: a dot product is D / 16 product steps of 16 elements, at most 16 + D / 16 roundings
  of 2^-23 (a step may cut where it does not round); four more of 2^-24 of the largest score (the scale,
  the FMA, the maximum; over INT8 of the exponent, at most 32, too), and 2^-21 for the exponential.
  With e_j their sum for position j: sum p e |v| + |o| sum p e;
* the fp32 sums: of values n / 16 product steps, one rescaling a tile and the join of at most 152
  pieces, of 2^-23 each; of weights 32 in a tile, one a tile and the pieces, of 2^-24 each."""
from __future__ import annotations

import math

import torch

import _operators as op


def row_bound(q, k, v, scale, v_scale=None):
    """(out, bound), [rows][dimension] in 64 bits, of rows that all see k and v (one head's, n positions; an
    INT8 cache's v comes with its V scales [n])."""
    u = op.HALF_STEP[q.dtype]
    k, v = k.double(), v.double()
    n, d = k.shape
    x = q.double()
    s = x @ k.T * scale
    p = torch.softmax(s, -1)
    o, big = p @ v, p @ v.abs()
    wide = s.abs().amax(-1, keepdim=True) + (0.0 if v_scale is None else 32 * math.log(2.0))
    e = (16 + d / 16) * 2.0 ** -23 * scale * (x.abs() @ k.abs().T) + 4 * 2.0 ** -24 * wide + 2.0 ** -21
    pe = p * e
    tol = u * o.abs() + u * big + pe @ v.abs() + o.abs() * pe.sum(-1, keepdim=True)
    tol += (n / 16 + n / 128 + 152) * 2.0 ** -23 * big + (32 + n / 128 + 152) * 2.0 ** -24 * o.abs()
    if v_scale is not None:
        tol += n * 2.0 ** -29 * (p * (127.0 * v_scale.double().abs().clamp(min=2.0 ** -32))).amax(-1, keepdim=True)
    elif q.dtype == torch.float16:
        tol += n * 2.0 ** -32 * p.amax(-1, keepdim=True) * v.abs().max()
    return o, tol + (2.0 ** -25 if q.dtype == torch.float16 else 0.0)


def seen_rows(b, s):
    """(k, v, V scales or None) of a test batch's sequence s in 64 bits, [kv head][position][dimension]."""
    ctx, hkv, d = b.lens[s], b.kc.shape[1], b.kc.shape[3]
    ids = b.bt[s, :-(-ctx // op.BLOCK)].long()
    sc = None if b.sc is None else b.sc[ids]

    def rows(cache, which):
        return op.cache_rows(cache[ids], sc, which).transpose(0, 1).reshape(hkv, -1, d)[:, :ctx]
    return rows(b.kc, 0), rows(b.vc, 1), None if sc is None else sc[:, :, 1].transpose(0, 1).reshape(hkv, -1)[:, :ctx]


def attention_rows(b, s, tokens=None):
    """(rows of q/out, out, bound) of sequence s of a test batch: the given (default: all) new tokens, all
    heads, in 64 bits."""
    a, e, ctx = b.cu_host[s], b.cu_host[s + 1], b.lens[s]
    hq, d = b.q.shape[1:]
    k, v, vs = seen_rows(b, s)
    at = list(range(e - a)) if tokens is None else list(tokens)
    out = torch.empty((len(at), hq, d), dtype=torch.float64, device=b.q.device)
    tol = torch.empty_like(out)
    group = hq // b.kc.shape[1]
    for i, j in enumerate(at):
        n = ctx - (e - a) + j + 1
        for g in range(b.kc.shape[1]):
            h = slice(g * group, (g + 1) * group)
            out[i, h], tol[i, h] = row_bound(b.q[a + j, h], k[g, :n], v[g, :n], b.scale, None if vs is None else vs[g, :n])
    return (slice(a, e) if tokens is None else [a + j for j in at]), out, tol


def check_rows(b, what=""):
    """The batch's outputs against 64 bits, every sequence by itself."""
    worst = 0.0
    for s in range(len(b.lens)):
        if b.cu_host[s + 1] > b.cu_host[s]:
            at, want, tol = attention_rows(b, s)
            worst = max(worst, op.assert_within(b.out[at], want, tol, f"{what} sequence {s}"))
    print(f"{what}: at most {worst:.2f} of the bound")
