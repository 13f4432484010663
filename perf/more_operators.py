"""What is measured of the 4-bit KV cache: quantising tokens as they are written, reading
a cache back, and the attention of decode and verify steps over it.

Each case names one operator ("op"):

* ``store``: new tokens' keys and values quantised into their slots of the INT4 cache, and
  read back as the values the cache then stands for.
* ``read``: rows of a cache (INT4 or INT8) gathered by slot into dense keys and values.
* ``attend``: attention of every sequence's newest tokens over its blocks of the INT4 cache:
  one token each, draft chains, ragged counts, token trees.

The INT4 cache. A row (token, KV head) of D dimensions is D/64 groups of 64. A group holds
its least value z and a scale s, both fp16, and 64 codes c of 4 bits: dimension d stands for
z + s c_d, with z the largest fp16 number not above the group's least value, s the smallest one
not below (largest - z) / 15, c the code whose value is nearest (halfway: the even one).
Codes are bytes [block][KV head][16][D/2], scales fp16 [block][KV head][K, V][16][D/64][s, z].
A row is D/8 32-bit words; word i * D/64 + g holds the eight dimensions 64 g + 8 i + e, even e
at bit 2 e, odd e at bit 16 + 2 (e - 1).

``run`` computes an operator in plain torch operations where ``own`` is false and
through the package where it is true; ``exact`` computes it in 64 bits.
"""
import math
import random

import torch

own = False

DEVICE = "cuda"
BLOCK = 16
GROUP = 64
TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


# ---- cases ---------------------------------------------------------------------------

def listed():
    heads8b = {"hq": 32, "hkv": 8, "d": 128}
    heads70b = {"hq": 64, "hkv": 8, "d": 128}
    return [
        # the new tokens of one decode step of 64 sequences, where latency counts
        {"name": "store-decode-fp16", "op": "store", "type": "fp16", "hkv": 8, "d": 128, "tokens": 64},
        # a whole prompt
        {"name": "store-prompt-bf16", "op": "store", "type": "bf16", "hkv": 8, "d": 128, "tokens": 8192},
        # head size 64, an odd number of tokens
        {"name": "store-odd-fp16", "op": "store", "type": "fp16", "hkv": 4, "d": 64, "tokens": 2001},
        # a cached prefix handed on as dense rows
        {"name": "read-prefix-bf16", "op": "read", "kv": "int4", "type": "bf16", "hkv": 8, "d": 128, "tokens": 4097},
        # a long document's cache moved out: the largest read
        {"name": "read-document-fp16", "op": "read", "kv": "int4", "type": "fp16", "hkv": 8, "d": 128, "tokens": 65536},
        # an INT8 cache of a small model
        {"name": "read-int8-fp16", "op": "read", "kv": "int8", "type": "fp16", "hkv": 4, "d": 64, "tokens": 1000},
        # one token over a short context: the smallest call
        {"name": "attend-short-fp16", "op": "attend", "type": "fp16", **heads8b, "seqs": 1, "n": 1, "ragged": False,
         "tree": False, "ctx_lo": 33, "ctx_hi": 33, "shape": 1},
        # a decode step of 64 sequences
        {"name": "attend-batch64-fp16", "op": "attend", "type": "fp16", **heads8b, "seqs": 64, "n": 1, "ragged": False,
         "tree": False, "ctx_lo": 128, "ctx_hi": 2048, "shape": 2},
        # a decode step of 256 sequences
        {"name": "attend-batch256-bf16", "op": "attend", "type": "bf16", **heads8b, "seqs": 256, "n": 1, "ragged": False,
         "tree": False, "ctx_lo": 128, "ctx_hi": 4096, "shape": 3},
        # four long documents: a sequence's context split over many CTAs
        {"name": "attend-long-bf16", "op": "attend", "type": "bf16", **heads8b, "seqs": 4, "n": 1, "ragged": False,
         "tree": False, "ctx_lo": 100000, "ctx_hi": 131072, "shape": 4},
        # a verify step: four draft tokens in a chain
        {"name": "attend-verify-fp16", "op": "attend", "type": "fp16", **heads70b, "seqs": 128, "n": 4, "ragged": False,
         "tree": False, "ctx_lo": 256, "ctx_hi": 8192, "shape": 5},
        # token trees of up to 16 drafts, a different number a sequence, head size 64
        {"name": "attend-tree-bf16", "op": "attend", "type": "bf16", "hq": 16, "hkv": 4, "d": 64, "seqs": 16, "n": 16,
         "ragged": True, "tree": True, "ctx_lo": 100, "ctx_hi": 4000, "shape": 6},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["store", "read", "attend", "attend"])
    d, hkv, kind = rng.choice([64, 128]), rng.choice([1, 2, 4, 8]), rng.choice(["fp16", "bf16"])
    if op == "store":
        return {"op": op, "type": kind, "hkv": hkv, "d": d, "tokens": _log_int(rng, 1, 8192)}
    if op == "read":
        return {"op": op, "kv": rng.choice(["int4", "int4", "int8"]), "type": kind, "hkv": hkv, "d": d,
                "tokens": _log_int(rng, 1, 65536)}
    g = rng.choice([1, 2, 3, 4, 6, 8])
    hi = _log_int(rng, 16, 131072)
    n = rng.choice([1, 1, 1, rng.randint(2, 64 // g)])
    case = {"op": op, "type": kind, "hq": hkv * g, "hkv": hkv, "d": d, "seqs": _log_int(rng, 1, 256), "n": n,
            "ragged": n > 1 and rng.random() < 0.5, "tree": n > 1 and rng.random() < 0.5,
            "ctx_lo": max(1, hi // rng.randint(1, 16)), "ctx_hi": hi, "shape": rng.randrange(1 << 30)}
    top_b, top_f = (max(work(c)[k] for c in listed() if c["op"] == "attend") for k in ("bytes", "flops"))
    while work(case)["bytes"] > top_b or work(case)["flops"] > top_f:
        k = rng.choice(["seqs", "ctx_hi"])
        case[k] = max(1, case[k] * 2 // 3)
        case["ctx_lo"] = min(case["ctx_lo"], case["ctx_hi"])
    return case


def _lens(case):
    """The sequences' (query tokens, context length with them), the same for every seed."""
    r = random.Random(case["shape"])
    lens = []
    for _ in range(case["seqs"]):
        n = r.randint(1, case["n"]) if case["ragged"] else case["n"]
        lens.append((n, max(n, r.randint(case["ctx_lo"], case["ctx_hi"]))))
    return lens


def _masks(case):
    """One mask of visible drafts for every query token: its ancestors in its sequence's token
    tree and itself (without a tree: every earlier draft)."""
    r = random.Random(case["shape"] + 1)
    masks = []
    for n, _ in _lens(case):
        seen = []
        for j in range(n):
            parent = (r.randint(-1, j - 1) if case["tree"] else j - 1) if j else -1
            seen.append((seen[parent] if parent >= 0 else 0) | 1 << j)
        masks.append(seen)
    return masks


def _row_bytes(kv, d):
    """Bytes of one row of K or V with its scales."""
    return d // 2 + 4 * (d // GROUP) if kv == "int4" else d + 4


def work(case):
    if case["op"] in ("store", "read"):
        rows = 2 * case["tokens"] * case["hkv"]
        passes = 2 if case["op"] == "store" else 1   # dense values in and out, or out alone
        return {"bytes": rows * (2 * passes * case["d"] + _row_bytes(case.get("kv", "int4"), case["d"])) +
                4 * case["tokens"], "flops": 0}
    b = f = 0
    for (n, ctx), seen in zip(_lens(case), _masks(case)):
        b += n * case["hq"] * case["d"] * 4 + 2 * ctx * case["hkv"] * _row_bytes("int4", case["d"])
        f += 4 * case["d"] * case["hq"] * (n * (ctx - n) + sum(bin(m).count("1") for m in seen))
    return {"bytes": b, "flops": f}


# ---- the cache's numbers -----------------------------------------------------------------

def _half_not_above(x):
    t = x.half()
    bits = t.view(torch.int16).int()
    down = torch.where(t > 0, bits - 1, torch.where(t == 0, -32767, bits + 1)).to(torch.int16).view(torch.float16)
    return torch.where(t.double() > x, down, t)


def _half_not_below(x):
    t = x.half()   # (x is not negative)
    up = (t.view(torch.int16) + 1).view(torch.float16)
    return torch.where(t.double() < x, up, t)


def _quantised(x):
    """(codes, s, z) of rows of D dimensions, in 64 bits where a value may lie beside a border
    between two codes."""
    x = x.double().unflatten(-1, (-1, GROUP))
    z = _half_not_above(x.amin(-1)) + 0.0
    s = _half_not_below((x.amax(-1) - z.double()) / 15)
    step = torch.where(s == 0, 1.0, s.double())
    return ((x - z.double().unsqueeze(-1)) / step.unsqueeze(-1)).round_().to(torch.uint8).flatten(-2), s, z


def _packed(codes):
    """Codes [..., D] as the cache's bytes [..., D/2]."""
    w = codes.int().unflatten(-1, (-1, 8, 8)).transpose(-2, -3)   # [..., i, g, e]
    shift = torch.tensor([2 * e if e % 2 == 0 else 16 + 2 * (e - 1) for e in range(8)], device=codes.device)
    return (w << shift).sum(-1, dtype=torch.int64).to(torch.int32).flatten(-2).view(torch.uint8)


def _codes(cache, kind):
    """Codes of a cache's rows [..., D] (INT8 codes lie in offset binary)."""
    if kind == "int8":
        return cache.view(torch.uint8).to(torch.int16) - 128
    w = cache.contiguous().view(torch.int32)
    out = torch.empty((*w.shape, 8), device=cache.device, dtype=torch.uint8)
    for e in range(8):
        out[..., e] = (w >> (2 * e if e % 2 == 0 else 16 + 2 * (e - 1))) & 15
    groups = w.shape[-1] // 8
    return out.unflatten(-2, (8, groups)).transpose(-2, -3).flatten(-3)


def _values(cache, scales, kind, blk, which, off=None):
    """Rows of one cache in 32 bits: whole blocks [n, head, 16, D], or single tokens [n, head, D]."""
    if off is None:
        c, sc = cache[blk], scales[blk][:, :, which]
    else:
        c, sc = cache[blk, :, off], scales[blk, :, which, off]
    x = _codes(c, kind).float()
    if kind == "int8":
        return x.mul_(sc.unsqueeze(-1))
    x = x.unflatten(-1, (-1, GROUP)).mul_(sc[..., 0].float().unsqueeze(-1)).add_(sc[..., 1].float().unsqueeze(-1))
    return x.flatten(-2)


# ---- inputs --------------------------------------------------------------------------

def _randn(g, shape, dtype=torch.float32):
    return torch.randn(shape, generator=g, device=DEVICE, dtype=torch.float32).to(dtype)


def _keys(g, shape, bias):
    """Keys: unit variance around a mean that differs from dimension to dimension."""
    return _randn(g, shape).add_(bias)


def _cache(case, blocks, g, empty=False):
    """A pool of blocks that earlier steps filled (or an empty one)."""
    hkv, d = case["hkv"], case["d"]
    kind = case.get("kv", "int4")
    if kind == "int8":
        k, v = (torch.randint(-127, 128, (blocks, hkv, BLOCK, d), generator=g, device=DEVICE, dtype=torch.int16)
                .sub_(128).to(torch.int8) for _ in range(2))
        return k, v, (torch.rand((blocks, hkv, 2, BLOCK), generator=g, device=DEVICE) * 0.02 + 0.01).half().float()
    k, v = (torch.zeros((blocks, hkv, BLOCK, d // 2), device=DEVICE, dtype=torch.uint8) for _ in range(2))
    scales = torch.zeros((blocks, hkv, 2, BLOCK, d // GROUP, 2), device=DEVICE, dtype=torch.float16)
    if empty:
        return k, v, scales
    bias = 2 * _randn(g, (hkv, 1, d))
    for b in range(0, blocks, 2048):
        n = min(2048, blocks - b)
        for which, (cache, x) in enumerate(((k, _keys(g, (n, hkv, BLOCK, d), bias)), (v, _randn(g, (n, hkv, BLOCK, d))))):
            codes, s, z = _quantised(x.half())
            cache[b:b + n] = _packed(codes)
            scales[b:b + n, :, which, :, :, 0], scales[b:b + n, :, which, :, :, 1] = s, z
    return k, v, scales


def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    st = {"case": case}
    dtype, d, hkv = TYPES[case["type"]], case["d"], case["hkv"]
    if case["op"] in ("store", "read"):
        t = case["tokens"]
        blocks = -(-t * 5 // (4 * BLOCK)) + 1
        st["k_cache"], st["v_cache"], st["scales"] = _cache(case, blocks, g, empty=case["op"] == "store")
        # the tokens' blocks lie anywhere in the pool, the tokens of a block in order
        pos = torch.arange(t, device=DEVICE)
        order = torch.randperm(blocks, generator=g, device=DEVICE)
        st["slots"] = (order[pos // BLOCK] * BLOCK + pos % BLOCK).to(torch.int32)
        if case["op"] == "store":
            st["key"] = _keys(g, (t, hkv, d), 2 * _randn(g, (hkv, d))).to(dtype)
            st["value"] = _randn(g, (t, hkv, d), dtype)
        return st
    lens = _lens(case)
    st["lens"] = lens
    need = [-(-ctx // BLOCK) for _, ctx in lens]
    total = sum(need) * 5 // 4 + 1
    order = torch.randperm(total, generator=g, device=DEVICE).to(torch.int32)
    st["tables"] = torch.zeros((len(lens), max(need)), device=DEVICE, dtype=torch.int32)
    at, cu = 0, [0]
    for s, n in enumerate(need):
        st["tables"][s, :n] = order[at:at + n]
        at += n
        cu.append(cu[-1] + lens[s][0])
    st["k_cache"], st["v_cache"], st["scales"] = _cache(case, total, g)
    st["context_lens"] = torch.tensor([ctx for _, ctx in lens], device=DEVICE, dtype=torch.int32)
    st["cu"] = torch.tensor(cu, device=DEVICE, dtype=torch.int32) if case["ragged"] else None
    masks = [m for seen in _masks(case) for m in seen]
    st["masks"] = torch.tensor([m - (1 << 64) if m >> 63 else m for m in masks], device=DEVICE, dtype=torch.int64)
    st["q"] = _randn(g, (cu[-1], case["hq"], d), dtype)
    st["scale"] = 1.0 / math.sqrt(d)
    return st


# ---- one pass ------------------------------------------------------------------------

def run(st):
    return {"store": _store, "read": _read, "attend": _attend}[st["case"]["op"]](st)


def _store(st):
    key, value, slots = st["key"], st["value"], st["slots"]
    k_cache, v_cache, scales = st["k_cache"], st["v_cache"], st["scales"]
    if own:
        import paged_kv_cache_252_gb300 as pkv
        pkv.kv_cache_write_int4(key, value, slots, k_cache, v_cache, scales)
        k, v = torch.empty_like(key), torch.empty_like(value)
        pkv.kv_cache_read(k, v, slots, k_cache, v_cache, "int4", scales=scales)
        return {"key": k, "value": v}
    blk, off = slots.long() // BLOCK, slots.long() % BLOCK
    out = {}
    for which, (name, x, cache) in enumerate((("key", key, k_cache), ("value", value, v_cache))):
        codes, s, z = _quantised(x)
        cache[blk, :, off] = _packed(codes)
        scales[blk, :, which, off] = torch.stack((s, z), -1)
        out[name] = _values(cache, scales, "int4", blk, which, off).to(x.dtype)
    return out


def _read(st):
    case, slots = st["case"], st["slots"]
    k_cache, v_cache, scales = st["k_cache"], st["v_cache"], st["scales"]
    dtype = TYPES[case["type"]]
    if own:
        import paged_kv_cache_252_gb300 as pkv
        k, v = (torch.empty((case["tokens"], case["hkv"], case["d"]), device=slots.device, dtype=dtype) for _ in range(2))
        pkv.kv_cache_read(k, v, slots, k_cache, v_cache, case["kv"], scales=scales)
        return {"key": k, "value": v}
    blk, off = slots.long() // BLOCK, slots.long() % BLOCK
    return {name: _values(cache, scales, case["kv"], blk, which, off).to(dtype)
            for which, (name, cache) in enumerate((("key", k_cache), ("value", v_cache)))}


def _visible(mask, n, ctx):
    """[n, ctx]: the context before the drafts, and the drafts that each token's mask names."""
    i = torch.arange(ctx, device=mask.device) - (ctx - n)
    return (i < 0) | ((mask[:, None] >> i.clamp(0, 63)) & 1).bool()


def _attend(st):
    q, case = st["q"], st["case"]
    if own:
        import paged_kv_cache_252_gb300 as pkv
        out = torch.empty_like(q)
        cache = (st["k_cache"], st["v_cache"])
        if case["tree"]:
            return pkv.paged_attention_decode_tree(out, q, st["masks"], *cache, st["tables"], st["context_lens"],
                                                   case["n"], st["scale"], "int4", cu_q_lens=st["cu"],
                                                   scales=st["scales"])
        if case["ragged"]:
            return pkv.paged_attention_decode_varlen(out, q, st["cu"], *cache, st["tables"], st["context_lens"],
                                                     case["n"], st["scale"], "int4", scales=st["scales"])
        return pkv.paged_attention_decode_int4(out, q, *cache, st["scales"], st["tables"], st["context_lens"], case["n"],
                                               st["scale"])
    hkv, d = case["hkv"], case["d"]
    g = case["hq"] // hkv
    out, row = torch.empty_like(q), 0
    # Sequences one by one: padding a ragged batch to its longest would cost far more.
    for s, (n, ctx) in enumerate(st["lens"]):
        ids = st["tables"][s, :-(-ctx // BLOCK)].long()
        k, v = (_values(c, st["scales"], "int4", ids, w).transpose(0, 1).flatten(1, 2)[:, :ctx]
                for w, c in enumerate((st["k_cache"], st["v_cache"])))
        x = q[row:row + n].float().mul_(st["scale"]).view(n, hkv, g, d).permute(1, 2, 0, 3).reshape(hkv, g * n, d)
        p = torch.matmul(x, k.transpose(1, 2)).view(hkv * g, n, ctx)
        if n > 1:
            p.masked_fill_(~_visible(st["masks"][row:row + n], n, ctx), -math.inf)
        p.sub_(p.amax(-1, keepdim=True)).exp_()
        total = p.sum(-1, keepdim=True)
        o = torch.matmul(p.view(hkv, g * n, ctx), v).view(hkv * g, n, d).div_(total)
        out[row:row + n] = o.transpose(0, 1).to(q.dtype)
        row += n
    return out


# ---- the same in 64 bits ---------------------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    return {"store": _exact_store, "read": _exact_read, "attend": _exact_attend}[case["op"]](case, st)


def _nearest_fp16(x, toward):
    """The fp16 number nearest to x on the side that ``toward`` names (-1: not above, 1: not below),
    by its steps: 2^(e - 10) from 2^e on, never below 2^-24."""
    step = torch.exp2((torch.frexp(x)[1].double() - 11).clamp(min=-24))
    return torch.ceil(x / step) * step if toward > 0 else torch.floor(x / step) * step


def _stands_for(x):
    """What the INT4 cache stands for after it has taken x: of a group's sixteen values the nearest."""
    x = x.double().reshape(*x.shape[:-1], -1, GROUP)
    z = _nearest_fp16(x.min(-1, keepdim=True)[0], -1)
    s = _nearest_fp16((x.max(-1, keepdim=True)[0] - z) / 15, 1)
    best = z + torch.zeros_like(x)
    for c in (2, 4, 6, 8, 10, 12, 14, 1, 3, 5, 7, 9, 11, 13, 15):   # halfway between two, the even code stays
        y = z + c * s
        best = torch.where((x - y).abs() < (x - best).abs(), y, best)
    return best.flatten(-2)


def _exact_store(case, st):
    return {"key": _stands_for(st["key"]), "value": _stands_for(st["value"])}


def _dense(case, st, which, slots):
    """Rows of K or V by slot, [slot][head][dimension] in 64 bits, a dimension at a time."""
    cache = (st["k_cache"], st["v_cache"])[which]
    b, t, d = slots // BLOCK, slots % BLOCK, case["d"]
    rows = cache[b, :, t]
    out = torch.empty((*rows.shape[:2], d), device=rows.device, dtype=torch.float64)
    if case.get("kv", "int4") == "int8":
        sc = st["scales"][b, :, which, t].double()
        for i in range(d):
            out[..., i] = (rows[..., i].to(torch.int64) % 256 - 128) * sc
        return out
    rows = rows.to(torch.int64)
    sc = st["scales"][b, :, which, t].double()
    for i in range(d):
        g, unit, e = i // GROUP, i % GROUP // 8, i % 8
        nibble = e // 2 + 4 * (e % 2)            # of the 32-bit word, lowest first
        at = 4 * (unit * (d // GROUP) + g) + nibble // 2
        out[..., i] = sc[..., g, 1] + sc[..., g, 0] * ((rows[..., at] // 16 ** (nibble % 2)) % 16)
    return out


def _exact_read(case, st):
    slots = st["slots"].long()
    return {"key": _dense(case, st, 0, slots), "value": _dense(case, st, 1, slots)}


def _exact_attend(case, st):
    g, out, row = case["hq"] // case["hkv"], [], 0
    for s, ((n, ctx), seen) in enumerate(zip(st["lens"], _masks(case))):
        p = torch.arange(ctx, device=DEVICE)
        slots = st["tables"][s].long()[p // BLOCK] * BLOCK + p % BLOCK
        k, v = (_dense(case, st, w, slots).transpose(0, 1) for w in range(2))
        blind = torch.zeros((n, ctx), device=DEVICE, dtype=torch.bool)
        blind[:, ctx - n:] = torch.tensor([[not m >> i & 1 for i in range(n)] for m in seen], device=DEVICE)
        x = st["q"][row:row + n].double().permute(1, 0, 2).reshape(case["hkv"], g, n, case["d"])
        a = torch.einsum("hgnd,hcd->hgnc", x, k) * st["scale"]
        a = a.masked_fill(blind, -math.inf)
        o = torch.einsum("hgnc,hcd->hgnd", torch.exp(a - torch.logsumexp(a, -1, keepdim=True)), v)
        out.append(o.reshape(case["hq"], n, case["d"]).transpose(0, 1))
        row += n
    return torch.cat(out)
