"""What is measured of the operators beside paged decode attention: the rotary
embedding with its cache write, attention of a chunk of new tokens over the paged
cache, and the acceptance of verified draft tokens.

Each case names one operator ("op"):

* ``rotary``: one layer's packed QKV rows -> rotated queries, and the rotated keys and
  the values written to their slots of the paged cache (fp16, bf16 or E5M2).
* ``prefill``: causal attention of every sequence's newest tokens (whole prompts,
  chunks of a prompt, single decode rows beside them) over its blocks.
* ``accept``: the cache side of a verify step: the draft tokens' rows are written, then
  the accepted ones are moved together behind the context and the new lengths returned.

``run`` computes an operator in plain torch operations where ``own`` is false and
through the package where it is true; ``exact`` computes it in 64 bits.
"""
import math
import random

import torch

own = False

DEVICE = "cuda"
BLOCK = 16
DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "e5m2": torch.uint8, "int8": torch.int8}


# ---- cases ---------------------------------------------------------------------------

def listed():
    heads8b = {"hq": 32, "hkv": 8, "d": 128}
    heads70b = {"hq": 64, "hkv": 8, "d": 128}
    return [
        # one decode step of 64 sequences: one row each, where latency counts
        {"name": "rotary-decode-fp16", "op": "rotary", "kv": "fp16", **heads8b, "tokens": 64, "rot": 128,
         "interleaved": False, "base": 500000.0, "factor": 1.0, "first": 511},
        # a whole prompt, its positions stretched by 8 for a long context
        {"name": "rotary-prompt-bf16", "op": "rotary", "kv": "bf16", **heads8b, "tokens": 8192, "rot": 128,
         "interleaved": False, "base": 500000.0, "factor": 8.0, "first": 0},
        # 128 sequences x 4 draft tokens over the E5M2 cache, neighbouring pairs
        {"name": "rotary-verify-e5m2", "op": "rotary", "kv": "e5m2", **heads70b, "tokens": 512, "rot": 128,
         "interleaved": True, "base": 10000.0, "factor": 1.0, "first": 16384},
        # head size 64 with half of the head rotated, an odd number of rows far into a context
        {"name": "rotary-partial-fp16", "op": "rotary", "kv": "fp16", "hq": 16, "hkv": 4, "d": 64, "tokens": 2001,
         "rot": 32, "interleaved": False, "base": 10000.0, "factor": 1.0, "first": 131072},
        # four short prompts of a small model: the smallest call
        {"name": "prefill-tiny-fp16", "op": "prefill", "kv": "fp16", "hq": 4, "hkv": 2, "d": 64, "seqs": 4,
         "n_lo": 1, "n_hi": 64, "past_lo": 0, "past_hi": 0, "decodes": 0, "shape": 1},
        # one whole prompt: the largest call
        {"name": "prefill-prompt-bf16", "op": "prefill", "kv": "bf16", **heads8b, "seqs": 1,
         "n_lo": 8192, "n_hi": 8192, "past_lo": 0, "past_hi": 0, "decodes": 0, "shape": 2},
        # a chunk of a prompt beside the decode rows of 31 running sequences
        {"name": "prefill-mixed-fp16", "op": "prefill", "kv": "fp16", **heads8b, "seqs": 1,
         "n_lo": 2048, "n_hi": 2048, "past_lo": 2048, "past_hi": 2048, "decodes": 31, "shape": 3},
        # chunks of eight sequences of ragged lengths over the E5M2 cache
        {"name": "prefill-ragged-e5m2", "op": "prefill", "kv": "e5m2", **heads70b, "seqs": 8,
         "n_lo": 33, "n_hi": 700, "past_lo": 100, "past_hi": 8192, "decodes": 0, "shape": 4},
        # four chunks over the INT8 cache
        {"name": "prefill-chunks-int8", "op": "prefill", "kv": "int8", **heads8b, "seqs": 4,
         "n_lo": 500, "n_hi": 1024, "past_lo": 1024, "past_hi": 4096, "decodes": 0, "shape": 5},
        # few rows over a long context: the last chunk of a long document
        {"name": "prefill-long-bf16", "op": "prefill", "kv": "bf16", **heads8b, "seqs": 1,
         "n_lo": 100, "n_hi": 100, "past_lo": 130972, "past_hi": 130972, "decodes": 0, "shape": 6},
        # 128 sequences x 4 drafts over the E5M2 cache
        {"name": "accept-verify4-e5m2", "op": "accept", "kv": "e5m2", "hkv": 8, "d": 128, "seqs": 128, "drafts": 4,
         "past_lo": 16, "past_hi": 2048, "shape": 7},
        # token trees of 64 drafts
        {"name": "accept-tree64-fp16", "op": "accept", "kv": "fp16", "hkv": 8, "d": 128, "seqs": 64, "drafts": 64,
         "past_lo": 512, "past_hi": 2048, "shape": 8},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotary", "prefill", "prefill", "accept"])
    d = rng.choice([64, 128])
    if op == "rotary":
        kv = rng.choice(["fp16", "bf16", "e5m2"])
        hkv = rng.choice([1, 2, 4, 8])
        return {"op": op, "kv": kv, "hq": hkv * rng.choice([1, 2, 3, 4, 8]), "hkv": hkv, "d": d,
                "tokens": _log_int(rng, 1, 8192), "rot": 16 * rng.randint(1, d // 16),
                "interleaved": rng.random() < 0.5, "base": rng.choice([10000.0, 500000.0]),
                "factor": rng.choice([1.0, 4.0, 16.0]), "first": _log_int(rng, 1, 131072) - 1}
    if op == "accept":
        return {"op": op, "kv": rng.choice(["fp16", "bf16", "e5m2"]), "hkv": rng.choice([1, 2, 4, 8]), "d": d,
                "seqs": _log_int(rng, 1, 128), "drafts": rng.randint(1, 64), "past_lo": rng.randint(0, 64),
                "past_hi": rng.randint(64, 2048), "shape": rng.randrange(1 << 30)}
    hkv = rng.choice([1, 2, 4, 8])
    case = {"op": op, "kv": rng.choice(["fp16", "bf16", "e5m2", "int8"]),
            "hq": hkv * rng.choice([1, 2, 3, 4, 6, 8]), "hkv": hkv, "d": d, "seqs": _log_int(rng, 1, 16)}
    hi = _log_int(rng, 1, 8192)
    case.update(n_lo=max(1, hi // rng.randint(1, 4)), n_hi=hi)
    past = _log_int(rng, 1, 131072) - 1
    case.update(past_lo=past // rng.randint(1, 4), past_hi=past, decodes=rng.choice([0, 0, 7, 30]),
                shape=rng.randrange(1 << 30))
    top = work(listed()[5])["flops"]
    while work(case)["flops"] > top or case["n_hi"] * (case["n_hi"] + case["past_hi"]) * case["hq"] > 1 << 31:
        for k in ("n_lo", "n_hi", "past_lo", "past_hi"):
            case[k] = max(1 if k[0] == "n" else 0, case[k] * 2 // 3)
    return case


def _lens(case):
    """The sequences' (new tokens, context length with them), the same for every seed."""
    r = random.Random(case["shape"])
    if case["op"] == "accept":
        return [(case["drafts"], r.randint(case["past_lo"], case["past_hi"]) + case["drafts"]) for _ in range(case["seqs"])]
    lens = []
    for _ in range(case["seqs"]):
        n = r.randint(case["n_lo"], case["n_hi"])
        lens.append((n, n + r.randint(case["past_lo"], case["past_hi"])))
    for _ in range(case["decodes"]):
        lens.append((1, r.randint(512, 2048)))
    r.shuffle(lens)
    return lens


def _esize(case):
    return 1 if case["kv"] in ("e5m2", "int8") else 2


def work(case):
    es = _esize(case)
    if case["op"] == "rotary":
        t, q, k = case["tokens"], case["hq"] * case["d"], case["hkv"] * case["d"]
        pairs = t * (case["hq"] + case["hkv"]) * case["rot"] / 2
        return {"bytes": t * (q * 4 + k * 4 + 2 * k * es + 12), "flops": 6 * pairs}
    if case["op"] == "accept":
        row = case["hkv"] * case["d"]
        drafts = case["seqs"] * case["drafts"]
        moved = sum(len(path) - sum(1 for i, j in enumerate(path) if i == j) for path in _accepted(case))
        return {"bytes": drafts * row * 2 * (2 + es) + moved * row * 2 * 2 * es + case["seqs"] * 12, "flops": 0}
    b = f = 0
    for n, ctx in _lens(case):
        b += n * case["hq"] * case["d"] * 4 + ctx * case["hkv"] * (2 * case["d"] * es + (8 if case["kv"] == "int8" else 0))
        f += 4 * case["d"] * case["hq"] * (n * (ctx - n) + n * (n + 1) // 2)
    return {"bytes": b, "flops": f}


def _accepted(case):
    """Each sequence's accepted drafts: one path from the root of its token tree."""
    r = random.Random(case["shape"] + 1)
    paths = []
    for _ in range(case["seqs"]):
        parent = [r.randint(-1, i - 1) if i else -1 for i in range(case["drafts"])]
        node, path = r.randrange(case["drafts"]), []
        while node >= 0:
            path.append(node)
            node = parent[node]
        paths.append(path[::-1])
    return paths


# ---- inputs --------------------------------------------------------------------------

def _randn(g, shape, dtype):
    return torch.randn(shape, generator=g, device=DEVICE, dtype=torch.float32).to(dtype)


def _cache(case, blocks, g):
    """A pool that earlier steps filled: keys and values of unit variance."""
    shape = (blocks, case["hkv"], BLOCK, case["d"])
    if case["kv"] == "int8":
        kv = [torch.randint(-127, 128, shape, generator=g, device=DEVICE, dtype=torch.int16).sub_(128).to(torch.int8) for _ in range(2)]
        scales = (torch.rand((blocks, case["hkv"], 2, BLOCK), generator=g, device=DEVICE) * 0.02 + 0.01).half().float()
        return kv[0], kv[1], scales
    if case["kv"] == "e5m2":
        return tuple(_randn(g, shape, torch.float16).to(torch.float8_e5m2).view(torch.uint8) for _ in range(2)) + (None,)
    return _randn(g, shape, DTYPES[case["kv"]]), _randn(g, shape, DTYPES[case["kv"]]), None


def _tables(lens, g):
    """Block tables over a shuffled pool with a quarter more blocks than are used."""
    need = [-(-ctx // BLOCK) for _, ctx in lens]
    total = max(1, sum(need) * 5 // 4)
    order = torch.randperm(total, generator=g, device=DEVICE).to(torch.int32)
    tables = torch.zeros((len(lens), max(1, max(need))), device=DEVICE, dtype=torch.int32)
    at = 0
    for s, n in enumerate(need):
        tables[s, :n] = order[at:at + n]
        at += n
    return tables, total


def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    st = {"case": case}
    src = torch.bfloat16 if case["kv"] == "bf16" else torch.float16
    d, hkv = case["d"], case["hkv"]
    if case["op"] == "rotary":
        t, hq = case["tokens"], case["hq"]
        blocks = -(-t // BLOCK)
        st["k_cache"], st["v_cache"], _ = _cache(case, blocks, g)
        # what a fused projection leaves: one row of query, key and value heads per token
        qkv = _randn(g, (t, (hq + 2 * hkv) * d), src)
        st["q"] = qkv[:, :hq * d].view(t, hq, d)
        st["key"] = qkv[:, hq * d:(hq + hkv) * d].view(t, hkv, d)
        st["value"] = qkv[:, (hq + hkv) * d:].view(t, hkv, d)
        st["positions"] = torch.arange(case["first"], case["first"] + t, device=DEVICE)
        st["slots"] = torch.randperm(blocks * BLOCK, generator=g, device=DEVICE)[:t].to(torch.int32)
        i = torch.arange(case["rot"] // 2, device=DEVICE, dtype=torch.float64)
        st["inv_freq"] = case["base"] ** (-2.0 * i / case["rot"]) / case["factor"]
        st["attn_factor"] = 1.0 if case["factor"] == 1.0 else 0.1 * math.log(case["factor"]) + 1.0
        return st
    lens = _lens(case)
    st["lens"] = lens
    st["tables"], blocks = _tables(lens, g)
    st["k_cache"], st["v_cache"], st["scales"] = _cache(case, blocks, g)
    st["context_lens"] = torch.tensor([ctx for _, ctx in lens], device=DEVICE, dtype=torch.int32)
    cu = [0]
    for n, _ in lens:
        cu.append(cu[-1] + n)
    st["cu"] = torch.tensor(cu, device=DEVICE, dtype=torch.int32)
    if case["op"] == "prefill":
        st["q"] = _randn(g, (cu[-1], case["hq"], d), src)
        st["scale"] = 1.0 / math.sqrt(d)
        return st
    n = case["drafts"]
    st["key"], st["value"] = _randn(g, (cu[-1], hkv, d), src), _randn(g, (cu[-1], hkv, d), src)
    pos = (st["context_lens"].long() - n)[:, None] + torch.arange(n, device=DEVICE)
    st["slots"] = (st["tables"].gather(1, pos // BLOCK) * BLOCK + pos % BLOCK).to(torch.int32).reshape(-1)
    paths = _accepted(case)
    width = max(len(p) for p in paths)
    st["accepted"] = torch.tensor([p + [0] * (width - len(p)) for p in paths], device=DEVICE, dtype=torch.int32)
    st["num_accepted"] = torch.tensor([len(p) for p in paths], device=DEVICE, dtype=torch.int32)
    return st


# ---- one pass ------------------------------------------------------------------------

def run(st):
    return {"rotary": _rotary, "prefill": _prefill, "accept": _accept}[st["case"]["op"]](st)


def _values(cache):
    """The cache as the numbers it stands for (an E5M2 cache is kept as bytes)."""
    return cache.view(torch.float8_e5m2) if cache.dtype == torch.uint8 else cache


def _rotate(x, cos, sin, rot, interleaved):
    x = x.float()
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
    return torch.cat((turned, x[..., rot:]), -1)


def _rotary(st):
    case, q, key, value = st["case"], st["q"], st["key"], st["value"]
    k_cache, v_cache = st["k_cache"], st["v_cache"]
    if own:
        import paged_kv_cache_252_gb300 as pkv
        q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        pkv.rotary_write(q_out, q, key, value, st["positions"], st["slots"], k_cache, v_cache, st["inv_freq"],
                         interleaved=case["interleaved"], attn_factor=st["attn_factor"])
        return {"q": q_out, "k": _values(k_cache), "v": _values(v_cache)}
    angle = st["positions"].double()[:, None] * st["inv_freq"]
    cos = (angle.cos() * st["attn_factor"]).float()[:, None]
    sin = (angle.sin() * st["attn_factor"]).float()[:, None]
    rot, inter = case["rot"], case["interleaved"]
    blk, off = st["slots"].long() // BLOCK, st["slots"].long() % BLOCK
    kv = torch.float8_e5m2 if case["kv"] == "e5m2" else k_cache.dtype
    k_cache[blk, :, off] = _rotate(key, cos, sin, rot, inter).to(kv).view(k_cache.dtype)
    v_cache[blk, :, off] = value.to(kv).view(v_cache.dtype)
    return {"q": _rotate(q, cos, sin, rot, inter).to(q.dtype), "k": _values(k_cache), "v": _values(v_cache)}


def _gathered(st, cache, which, s, ctx):
    """A sequence's rows of one cache in 32 bits, [kv head][position][dimension]."""
    ids = st["tables"][s, :-(-ctx // BLOCK)].long()
    if cache.dtype == torch.int8:
        x = cache[ids].view(torch.uint8).float().sub_(128).mul_(st["scales"][ids, :, which, :, None])
    else:
        x = _values(cache)[ids].float()
    return x.transpose(0, 1).flatten(1, 2)[:, :ctx]


def _prefill(st):
    q, case = st["q"], st["case"]
    if own:
        import paged_kv_cache_252_gb300 as pkv
        out = torch.empty_like(q)
        return pkv.paged_attention_prefill(out, q, st["cu"], st["k_cache"], st["v_cache"], st["tables"],
                                           st["context_lens"], st["scale"], scales=st["scales"])
    hkv, d = case["hkv"], case["d"]
    g = case["hq"] // hkv
    out, row = torch.empty_like(q), 0
    # Sequences one by one: padding a ragged batch to its longest would cost far more.
    for s, (n, ctx) in enumerate(st["lens"]):
        k, v = (_gathered(st, c, w, s, ctx) for w, c in enumerate((st["k_cache"], st["v_cache"])))
        x = q[row:row + n].float().mul_(st["scale"]).view(n, hkv, g, d).permute(1, 2, 0, 3).reshape(hkv, g * n, d)
        p = torch.matmul(x, k.transpose(1, 2)).view(hkv * g, n, ctx)
        if n > 1:
            seen = torch.arange(ctx, device=q.device) <= torch.arange(ctx - n, ctx, device=q.device)[:, None]
            p.masked_fill_(~seen, -math.inf)
        p.sub_(p.amax(-1, keepdim=True)).exp_()
        total = p.sum(-1, keepdim=True)
        o = torch.matmul(p.view(hkv, g * n, ctx), v).view(hkv * g, n, d).div_(total)
        out[row:row + n] = o.transpose(0, 1).to(q.dtype)
        row += n
    return out


def _accept(st):
    case, key, value = st["case"], st["key"], st["value"]
    k_cache, v_cache, n = st["k_cache"], st["v_cache"], case["drafts"]
    if own:
        import paged_kv_cache_252_gb300 as pkv
        pkv.kv_cache_write(key, value, st["slots"], k_cache, v_cache)
        lens = torch.empty_like(st["context_lens"])
        pkv.kv_cache_accept(k_cache, v_cache, st["tables"], st["context_lens"], st["accepted"], st["num_accepted"],
                            lens, n)
        return {"k": _values(k_cache), "v": _values(v_cache), "lens": lens}
    base = (st["context_lens"] - n).long()
    i = torch.arange(st["accepted"].shape[1], device=base.device)
    valid = (i < st["num_accepted"][:, None])[..., None, None]

    def place(pos):
        return st["tables"].gather(1, pos // BLOCK).long(), pos % BLOCK

    (sb, so), (db, do) = place(base[:, None] + st["accepted"]), place(base[:, None] + i)
    blk, off = st["slots"].long() // BLOCK, st["slots"].long() % BLOCK
    kv = torch.float8_e5m2 if case["kv"] == "e5m2" else k_cache.dtype
    k_cache[blk, :, off] = key.to(kv).view(k_cache.dtype)
    v_cache[blk, :, off] = value.to(kv).view(v_cache.dtype)
    k_cache[db, :, do] = torch.where(valid, k_cache[sb, :, so], k_cache[db, :, do])
    v_cache[db, :, do] = torch.where(valid, v_cache[sb, :, so], v_cache[db, :, do])
    return {"k": _values(k_cache), "v": _values(v_cache), "lens": st["context_lens"] - n + st["num_accepted"]}


# ---- the same in 64 bits ---------------------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    return {"rotary": _exact_rotary, "prefill": _exact_prefill, "accept": _exact_accept}[case["op"]](case, st)


def _slot_rows(cache):
    """The cache as [slot][head][dimension], a copy in 64 bits."""
    return _values(cache).double().permute(0, 2, 1, 3).reshape(-1, cache.shape[1], cache.shape[3])


def _as_cache(rows, cache):
    return rows.view(cache.shape[0], BLOCK, cache.shape[1], cache.shape[3]).permute(0, 2, 1, 3).contiguous()


def _stored(x, cache):
    """x as the cache defines it: an E5M2 cache holds the nearest of its values (two fraction
    bits, ties to even, steps of 2^-16 below 2^-14, at most 57344); others hold x, rounded as any output."""
    x = x.double()
    if cache.dtype != torch.uint8:
        return x
    step = torch.exp2(torch.frexp(x)[1].double().sub(3).clamp(min=-16))
    return (x / step).round().mul(step).clamp(-57344, 57344)


def _exact_rotary(case, st):
    # each pair as a complex number, turned by e^(i * position * frequency)
    half = case["rot"] // 2
    turn = torch.polar(torch.full((case["tokens"], half), st["attn_factor"], device=DEVICE, dtype=torch.float64),
                       torch.outer(st["positions"].double(), st["inv_freq"]))
    j = torch.arange(half, device=DEVICE)
    re, im = (2 * j, 2 * j + 1) if case["interleaved"] else (j, j + half)

    def turned(x):
        y = x.double().clone()
        z = torch.complex(y[..., re], y[..., im]) * turn.unsqueeze(1)
        y[..., re], y[..., im] = z.real, z.imag
        return y

    k, v = _slot_rows(st["k_cache"]), _slot_rows(st["v_cache"])
    at = st["slots"].long()
    k[at], v[at] = _stored(turned(st["key"]), st["k_cache"]), _stored(st["value"], st["v_cache"])
    return {"q": turned(st["q"]), "k": _as_cache(k, st["k_cache"]), "v": _as_cache(v, st["v_cache"])}


def _exact_prefill(case, st):
    k, v = st["k_cache"], st["v_cache"]
    if case["kv"] == "int8":
        sc = st["scales"].double().unsqueeze(-1)
        k, v = ((c.to(torch.int64) % 256 - 128).double() * sc[:, :, w] for w, c in enumerate((k, v)))
        k, v = (c.permute(0, 2, 1, 3).reshape(-1, case["hkv"], case["d"]) for c in (k, v))
    else:
        k, v = _slot_rows(k), _slot_rows(v)
    g, out, row = case["hq"] // case["hkv"], [], 0
    for s, (n, ctx) in enumerate(st["lens"]):
        p = torch.arange(ctx, device=DEVICE)
        slots = st["tables"][s].long()[p // BLOCK] * BLOCK + p % BLOCK
        o = torch.empty((n, case["hq"], case["d"]), device=DEVICE, dtype=torch.float64)
        for h in range(case["hq"]):
            kh, vh = k[slots, h // g], v[slots, h // g]
            x = st["q"][row:row + n, h].double() @ kh.T * st["scale"]
            x = x.masked_fill(p > torch.arange(ctx - n, ctx, device=DEVICE)[:, None], -math.inf)
            o[:, h] = torch.exp(x - torch.logsumexp(x, 1, keepdim=True)) @ vh
        out.append(o)
        row += n
    return torch.cat(out)


def _exact_accept(case, st):
    k, v = _slot_rows(st["k_cache"]), _slot_rows(st["v_cache"])
    n, tables, lens = case["drafts"], st["tables"].cpu(), []
    src, rows = [], []
    for s, (path, (_, ctx)) in enumerate(zip(_accepted(case), st["lens"])):
        kept = path + list(range(len(path), n))  # what is not overwritten stays the draft it was
        src += [s * n + j for j in kept]
        rows += [int(tables[s, p // BLOCK]) * BLOCK + p % BLOCK for p in range(ctx - n, ctx)]
        lens.append(ctx - n + len(path))
    src, rows = torch.tensor(src, device=DEVICE), torch.tensor(rows, device=DEVICE)
    k[rows], v[rows] = _stored(st["key"], st["k_cache"])[src], _stored(st["value"], st["v_cache"])[src]
    return {"k": _as_cache(k, st["k_cache"]), "v": _as_cache(v, st["v_cache"]),
            "lens": torch.tensor(lens, device=DEVICE, dtype=torch.int32)}
