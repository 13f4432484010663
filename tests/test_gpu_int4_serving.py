"""A server's steps over an INT4 cache: prompts, decode, a verified tree, acceptance, fork with copy-on-write, a prefix
read back; every step against the 64-bit form over what the cache holds."""
import pytest
import torch

import paged_kv_cache_252_gb300 as pkv
import _int4 as i4

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("dtype,d", [(torch.float16, 128), (torch.bfloat16, 64)])
def test_steps(dtype, d):
    hq, hkv, blocks = 8, 2, 64
    g = torch.Generator(device=DEV)
    g.manual_seed(d)
    kc, vc = pkv.alloc_kv_cache(blocks, hkv, d, "int4", DEV)
    sc = pkv.alloc_kv_scales(blocks, hkv, DEV, kv_dtype="int4", head_size=d)
    pool = pkv.BlockAllocator(blocks)
    inv, factor = pkv.rotary_inv_freq(d, device=DEV)
    scale = d ** -0.5
    lens = {}

    def write(seq, n):
        """n new tokens of seq: turned keys, values, and the queries for them."""
        slots, copies = pool.append(seq, n)
        if copies:
            src, dst = (torch.tensor(x, device=DEV, dtype=torch.int32) for x in zip(*copies))
            pkv.copy_blocks(kc, vc, src, dst, "int4", scales=sc)
        pos = torch.arange(lens[seq], lens[seq] + n, device=DEV)
        q, k, v = (torch.randn((n, h, d), generator=g, device=DEV).to(dtype) for h in (hq, hkv, hkv))
        pkv.rotary_embed(q, q, pos, inv, attn_factor=factor)
        pkv.rotary_embed(k, k, pos, inv, attn_factor=factor)
        pkv.kv_cache_write_int4(k, v, torch.tensor(slots, device=DEV, dtype=torch.int32), kc, vc, sc)
        lens[seq] += n
        return q

    def tables(seqs):
        rows = [pool.block_table(s) for s in seqs]
        width = max(len(r) for r in rows)
        return torch.tensor([r + [-1] * (width - len(r)) for r in rows], device=DEV, dtype=torch.int32)

    def check(out, q, seqs, cu, masks=None):
        ctx = [lens[s] for s in seqs]
        i4.assert_within(out, *i4.attention(q, kc, vc, sc, tables(seqs), ctx, cu, scale, masks))

    # prompts of two sequences in one call
    for s in (0, 1):
        pool.add(s)
        lens[s] = 0
    q = torch.cat((write(0, 45), write(1, 7)))
    out = torch.empty_like(q)
    pkv.paged_attention_decode_chunked(out, q, [45, 7], [45, 7], kc, vc, tables((0, 1)), scale, "int4", scales=sc)
    check(out, q, (0, 1), [0, 45, 52])
    # a fork writes into a shared, partly filled block: copied first
    pool.fork(0, 2)
    lens[2] = lens[0]
    before = pool.block_table(0)
    q = torch.cat([write(s, 1) for s in (0, 1, 2)])
    assert pool.block_table(0)[-1] != pool.block_table(2)[-1] and pool.block_table(2)[:2] == before[:2]
    out = torch.empty_like(q)
    ctx = torch.tensor([lens[s] for s in (0, 1, 2)], device=DEV, dtype=torch.int32)
    pkv.paged_attention_decode_int4(out, q, kc, vc, sc, tables((0, 1, 2)), ctx, 1, scale)
    check(out, q, (0, 1, 2), [0, 1, 2, 3])
    # a tree of five drafts; the path 0, 2, 4 is accepted
    q = torch.cat([write(s, 5) for s in (0, 1)])
    masks = torch.tensor([1, 3, 5, 8 | 3, 16 | 5] * 2, device=DEV, dtype=torch.int64)
    ctx = torch.tensor([lens[s] for s in (0, 1)], device=DEV, dtype=torch.int32)
    out = torch.empty_like(q)
    pkv.paged_attention_decode_tree(out, q, masks, kc, vc, tables((0, 1)), ctx, 5, scale, "int4", scales=sc)
    check(out, q, (0, 1), [0, 5, 10], masks)

    def rows(seq, a, b):
        at = torch.arange(a, b, device=DEV)
        slots = (torch.tensor(pool.block_table(seq), device=DEV)[at // 16] * 16 + at % 16).to(torch.int32)
        k, v = (torch.empty((b - a, hkv, d), dtype=dtype, device=DEV) for _ in range(2))
        pkv.kv_cache_read(k, v, slots, kc, vc, "int4", scales=sc)
        return k, v

    base = lens[0] - 5
    drafts = rows(0, base, base + 5)
    new = torch.empty_like(ctx)
    acc = torch.tensor([[0, 2, 4]] * 2, device=DEV, dtype=torch.int32)
    pkv.kv_cache_accept(kc, vc, tables((0, 1)), ctx, acc, torch.full_like(ctx, 3), new, 5, "int4", scales=sc)
    for k, s in enumerate((0, 1)):
        lens[s] -= 2
        assert int(new[k]) == lens[s]
        pool.truncate(s, lens[s])
    kept = rows(0, base, base + 3)
    assert all(torch.equal(x, y[[0, 2, 4]]) for x, y in zip(kept, drafts))
    # and on: different numbers of tokens
    q = torch.cat((write(0, 1), write(1, 4), write(2, 2)))
    cu = torch.tensor([0, 1, 5, 7], device=DEV, dtype=torch.int32)
    ctx = torch.tensor([lens[s] for s in (0, 1, 2)], device=DEV, dtype=torch.int32)
    out = torch.empty_like(q)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    pkv.paged_attention_decode_varlen(out, q, cu, kc, vc, tables((0, 1, 2)), ctx, 4, scale, "int4", scales=sc, device_status=st)
    check(out, q, (0, 1, 2), [0, 1, 5, 7])
    assert int(st) == 0


@pytest.mark.parametrize("d", [64, 128])
def test_the_call_with_a_buffer_of_its_own_takes_what_it_took(d):
    """pkv_decode_workspace_bytes covers an INT4 cache, whose units of 16 rows need more than the others'; the call that takes no
    workspace keeps its limit. (Misaligned pointers: no call gets as far as a launch.)"""
    import ctypes
    from paged_kv_cache_252_gb300.api import _CacheDesc, load_library
    lib, desc, fake = load_library(), _CacheDesc(1024, 16, 8, d), ctypes.c_void_p(257)

    def status(S):
        return lib.pkv_paged_attention_decode_noalloc(fake, fake, S, 64, 2, fake, fake, 0, ctypes.byref(desc), fake, 4, fake,
                                                      ctypes.c_float(0.1), None, None)
    S = next(S for S in range(1, 5000) if lib.pkv_decode_workspace_bytes(S, 64, 2, ctypes.byref(desc)) > 32 << 20)
    assert status(S) == -1 and status(2 * S) == -3
