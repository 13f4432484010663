"""The operators one after another as a server runs them: prompts in chunks (rotary write, then
prefill), a token tree verified, its accepted path kept, the sequences cut back, a decode step."""
import numpy as np
import pytest
import torch

import _gpu
import _operators as op

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    return torch.device("cuda:0")


class Server:
    """Sequences with their raw q, key and value per token, and the cache they are written to."""

    def __init__(self, dev, kv, D, hq, hkv, seqs, seed, interleaved):
        import paged_kv_cache_252_gb300 as pkv
        self.pkv, self.dev, self.hq, self.hkv, self.D = pkv, dev, hq, hkv, D
        self.g = torch.Generator(device=dev)
        self.g.manual_seed(seed)
        self.pool = pkv.BlockAllocator(96)
        self.kc, self.vc, self.sc = op.make_cache(kv, 96, hkv, D, self.g, dev)
        self.k0, self.v0, self.s0 = (None if t is None else t.clone() for t in (self.kc, self.vc, self.sc))
        self.inv, self.f = pkv.rotary_inv_freq(D, 10000.0, device=dev)
        self.inter, self.dt, self.scale = interleaved, op.src_dtype(kv), D ** -0.5
        self.seqs = list(range(seqs))
        for s in self.seqs:
            self.pool.add(s)
        self.kept = [[] for _ in self.seqs]          # raw (key, value) rows of the kept tokens
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)

    def i32(self, x):
        return torch.tensor(x, dtype=torch.int32, device=self.dev)

    def raw(self, n):
        return torch.randn((n, (self.hq + 2 * self.hkv) * self.D), generator=self.g, device=self.dev).to(self.dt)

    def split(self, qkv):
        a, b = self.hq * self.D, (self.hq + self.hkv) * self.D
        return (qkv[:, :a].view(-1, self.hq, self.D), qkv[:, a:b].view(-1, self.hkv, self.D),
                qkv[:, b:].view(-1, self.hkv, self.D))

    def tables(self):
        rows = [self.pool.block_table(s) for s in self.seqs]
        return self.i32([r + [0] * (max(map(len, rows)) - len(r)) for r in rows])

    def write(self, qkv, positions, slots, cache=None):
        kc, vc, sc = cache or (self.kc, self.vc, self.sc)
        q, k, v = self.split(qkv)
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
        self.pkv.rotary_write(out, q, k, v, torch.tensor(positions, device=self.dev), self.i32(slots), kc, vc, self.inv,
                              interleaved=self.inter, attn_factor=self.f, scales=sc, device_status=self.status)
        return out

    def prefill(self, q, ns, what):
        cu = [0] + np.cumsum(ns).tolist()
        lens = [self.pool.length(s) for s in self.seqs]
        bt, out = self.tables(), torch.empty_like(q)
        self.pkv.paged_attention_prefill(out, q, self.i32(cu), self.kc, self.vc, bt, self.i32(lens), self.scale,
                                         scales=self.sc, device_status=self.status)
        want, tol = op.attention_bound(q, self.kc, self.vc, self.sc, bt, cu, lens, self.scale)
        op.assert_within(out, want, tol, what)
        return want, tol


@pytest.mark.parametrize("kv,D,hq,hkv,interleaved", [("fp16", 128, 8, 2, False), ("bf16", 64, 6, 2, True),
                                                     ("e5m2", 128, 14, 2, False), ("e5m2", 64, 4, 4, True),
                                                     ("int8", 128, 7, 1, False), ("int8", 64, 8, 2, True)])
def test_prompts_verify_accept_decode(dev, kv, D, hq, hkv, interleaved):
    rng = np.random.default_rng(D + hq)
    prompts, chunk, drafts = [100, 17, 260], 64, 9
    sv = Server(dev, kv, D, hq, hkv, len(prompts), 5, interleaved)
    pkv = sv.pkv
    # prompts, at most `chunk` tokens of each a step; finished ones sit the step out with no rows
    while True:
        ns = [min(chunk, p - len(sv.kept[s])) for s, p in enumerate(prompts)]
        if not sum(ns):
            break
        slots, pos = [], []
        qkv = sv.raw(sum(ns))
        at = 0
        for s, n in enumerate(ns):
            pos += range(len(sv.kept[s]), len(sv.kept[s]) + n)
            slots += sv.pool.append(s, n)[0]
            sv.kept[s] += list(qkv[at:at + n])
            at += n
        sv.prefill(sv.write(qkv, pos, slots), ns, f"chunk {ns}")
    for step in range(3):
        # a tree of drafts behind every sequence: draft i hangs from an earlier one or the context
        base = [len(k) for k in sv.kept]
        parent = [[int(rng.integers(-1, i)) for i in range(drafts)] for _ in prompts]
        paths = []
        for p in parent:
            w = []
            for i in range(drafts):
                w.append((w[p[i]] if p[i] >= 0 else []) + [i])
            paths.append(w)
        masks = torch.tensor([sum(1 << j for j in w) for t in paths for w in t], dtype=torch.int64, device=dev)
        qkv = sv.raw(drafts * len(prompts))
        slots = [x for s in sv.seqs for x in sv.pool.append(s, drafts)[0]]
        q = sv.write(qkv, [b + len(w) - 1 for b, t in zip(base, paths) for w in t], slots)
        lens = [sv.pool.length(s) for s in sv.seqs]
        verified = torch.empty_like(q)
        bt = sv.tables()
        pkv.paged_attention_decode_tree(verified, q, masks, sv.kc, sv.vc, bt, sv.i32(lens), drafts, sv.scale,
                                        scales=sv.sc, device_status=sv.status)
        # keep one draft's path, a part of it, nothing
        chosen = []
        for s, t in enumerate(paths):
            w = max(t, key=len)
            chosen.append(w[:(len(w), 1, 0)[(s + step) % 3]])
        acc = sv.i32([w + [0] * (drafts - len(w)) for w in chosen])
        num = sv.i32([len(w) for w in chosen])
        new = torch.empty_like(num)
        pkv.kv_cache_accept(sv.kc, sv.vc, bt, sv.i32(lens), acc, num, new, drafts, scales=sv.sc,
                            device_status=sv.status)
        rows, ns = [], []
        for s, w in enumerate(chosen):
            sv.pool.truncate(s, base[s] + len(w))
            sv.kept[s] += [qkv[s * drafts + i] for i in w]
            rows += [s * drafts + i for i in w]
            ns.append(len(w))
        assert new.tolist() == [sv.pool.length(s) for s in sv.seqs] == [len(k) for k in sv.kept]
        # the accepted rows' attention over the cut cache is what the verify gave for them (within
        # the gate that holds for the decode calls)
        want, _ = sv.prefill(q[rows].contiguous(), ns, f"accepted {chosen}")
        _gpu.compare(verified[rows], want.cpu().numpy(), label=f"verify {kv} step {step}")
        # the cache holds what writing the kept tokens one after another would have left
        straight = tuple(None if t is None else t.clone() for t in (sv.k0, sv.v0, sv.s0))
        bt_host = [sv.pool.block_table(s) for s in sv.seqs]
        where = [[bt_host[s][p // 16] * 16 + p % 16 for p in range(len(sv.kept[s]))] for s in sv.seqs]
        flat = sum(where, [])
        sv.write(torch.stack([r for k in sv.kept for r in k]), [p for k in sv.kept for p in range(len(k))], flat, straight)
        at = torch.tensor(flat, device=dev)
        for got, exp in ((sv.kc, straight[0]), (sv.vc, straight[1])):
            got, exp = (c.transpose(1, 2).reshape(-1, hkv, D)[at] for c in (got, exp))
            assert torch.equal(got.view(torch.uint8), exp.view(torch.uint8))
        if sv.sc is not None:
            got, exp = (c.permute(0, 3, 1, 2).reshape(-1, hkv, 2)[at] for c in (sv.sc, straight[2]))
            assert torch.equal(got, exp)
        # a plain step of one token a sequence
        one = sv.raw(len(prompts))
        q1 = sv.write(one, [len(k) for k in sv.kept], [x for s in sv.seqs for x in sv.pool.append(s, 1)[0]])
        for s in sv.seqs:
            sv.kept[s].append(one[s])
        want, _ = sv.prefill(q1, [1] * len(prompts), "one token each")
        lens = sv.i32([sv.pool.length(s) for s in sv.seqs])
        out = torch.empty_like(q1)
        if kv == "int8":
            pkv.paged_attention_decode_int8(out, q1, sv.kc, sv.vc, sv.sc, sv.tables(), lens, 1, sv.scale)
        else:
            pkv.paged_attention_decode(out, q1, sv.kc, sv.vc, sv.tables(), lens, 1, sv.scale)
        _gpu.compare(out, want.cpu().numpy(), label=f"decode {kv} step {step}")
    assert sv.status.item() == 0
