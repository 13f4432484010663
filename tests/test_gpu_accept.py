"""Accepting verified drafts: rows moved within the cache, against plain indexing."""
import numpy as np
import pytest
import torch

import _operators as op

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    return torch.device("cuda:0")


def _rows(c, hkv):
    return c.transpose(1, 2).reshape(-1, hkv, c.shape[-1])


def _expect(cache, bt, lens, ns, acc, num, hkv):
    """The cache after acceptance, row by row (reads from the cache before)."""
    before = _rows(cache, hkv).clone()
    after = before.clone()
    for s, (ctx, n) in enumerate(zip(lens, ns)):
        slot = lambda p: int(bt[s, p // 16]) * 16 + p % 16
        for i in range(num[s]):
            after[slot(ctx - n + i)] = before[slot(ctx - n + acc[s][i])]
    return after


CASES = [
    # (kv, D, hkv, drafts of each sequence, past lengths)
    ("fp16", 128, 8, [4, 4, 4, 4], [0, 15, 16, 300]),
    ("bf16", 64, 3, [1, 9, 33, 64], [5, 12, 0, 77]),
    ("e5m2", 128, 2, [64, 64, 1], [8, 100, 15]),
    ("e5m2", 64, 1, [20, 0, 17], [3, 40, 31]),
    ("int8", 128, 4, [16, 64, 5], [1, 9, 16]),
    ("int8", 64, 2, [64, 2], [60, 15]),
]


@pytest.mark.parametrize("case", CASES, ids=[f"{c[0]}-D{c[1]}-{len(c[3])}" for c in CASES])
@pytest.mark.parametrize("how", ["path", "any", "all", "none"])
def test_accepted_rows_move_together(dev, case, how):
    import paged_kv_cache_252_gb300 as pkv
    kv, D, hkv, ns, past = case
    rng = np.random.default_rng(11)
    g = torch.Generator(device=dev)
    g.manual_seed(3)
    lens = [p + n for p, n in zip(past, ns)]
    bt, total = op.tables(lens, g, dev)
    kc, vc, sc = op.make_cache(kv, total, hkv, D, g, dev)
    acc, num = [], []
    for n in ns:
        m = {"path": rng.integers(0, n + 1), "any": n, "all": n, "none": 0}[how]
        if how == "any":      # any order, indices repeated
            a = rng.integers(0, max(n, 1), size=n)
        else:
            a = np.sort(rng.permutation(n)[:m])
        acc.append([int(x) for x in a[:m]])
        num.append(int(m))
    width = max(1, max(num)) + 1
    at = torch.tensor([a + [99] * (width - len(a)) for a in acc], dtype=torch.int32, device=dev)   # padding is not read
    cu = torch.tensor(np.concatenate([[0], np.cumsum(ns)]), dtype=torch.int32, device=dev)
    cl = torch.tensor(lens, dtype=torch.int32, device=dev)
    new = torch.full((len(ns),), -7, dtype=torch.int32, device=dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    btc = bt.cpu()
    want = [_expect(c, btc, lens, ns, acc, num, hkv) for c in (kc, vc)]
    if sc is not None:
        want_s = [_expect(sc[:, :, w].unsqueeze(-1), btc, lens, ns, acc, num, hkv) for w in range(2)]
    pkv.kv_cache_accept(kc, vc, bt, cl, at, torch.tensor(num, dtype=torch.int32, device=dev), new, max(ns), cu_q_lens=cu,
                        scales=sc, device_status=status)
    assert status.item() == 0
    assert new.tolist() == [c - n + m for c, n, m in zip(lens, ns, num)]
    for c, w in zip((kc, vc), want):
        assert torch.equal(_rows(c, hkv), w)
    if sc is not None:
        for w in range(2):
            assert torch.equal(_rows(sc[:, :, w].unsqueeze(-1), hkv), want_s[w])


def test_a_sequence_that_breaks_a_rule_is_left_as_it_is(dev):
    import paged_kv_cache_252_gb300 as pkv
    g = torch.Generator(device=dev)
    g.manual_seed(1)
    S, n = 6, 4
    lens = [20, 20, 20, 20, 20, 20]
    bt, total = op.tables(lens, g, dev)
    kc, vc, _ = op.make_cache("fp16", total, 2, 64, g, dev)
    acc = torch.tensor([[0, 2], [1, 4], [3, -1], [1, 3], [2, 3], [3, 3]], dtype=torch.int32, device=dev)
    num = torch.tensor([2, 2, 2, 3, 2, 2], dtype=torch.int32, device=dev)     # seq 3: more than max_accepted
    cl = torch.tensor([20, 20, 20, 20, 3, 20], dtype=torch.int32, device=dev)  # seq 4: fewer tokens than drafts
    bt[5, 1] = total                                                            # seq 5: a block out of range
    before = kc.clone(), vc.clone()
    new = torch.zeros(S, dtype=torch.int32, device=dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    pkv.kv_cache_accept(kc, vc, bt, cl, acc, num, new, n, device_status=status)
    assert status.item() == 0x4 | 0x2
    assert new.tolist() == [18, 20, 20, 20, 3, 20]
    lens0 = [[0, 2]] + [[]] * 5
    for c, b in zip((kc, vc), before):
        want = _expect(b, bt.cpu(), lens, [n] * S, lens0, [2] + [0] * 5, 2)
        assert torch.equal(_rows(c, 2), want)


def test_accept_replays_from_a_graph(dev):
    import paged_kv_cache_252_gb300 as pkv
    g = torch.Generator(device=dev)
    g.manual_seed(2)
    lens, n = [40, 23], 7
    bt, total = op.tables(lens, g, dev)
    kc, vc, _ = op.make_cache("bf16", total, 2, 128, g, dev)
    cl = torch.tensor(lens, dtype=torch.int32, device=dev)
    acc = torch.zeros((2, 3), dtype=torch.int32, device=dev)
    num = torch.zeros(2, dtype=torch.int32, device=dev)
    new = torch.zeros(2, dtype=torch.int32, device=dev)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkv.kv_cache_accept(kc, vc, bt, cl, acc, num, new, n)
    k0, v0 = kc.clone(), vc.clone()
    for a, m in (([[0, 3, 6], [1, 2, 5]], [3, 2]), ([[4, 0, 0], [6, 6, 6]], [1, 3])):
        acc.copy_(torch.tensor(a, dtype=torch.int32))
        num.copy_(torch.tensor(m, dtype=torch.int32))
        want = _expect(kc, bt.cpu(), lens, [n, n], a, m, 2)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(_rows(kc, 2), want) and new.tolist() == [c - n + x for c, x in zip(lens, m)]
