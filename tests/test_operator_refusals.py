"""Calls that the rotary, prefill and accept operators refuse, through the C ABI and the
Python binding, and the allocator's truncate. No GPU needed."""
import ctypes

import numpy as np
import pytest
import torch

import paged_kv_cache_252_gb300.api as api
from oracle.block_pool import BlockPoolModel, INVALID, OK

vp = ctypes.c_void_p
FAKE = vp(0x1000)


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    return api.load_library()


def _desc(nb=32, bs=16, hkv=2, d=64):
    return ctypes.byref(api._CacheDesc(nb, bs, hkv, d))


def _embed(lib, **kw):
    a = dict(out=FAKE, os=128, x=FAKE, xs=128, dt=0, T=4, H=2, D=64, pos=FAKE, pb=8, inv=FAKE, rd=32, inter=0, f=1.0)
    a.update(kw)
    return lib.pkv_rotary_embed(a["out"], a["os"], a["x"], a["xs"], a["dt"], a["T"], a["H"], a["D"], a["pos"], a["pb"],
                                a["inv"], a["rd"], a["inter"], a["f"], 0, None)


@pytest.mark.parametrize("kw,code", [
    ({"dt": 2}, -2), ({"T": -1}, -1), ({"H": 0}, -1), ({"D": 96}, -2), ({"rd": 8}, -2), ({"rd": 24}, -2),
    ({"rd": 80}, -2), ({"pb": 2}, -1), ({"pos": None}, -1), ({"inv": None}, -1), ({"inv": vp(0x1004)}, -1),
    ({"pos": vp(0x1004)}, -1), ({"f": float("inf")}, -1), ({"f": float("nan")}, -1), ({"out": None}, -1),
    ({"x": vp(0x1008)}, -1), ({"xs": 120}, -1), ({"os": 132}, -1)])
def test_rotary_embed_refuses(lib, kw, code):
    assert _embed(lib, **kw) == code


def test_rotary_embed_of_nothing(lib):
    assert _embed(lib, T=0, out=None, x=None, pos=None, inv=None) == 0


def _write(lib, **kw):
    a = dict(qo=FAKE, qos=256, q=FAKE, qs=256, k=FAKE, ks=128, v=FAKE, vs=128, sd=0, T=4, hq=4, pos=FAKE, pb=4,
             slots=FAKE, inv=FAKE, rd=64, f=1.0, kc=FAKE, vc=FAKE, sc=None, kv=0, desc=_desc(), st=None)
    a.update(kw)
    return lib.pkv_rotary_write(a["qo"], a["qos"], a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["sd"], a["T"],
                                a["hq"], a["pos"], a["pb"], a["slots"], a["inv"], a["rd"], 0, a["f"], a["kc"], a["vc"],
                                a["sc"], a["kv"], a["desc"], a["st"], None)


@pytest.mark.parametrize("kw,code", [
    ({"desc": None}, -1), ({"desc": _desc(d=96)}, -1), ({"desc": _desc(bs=8)}, -1), ({"sd": 1}, -2), ({"kv": 1}, -2),
    ({"sd": 1, "kv": 2}, -2), ({"kv": 3}, -1), ({"sc": FAKE}, -1), ({"rd": 128}, -2), ({"hq": 0}, -1),
    ({"slots": None}, -1), ({"slots": vp(0x1002)}, -1), ({"qs": 248}, -1), ({"ks": 120}, -1), ({"v": vp(0x1004)}, -1),
    ({"kc": None}, -1), ({"vc": vp(0x1008)}, -1), ({"st": vp(0x1001)}, -1), ({"qo": None}, -1)])
def test_rotary_write_refuses(lib, kw, code):
    assert _write(lib, **kw) == code


def _prefill(lib, **kw):
    a = dict(out=FAKE, q=FAKE, cu=FAKE, R=8, S=2, hq=4, kc=FAKE, vc=FAKE, sc=None, kv=0, desc=_desc(), bt=FAKE, mbs=4,
             cl=FAKE, scale=0.125, ws=FAKE, wb=0, st=None)
    a.update(kw)
    return lib.pkv_paged_attention_prefill(a["out"], a["q"], a["cu"], a["R"], a["S"], a["hq"], a["kc"], a["vc"], a["sc"],
                                           a["kv"], a["desc"], a["bt"], a["mbs"], a["cl"], a["scale"], a["ws"], a["wb"],
                                           a["st"], None)


@pytest.mark.parametrize("kw,code", [
    ({"S": -1}, -1), ({"R": -1}, -1), ({"hq": 0}, -1), ({"hq": 3}, -1), ({"hq": 130}, -2), ({"mbs": 0}, -1),
    ({"desc": None}, -1), ({"desc": _desc(d=32)}, -1), ({"kv": 4}, -2), ({"kv": 3}, -1), ({"sc": FAKE}, -1),
    ({"scale": 0.0}, -1), ({"scale": -1.0}, -1), ({"scale": float("nan")}, -1), ({"scale": float("inf")}, -1),
    ({"R": 1 << 29}, -2), ({"mbs": (1 << 26) + 1}, -2), ({"out": None}, -1), ({"cu": None}, -1), ({"ws": None}, -1),
    ({"q": vp(0x1008)}, -1), ({"bt": vp(0x1002)}, -1), ({"ws": vp(0x1008)}, -1), ({"st": vp(0x1002)}, -1)])
def test_prefill_refuses(lib, kw, code):
    assert _prefill(lib, **kw) == code


def test_prefill_of_nothing(lib):
    assert _prefill(lib, S=0, cu=None, bt=None, cl=None) == 0
    assert _prefill(lib, R=0, q=None, out=None) == 0


def _accept(lib, **kw):
    a = dict(kc=FAKE, vc=FAKE, sc=None, kv=0, desc=_desc(), bt=FAKE, mbs=4, cl=FAKE, cu=None, S=2, n=4, acc=FAKE, ma=4,
             num=FAKE, new=vp(0x2000), st=None)
    a.update(kw)
    return lib.pkv_kv_cache_accept(a["kc"], a["vc"], a["sc"], a["kv"], a["desc"], a["bt"], a["mbs"], a["cl"], a["cu"],
                                   a["S"], a["n"], a["acc"], a["ma"], a["num"], a["new"], a["st"], None)


@pytest.mark.parametrize("kw,code", [
    ({"S": -1}, -1), ({"n": 0}, -1), ({"n": 65}, -2), ({"ma": 0}, -1), ({"mbs": 0}, -1), ({"kv": 7}, -2),
    ({"kv": 3}, -1), ({"sc": FAKE}, -1), ({"desc": _desc(bs=32)}, -1), ({"acc": None}, -1), ({"num": None}, -1),
    ({"cl": None}, -1), ({"kc": vp(0x1004)}, -1), ({"num": vp(0x1001)}, -1),
    ({"new": FAKE}, -1), ({"new": vp(0x1004)}, -1), ({"new": vp(0xFFC)}, -1)])
def test_accept_refuses(lib, kw, code):
    assert _accept(lib, **kw) == code


def test_accept_of_nothing(lib):
    assert _accept(lib, S=0, bt=None, cl=None, acc=None, num=None) == 0


# ---- the binding's shape checks ---------------------------------------------------------

class _Reached(Exception):
    pass


@pytest.fixture
def stub(monkeypatch):
    """Host tensors stand in for CUDA ones, and the library is never reached."""
    class Cuda(torch.Tensor):
        def get_device(self):
            return 0
    real = api._head_rows
    monkeypatch.setattr(api, "_placed", lambda names, tensors: 0)
    monkeypatch.setattr(api, "_head_rows", lambda n, t, dev, h, d: real(n, t.as_subclass(Cuda), dev, h, d))
    monkeypatch.setattr(api, "_lib", None)

    def no_library():
        raise _Reached()
    monkeypatch.setattr(api, "load_library", no_library)


def _prefill_args():
    kc = torch.zeros(10, 2, 16, 64, dtype=torch.float16)
    q = torch.zeros(7, 8, 64, dtype=torch.float16)
    return dict(out=q.clone(), q=q, cu_q_lens=torch.zeros(4, dtype=torch.int32), k_cache=kc, v_cache=kc.clone(),
                block_tables=torch.zeros(3, 4, dtype=torch.int32), context_lens=torch.ones(3, dtype=torch.int32), scale=0.1)


@pytest.mark.parametrize("change", [
    {}, {"cu_q_lens": torch.zeros(3, dtype=torch.int32)}, {"cu_q_lens": torch.zeros(4, dtype=torch.int64)},
    {"out": torch.zeros(6, 8, 64, dtype=torch.float16)}, {"q": torch.zeros(7, 8, 64, dtype=torch.bfloat16)},
    {"block_tables": torch.zeros(2, 4, dtype=torch.int32)}, {"scales": torch.zeros(10, 2, 2, 16)},
    {"device_status": torch.zeros(1)}, {"v_cache": torch.zeros(10, 2, 16, 64, dtype=torch.bfloat16)},
    {"context_lens": torch.ones(3, 1, dtype=torch.int32)}])
def test_prefill_binding(stub, change):
    with pytest.raises(_Reached if not change else api.PagedKVError):
        api.paged_attention_prefill(**{**_prefill_args(), **change})


def _write_args():
    kc = torch.zeros(10, 2, 16, 64, dtype=torch.float16)
    qkv = torch.zeros(5, 8 * 64, dtype=torch.float16)
    q, k, v = (qkv[:, a * 64:b * 64].view(5, b - a, 64) for a, b in ((0, 4), (4, 6), (6, 8)))
    return dict(q_out=torch.zeros(5, 4, 64, dtype=torch.float16), q=q, key=k, value=v, positions=torch.arange(5),
                slot_mapping=torch.zeros(5, dtype=torch.int32), k_cache=kc, v_cache=kc.clone(),
                inv_freq=torch.zeros(16, dtype=torch.float64))


@pytest.mark.parametrize("change", [
    {}, {"q_out": torch.zeros(5, 4, 128, dtype=torch.float16)}, {"q_out": torch.zeros(4, 4, 64, dtype=torch.float16)},
    {"key": torch.zeros(5, 3, 64, dtype=torch.float16)}, {"value": torch.zeros(5, 2, 64, dtype=torch.bfloat16)},
    {"positions": torch.arange(6)}, {"positions": torch.arange(5.0)}, {"slot_mapping": torch.zeros(5, dtype=torch.int64)},
    {"inv_freq": torch.zeros(16)}, {"inv_freq": torch.zeros(4, dtype=torch.float64)},
    {"inv_freq": torch.zeros(40, dtype=torch.float64)}, {"attn_factor": float("nan")},
    {"q": torch.zeros(5, 64, 4, dtype=torch.float16).transpose(1, 2)},
    {"q": torch.zeros(5, 260, dtype=torch.float16)[:, :256].view(5, 4, 64)},
    {"q": torch.zeros(1, 4, 64, dtype=torch.float16).expand(5, 4, 64)}])
def test_rotary_write_binding(stub, change):
    with pytest.raises(_Reached if not change else api.PagedKVError):
        api.rotary_write(**{**_write_args(), **change})


def _accept_args():
    kc = torch.zeros(10, 2, 16, 64, dtype=torch.float16)
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)
    return dict(k_cache=kc, v_cache=kc.clone(), block_tables=i(3, 4), context_lens=i(3), accepted=i(3, 2),
                num_accepted=i(3), new_context_lens=i(3), max_q_per_seq=4)


@pytest.mark.parametrize("change", [
    {}, {"accepted": torch.zeros(2, 2, dtype=torch.int32)}, {"accepted": torch.zeros(3, 2, dtype=torch.int64)},
    {"num_accepted": torch.zeros(2, dtype=torch.int32)}, {"new_context_lens": torch.zeros(4, dtype=torch.int32)},
    {"cu_q_lens": torch.zeros(3, dtype=torch.int32)}, {"scales": torch.zeros(10, 2, 2, 16)},
    {"block_tables": torch.zeros(2, 4, dtype=torch.int32)}])
def test_accept_binding(stub, change):
    with pytest.raises(_Reached if not change else api.PagedKVError):
        api.kv_cache_accept(**{**_accept_args(), **change})


def test_host_tensors_are_refused():
    with pytest.raises(api.PagedKVError):
        api.paged_attention_prefill(**_prefill_args())
    with pytest.raises(api.PagedKVError):
        api.rotary_write(**_write_args())
    with pytest.raises(api.PagedKVError):
        api.kv_cache_accept(**_accept_args())


# ---- frequencies ----------------------------------------------------------------------------

def test_frequencies_and_their_scalings():
    f, a = api.rotary_inv_freq(128, 10000.0, device="cpu")
    assert a == 1.0 and f.dtype == torch.float64 and f[0] == 1.0
    assert abs(f[63].item() - 10000.0 ** (-126 / 128)) < 1e-18
    lin, _ = api.rotary_inv_freq(128, 10000.0, scaling="linear", factor=4.0, device="cpu")
    assert torch.allclose(lin, f / 4, rtol=1e-15)
    ntk, _ = api.rotary_inv_freq(128, 10000.0, scaling="base", factor=4.0, device="cpu")
    assert ntk[0] == 1.0 and abs(ntk[63] / f[63] - 0.25) < 1e-12
    band, a = api.rotary_inv_freq(128, 500000.0, scaling="bands", factor=8.0, original_context=8192, device="cpu")
    g, _ = api.rotary_inv_freq(128, 500000.0, device="cpu")
    turns = 8192 * g / (2 * np.pi)
    assert a == 1.0 and torch.equal(band[turns >= 4], g[turns >= 4])
    assert torch.allclose(band[turns <= 1], g[turns <= 1] / 8, rtol=1e-15)
    mid = (turns > 1) & (turns < 4)
    assert mid.any() and ((band < g) & (band > g / 8))[mid].all()
    ramp, a = api.rotary_inv_freq(128, 10000.0, scaling="ramp", factor=16.0, original_context=4096, device="cpu")
    assert abs(a - (0.1 * np.log(16.0) + 1)) < 1e-12
    turns = 4096 * f / (2 * np.pi)
    assert torch.equal(ramp[turns >= 33], f[turns >= 33])
    assert torch.allclose(ramp[turns <= 0.9], f[turns <= 0.9] / 16, rtol=1e-15)
    assert (ramp[1:] < ramp[:-1]).all()


@pytest.mark.parametrize("kw", [{"rotary_dim": 7}, {"rotary_dim": 0}, {"rotary_dim": 64, "base": 0.0},
                                {"rotary_dim": 64, "scaling": "other"}, {"rotary_dim": 64, "scaling": "ramp"},
                                {"rotary_dim": 2, "scaling": "base"},
                                {"rotary_dim": 64, "scaling": "bands", "original_context": 10, "low": 5.0, "high": 5.0}])
def test_frequencies_refuse(kw):
    with pytest.raises(api.PagedKVError):
        api.rotary_inv_freq(device="cpu", **kw)


# ---- truncate ----------------------------------------------------------------------------------

def _truncate(m, seq, n):
    """The plain model of the block pool, shortened: blocks behind the kept ones lose a reference."""
    if seq not in m.seqs or n < 0 or n > m.seqs[seq][1]:
        return INVALID
    blocks, _ = m.seqs[seq]
    keep = -(-n // 16)
    for b in blocks[keep:]:
        m._dec(b)
    m.seqs[seq] = [blocks[:keep], n]
    return OK


def test_truncate_by_hand(lib):
    a = api.BlockAllocator(6)
    a.add(1)
    a.append(1, 40)
    a.truncate(1, 33)
    assert a.length(1) == 33 and a.block_table(1) == [0, 1, 2] and a.free_blocks() == 3
    a.truncate(1, 32)
    assert a.block_table(1) == [0, 1] and a.free_blocks() == 4 and a.refcount(2) == 0
    a.fork(1, 2)
    a.truncate(1, 5)                       # block 1 stays with the fork, block 0 is shared
    assert a.block_table(1) == [0] and a.refcount(0) == 2 and a.refcount(1) == 1
    slots, copies = a.append(1, 1)         # writing into the shared block copies it first
    assert copies == [(0, 2)] and slots == [2 * 16 + 5]
    a.truncate(1, 0)
    assert a.block_table(1) == [] and a.length(1) == 0
    for bad in ((1, 1), (1, -1), (9, 0)):
        with pytest.raises(api.PagedKVError):
            a.truncate(*bad)


@pytest.mark.parametrize("seed", range(4))
def test_truncate_against_the_model(lib, seed):
    rng = np.random.default_rng(seed)
    a, m = api.BlockAllocator(24), BlockPoolModel(24)
    tok = lambda n: [int(x) for x in rng.integers(0, 2, n)]
    text, nxt = {}, 0
    for _ in range(400):
        what = rng.integers(0, 6)
        live = list(text)
        if what == 0 or not live:
            a.add(nxt), m.add(nxt)
            text[nxt] = []
            nxt += 1
        elif what == 1:
            s, n = live[rng.integers(len(live))], int(rng.integers(0, 30))
            try:
                got = a.append(s, n)
                assert m.append(s, n) == (OK, got[0], got[1])
                text[s] += tok(n)
            except api.PagedKVError:
                assert m.append(s, n)[0] != OK
        elif what == 2:
            s = live[rng.integers(len(live))]
            n = int(rng.integers(0, len(text[s]) + 1))
            a.truncate(s, n)
            assert _truncate(m, s, n) == OK
            text[s] = text[s][:n]
        elif what == 3:
            s = live[rng.integers(len(live))]
            a.fork(s, nxt), m.fork(s, nxt)
            text[nxt] = list(text[s])
            nxt += 1
        elif what == 4:
            s = live[rng.integers(len(live))]
            a.release(s), m.release(s)
            del text[s]
        else:
            s = live[rng.integers(len(live))]
            a.prefix_insert(s, text[s]), m.prefix_insert(s, text[s])
        assert a.free_blocks() == len(m.free)
        assert [a.refcount(b) for b in range(24)] == m.ref
        for s in text:
            assert a.block_table(s) == m.block_table(s) and a.length(s) == len(text[s])
