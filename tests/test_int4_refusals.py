"""Calls on an INT4 cache that are refused, on the host: C entries and the binding's checks."""
import ctypes

import pytest
import torch

import paged_kv_cache_252_gb300 as pkv
from paged_kv_cache_252_gb300 import api, build

vp = ctypes.c_void_p
FAKE = vp(0x1000)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return pkv.load_library()


def _desc(nb=32, bs=16, h=2, d=128):
    return ctypes.byref(api._CacheDesc(nb, bs, h, d))


def _write(lib, **kw):
    a = dict(key=FAKE, value=FAKE, dt=0, T=4, slots=FAKE, kc=FAKE, vc=FAKE, sc=FAKE, desc=_desc(), st=None)
    a.update(kw)
    return lib.pkv_kv_cache_write_int4(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    ({"T": -1}, -1), ({"dt": 2}, -2), ({"dt": 4}, -2), ({"desc": None}, -1), ({"desc": _desc(d=96)}, -1),
    ({"desc": _desc(bs=8)}, -1), ({"desc": _desc(nb=0)}, -1), ({"key": None}, -1), ({"value": vp(0x1008)}, -1),
    ({"slots": None}, -1), ({"slots": vp(0x1002)}, -1), ({"kc": None}, -1), ({"vc": vp(0x1004)}, -1), ({"sc": None}, -1),
    ({"sc": vp(0x1008)}, -1), ({"st": vp(0x1001)}, -1), ({"T": 0, "key": None}, 0)])
def test_write_refuses(lib, kw, code):
    assert _write(lib, **kw) == code


def _read(lib, **kw):
    a = dict(key=FAKE, value=FAKE, dt=0, T=4, slots=FAKE, kc=FAKE, vc=FAKE, sc=FAKE, kv=4, desc=_desc(), st=None)
    a.update(kw)
    return lib.pkv_kv_cache_read(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    ({"T": -1}, -1), ({"dt": 2}, -2), ({"kv": 5}, -2), ({"kv": -1}, -2), ({"sc": None}, -1), ({"kv": 3, "sc": None}, -1),
    ({"kv": 0}, -1), ({"kv": 2}, -1), ({"desc": None}, -1), ({"desc": _desc(d=256)}, -1), ({"key": vp(0x1004)}, -1),
    ({"value": None}, -1), ({"slots": vp(0x1001)}, -1), ({"kc": vp(0x1008)}, -1), ({"T": 0, "key": None}, 0)])
def test_read_refuses(lib, kw, code):
    assert _read(lib, **kw) == code


def _decode(lib, **kw):
    a = dict(out=FAKE, q=FAKE, dt=0, cu=None, masks=None, R=8, S=8, hq=8, n=1, kc=FAKE, vc=FAKE, sc=FAKE, desc=_desc(), bt=FAKE,
             mbs=4, cl=FAKE, scale=0.1, ws=FAKE, wb=1 << 30, st=None)
    a.update(kw)
    return lib.pkv_paged_attention_decode_int4(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    ({"S": -1}, -1), ({"hq": 0}, -1), ({"hq": 7}, -1), ({"n": 0}, -1), ({"mbs": 0}, -1), ({"dt": 2}, -2), ({"hq": 130}, -2),
    ({"n": 17}, -2), ({"masks": FAKE, "n": 65, "hq": 2}, -2), ({"desc": _desc(d=32)}, -1), ({"R": 7}, -1), ({"R": 0}, -1),
    ({"cu": FAKE, "R": 0}, -1), ({"sc": None}, -1), ({"q": None}, -1), ({"out": vp(0x1008)}, -1), ({"sc": vp(0x1004)}, -1),
    ({"masks": vp(0x1004)}, -1), ({"cu": vp(0x1002)}, -1), ({"bt": None}, -1), ({"cl": vp(0x1001)}, -1), ({"ws": None}, -1),
    ({"mbs": (1 << 26) + 1}, -2), ({"S": 1 << 30, "R": 1 << 30}, -2), ({"S": 0}, 0)])
def test_decode_refuses(lib, kw, code):
    assert _decode(lib, **kw) == code


def test_calls_that_do_not_take_an_int4_cache(lib):
    d = _desc()
    assert lib.pkv_paged_attention_decode(FAKE, FAKE, 4, 4, 1, FAKE, FAKE, 4, d, FAKE, 4, FAKE, 0.1, FAKE, 1 << 30, None, None) == -2
    assert lib.pkv_kv_cache_write(FAKE, FAKE, 0, 4, FAKE, FAKE, FAKE, 4, d, None, None) == -2
    assert lib.pkv_rotary_write(FAKE, 1024, FAKE, 1024, FAKE, 256, FAKE, 256, 0, 4, 8, FAKE, 8, FAKE, FAKE, 128, 0, 1.0, FAKE,
                                FAKE, FAKE, 4, d, None, None) == -2
    ql = (ctypes.c_int32 * 1)(1)
    assert lib.pkv_paged_attention_decode_chunked(FAKE, FAKE, ql, ql, 1, 4, FAKE, FAKE, None, 4, d, FAKE, 4, 0.1, FAKE, 1 << 30,
                                                  None, None) == -2
    bad = (ctypes.c_int32 * 1)(0)
    assert lib.pkv_paged_attention_decode_int4_chunked(FAKE, FAKE, 0, bad, ql, 1, 4, FAKE, FAKE, FAKE, d, FAKE, 4, 0.1, FAKE,
                                                       1 << 30, None, None) == -1
    assert lib.pkv_copy_blocks(FAKE, FAKE, None, 4, d, FAKE, FAKE, 1, None, None) == -1
    assert lib.pkv_kv_cache_accept(FAKE, FAKE, None, 4, d, FAKE, 4, FAKE, None, 2, 4, FAKE, 4, FAKE, None, None, None) == -1


def test_allocations():
    k, v = pkv.alloc_kv_cache(3, 2, 128, "int4", "cpu")
    assert k.shape == v.shape == (3, 2, 16, 64) and k.dtype == torch.uint8 and not k.any()
    sc = pkv.alloc_kv_scales(3, 2, "cpu", kv_dtype="int4", head_size=128)
    assert sc.shape == (3, 2, 2, 16, 2, 2) and sc.dtype == torch.float16 and not sc.any()
    assert pkv.alloc_kv_scales(3, 2, "cpu").shape == (3, 2, 2, 16)
    for bad in (lambda: pkv.alloc_kv_cache(3, 2, 96, "int4", "cpu"), lambda: pkv.alloc_kv_scales(3, 2, "cpu", kv_dtype="int4"),
                lambda: pkv.alloc_kv_scales(3, 2, "cpu", kv_dtype="fp16")):
        with pytest.raises(pkv.PagedKVError):
            bad()


def test_binding_refuses_host_tensors_and_wrong_scales(monkeypatch):
    k, v = pkv.alloc_kv_cache(3, 2, 128, "int4", "cpu")
    sc = pkv.alloc_kv_scales(3, 2, "cpu", kv_dtype="int4", head_size=128)
    x, slots = torch.zeros((4, 2, 128), dtype=torch.float16), torch.zeros(4, dtype=torch.int32)
    with pytest.raises(pkv.PagedKVError, match="CUDA"):
        pkv.kv_cache_write_int4(x, x, slots, k, v, sc)
    # the shape checks behind the placement's
    monkeypatch.setattr(api, "_placed", lambda names, tensors: 0)
    monkeypatch.setattr(api, "_need_cuda_contig", lambda name, t: None)
    write = lambda key=x, value=x, slots=slots, k=k, v=v, sc=sc: pkv.kv_cache_write_int4(key, value, slots, k, v, sc)
    read = lambda key=x, value=x, kv="int4", k=k, v=v, sc=sc: pkv.kv_cache_read(key, value, slots, k, v, kv, scales=sc)
    q, tables, lens = torch.zeros((4, 8, 128), dtype=torch.float16), torch.zeros((4, 2), dtype=torch.int32), torch.zeros(4, dtype=torch.int32)
    attend = lambda out=q, q=q, sc=sc, bt=tables, cl=lens, n=1, k=k, v=v: pkv.paged_attention_decode_int4(out, q, k, v, sc, bt, cl, n, 0.1)
    varlen = lambda cu, q=q: pkv.paged_attention_decode_varlen(q, q, cu, k, v, tables, lens, 2, 0.1, "int4", scales=sc)
    tree = lambda masks: pkv.paged_attention_decode_tree(q, q, masks, k, v, tables, lens, 1, 0.1, "int4", scales=sc)
    for bad in (lambda: write(key=x[:3]), lambda: write(value=x.bfloat16()), lambda: write(slots=slots.long()),
                lambda: write(slots=slots[:2]), lambda: write(sc=sc.float()), lambda: write(sc=sc[:, :, :1]),
                lambda: write(k=k.view(torch.int8), v=v.view(torch.int8)), lambda: write(v=v[:2]),
                lambda: write(key=x[..., :64], value=x[..., :64]),
                lambda: read(kv=None), lambda: read(sc=None), lambda: read(kv="int8"), lambda: read(key=x[:2], value=x[:2]),
                lambda: attend(out=q[:2]), lambda: attend(sc=None), lambda: attend(bt=tables[:2]), lambda: attend(n=2),
                lambda: attend(cl=lens.long()), lambda: attend(q=q[..., :64], out=q[..., :64]),
                lambda: attend(out=q.bfloat16()), lambda: varlen(torch.zeros(4, dtype=torch.int32)),
                lambda: varlen(torch.zeros(5, dtype=torch.int64)), lambda: varlen(torch.zeros(5, dtype=torch.int32), q[:3]),
                lambda: tree(torch.zeros(4, dtype=torch.int32)), lambda: tree(torch.zeros(3, dtype=torch.int64))):
        with pytest.raises(pkv.PagedKVError):
            bad()
