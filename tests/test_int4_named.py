"""An INT4 cache is bytes, as an E5M2 cache is: what calls do that say which it is, say nothing, or say it of another cache."""
import pytest
import torch

import paged_kv_cache_252_gb300 as pkv
from paged_kv_cache_252_gb300 import api


@pytest.fixture
def no_gpu(monkeypatch):
    """Argument checks on host tensors; a call that passes them must not get to the library."""
    class Library:
        def __getattr__(self, name):
            def call(*args):
                if name.endswith("_bytes"):
                    return 4096
                raise AssertionError(f"{name} was called")
            return call
    monkeypatch.setattr(api, "_lib", Library())
    monkeypatch.setattr(api, "_placed", lambda names, tensors: 0)
    monkeypatch.setattr(api, "_need_cuda_contig", lambda name, t: None)
    monkeypatch.setattr(api, "_head_rows", lambda name, t, dev, heads, head: heads)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("zero", [True, False])
def test_calls_that_do_not_name_the_type_are_refused(no_gpu, d, zero):
    k, v = pkv.alloc_kv_cache(3, 2, d, "int4", "cpu", zero)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32)
    x, slots = torch.zeros((4, 2, d // 2), dtype=torch.float16), i32(0, 1, 2, 3)
    q, tables, lens, cu = torch.zeros((4, 8, d // 2), dtype=torch.float16), i32(0, 1, 2, 0).view(4, 1), i32(1, 1, 1, 1), i32(0, 1, 2, 3, 4)
    masks = torch.ones(4, dtype=torch.int64)
    for call in (lambda: pkv.copy_blocks(k, v, i32(0), i32(1)),
                 lambda: pkv.kv_cache_accept(k, v, tables, lens, i32(0, 0, 0, 0).view(4, 1), lens, None, 1),
                 lambda: pkv.kv_cache_write(x, x, slots, k, v),
                 lambda: pkv.kv_cache_read(x, x, slots, k, v),
                 lambda: pkv.paged_attention_decode(q, q, k, v, tables, lens, 1, 0.1),
                 lambda: pkv.paged_attention_decode_noalloc(q, q, k, v, tables, lens, 1, 0.1),
                 lambda: pkv.paged_attention_decode_varlen(q, q, cu, k, v, tables, lens, 1, 0.1),
                 lambda: pkv.paged_attention_decode_tree(q, q, masks, k, v, tables, lens, 1, 0.1),
                 lambda: pkv.paged_attention_decode_chunked(q, q, [1] * 4, [1] * 4, k, v, tables, 0.1),
                 lambda: pkv.paged_attention_prefill(q, q, cu, k, v, tables, lens, 0.1),
                 lambda: pkv.rotary_write(q, q, x, x, slots, slots, k, v, torch.ones(8, dtype=torch.float64))):
        with pytest.raises(pkv.PagedKVError):
            call()


def test_other_caches_need_no_name():
    for kv, code in (("fp16", 0), ("bf16", 1), ("e5m2", 2), ("int8", 3)):
        k, _ = pkv.alloc_kv_cache(2, 1, 64, kv, "cpu")
        assert api._kv_code(None, k) == code
    k, _ = pkv.alloc_kv_cache(2, 1, 64, "int4", "cpu")
    assert api._kv_code("int4", k) == api._kv_code(pkv.KV_INT4, k) == 4


@pytest.mark.parametrize("d", [64, 128])
def test_workspace_of_an_int4_cache_is_of_its_head_size(monkeypatch, d):
    import contextlib
    asked = []

    class Library:
        def pkv_decode_workspace_bytes(self, S, Hq, n, desc):
            asked.append(desc._obj.head_size)
            return 1000 * desc._obj.head_size
    monkeypatch.setattr(api, "_lib", Library())
    monkeypatch.setattr(torch.cuda, "device", lambda dev: contextlib.nullcontext())
    k, _ = pkv.alloc_kv_cache(2, 1, d, "int4", "cpu")
    for name in ("int4", pkv.KV_INT4):
        assert pkv.decode_workspace_bytes(8, 4, 1, k, name) == 1000 * d
    with pytest.raises(pkv.PagedKVError):
        pkv.decode_workspace_bytes(8, 4, 1, k)
    e, _ = pkv.alloc_kv_cache(2, 1, d, "e5m2", "cpu")
    assert pkv.decode_workspace_bytes(8, 4, 1, e) == pkv.decode_workspace_bytes(8, 4, 1, e, "e5m2") == 1000 * d
    assert asked == [d] * 4


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", [torch.int8, torch.float8_e5m2, torch.float16])
def test_other_tensors_named_an_int4_cache_are_refused(no_gpu, d, dtype):
    k = torch.zeros((3, 2, 16, d // 2), dtype=torch.uint8).to(dtype)
    v, sc = k.clone(), pkv.alloc_kv_scales(3, 2, "cpu", kv_dtype="int4", head_size=d)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32)
    x, slots = torch.zeros((4, 2, d), dtype=torch.float16), i32(0, 1, 2, 3)
    q, tables, lens = torch.zeros((4, 8, d), dtype=torch.float16), i32(0, 1, 2, 0).view(4, 1), i32(1, 1, 1, 1)
    for call in (lambda: pkv.copy_blocks(k, v, i32(0), i32(1), "int4", scales=sc),
                 lambda: pkv.kv_cache_accept(k, v, tables, lens, i32(0, 0, 0, 0).view(4, 1), lens, None, 1, "int4", scales=sc),
                 lambda: pkv.kv_cache_write_int4(x, x, slots, k, v, sc),
                 lambda: pkv.kv_cache_read(x, x, slots, k, v, "int4", scales=sc),
                 lambda: pkv.paged_attention_decode_int4(q, q, k, v, sc, tables, lens, 1, 0.1),
                 lambda: pkv.paged_attention_decode_chunked(q, q, [1] * 4, [1] * 4, k, v, tables, 0.1, "int4", scales=sc)):
        with pytest.raises(pkv.PagedKVError, match="uint8"):
            call()


@pytest.mark.parametrize("held,named", [(a, b) for a in ("fp16", "bf16", "e5m2", "int8") for b in ("fp16", "bf16", "e5m2", "int8", "int4")
                                        if (a in ("fp16", "bf16")) != (b in ("fp16", "bf16"))])
def test_a_cache_named_wider_or_narrower_than_it_is_is_refused(no_gpu, held, named):
    """Elements twice as large as the tensor's would lie beyond it."""
    d = 64
    k, v = pkv.alloc_kv_cache(3, 2, d, held, "cpu")
    sc = pkv.alloc_kv_scales(3, 2, "cpu") if named == "int8" else (
        torch.zeros((3, 2, 2, 16, 2, 2), dtype=torch.float16) if named == "int4" else None)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32)
    head = 2 * d if named == "int4" else d
    x, slots = torch.zeros((4, 2, head), dtype=torch.float16), i32(0, 1, 2, 3)
    q, tables, lens, cu = torch.zeros((4, 8, head), dtype=torch.float16), i32(0, 1, 2, 0).view(4, 1), i32(1, 1, 1, 1), i32(0, 1, 2, 3, 4)
    for call in (lambda: pkv.copy_blocks(k, v, i32(0), i32(1), named, scales=sc),
                 lambda: pkv.kv_cache_accept(k, v, tables, lens, i32(0, 0, 0, 0).view(4, 1), lens, None, 1, named, scales=sc),
                 lambda: pkv.kv_cache_write(x, x, slots, k, v, named),
                 lambda: pkv.kv_cache_read(x, x, slots, k, v, named, scales=sc),
                 lambda: pkv.paged_attention_decode(q, q, k, v, tables, lens, 1, 0.1, named),
                 lambda: pkv.paged_attention_decode_noalloc(q, q, k, v, tables, lens, 1, 0.1, named),
                 lambda: pkv.paged_attention_decode_varlen(q, q, cu, k, v, tables, lens, 1, 0.1, named, scales=sc),
                 lambda: pkv.paged_attention_decode_tree(q, q, slots.long(), k, v, tables, lens, 1, 0.1, named, scales=sc),
                 lambda: pkv.paged_attention_decode_chunked(q, q, [1] * 4, [1] * 4, k, v, tables, 0.1, named, scales=sc),
                 lambda: pkv.paged_attention_prefill(q, q, cu, k, v, tables, lens, 0.1, named, scales=sc),
                 lambda: pkv.rotary_write(q, q, x, x, slots, slots, k, v, torch.ones(8, dtype=torch.float64), named, scales=sc)):
        with pytest.raises(pkv.PagedKVError):
            call()


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_a_workspace_of_the_told_size_serves_the_call(d):
    import _int4 as i4
    from test_gpu_scratch import Call
    c = Call("decode", "int4", [700, 3, 2000], d=d)
    want = c()
    ws = torch.zeros(pkv.decode_workspace_bytes(3, 8, 3, c.k, "int4"), dtype=torch.uint8, device="cuda")
    assert torch.equal(c(workspace=ws), want)
    i4.assert_within(want, *i4.attention(c.q, c.k, c.v, c.sc, c.tables, c.lens, c.cu, c.scale))
