"""kv_cache_accept refuses to write its new lengths over what its blocks read. No GPU needed."""
import ctypes

import pytest

import paged_kv_cache_252_gb300.api as api

vp = ctypes.c_void_p
AT = {"bt": 0x10000, "cl": 0x20000, "cu": 0x30000, "acc": 0x40000, "num": 0x50000}   # addresses, never read
S, BLOCKS, MOST = 3, 4, 5
SIZE = {"bt": S * BLOCKS, "cl": S, "cu": S + 1, "acc": S * MOST, "num": S}


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    return api.load_library()


def _accept(lib, new, cu=True):
    desc = ctypes.byref(api._CacheDesc(32, 16, 2, 64))
    return lib.pkv_kv_cache_accept(vp(0x100000), vp(0x200000), None, 0, desc, vp(AT["bt"]), BLOCKS, vp(AT["cl"]),
                                   vp(AT["cu"]) if cu else None, S, 8, vp(AT["acc"]), MOST, vp(AT["num"]), vp(new), None,
                                   None)


@pytest.mark.parametrize("name", list(AT))
def test_new_lengths_over_an_input(lib, name):
    a, n = AT[name], SIZE[name]
    for first in (a, a - 4 * (S - 1), a + 4 * (n - 1)):   # the same place, the last on its first, the first on its last
        assert _accept(lib, first) == -1


def test_new_lengths_beside_the_inputs(lib):
    """No refusal (here it then finds no device, or, where there is one, this is not run)."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("would launch on these addresses")
    for a, n in ((AT[k], SIZE[k]) for k in AT):
        assert _accept(lib, a - 4 * S) != -1 and _accept(lib, a + 4 * n) != -1
    assert _accept(lib, AT["cu"], cu=False) != -1
