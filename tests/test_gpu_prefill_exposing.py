"""Long contexts of which every tile, block and planted position shows in the outputs, against 64 bits.
(test_prefill_bound.py shows that the bound notices each of them missing.)"""
import pytest
import torch

import _bounds
import _exposing as ex
import _operators as op
from test_gpu_prefill import Batch, dev  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("how", ["blocks", "peaks"])
@pytest.mark.parametrize("kv", ["fp16", "bf16", "e5m2", "int8"])
@pytest.mark.parametrize("shape", list(ex.SHAPES))
def test_every_position_counts(dev, kv, shape, how):  # noqa: F811
    D, hq, hkv, ns, lens, s = ex.SHAPES[shape]
    b = Batch(dev, kv, D, hq, hkv, ns, lens)
    ex.fill(b, s, how)
    b.run()
    torch.cuda.synchronize()
    assert b.status.item() == 0
    at, want, tol = _bounds.attention_rows(b, s, ex.tokens_of(ns[s]))
    share = op.assert_within(b.out[at], want, tol, f"{shape} {kv} {how}")
    print(f"{shape} {kv} {how}: at most {share:.2f} of the bound")


@pytest.mark.parametrize("kv", ["fp16", "bf16", "e5m2", "int8"])
@pytest.mark.parametrize("shape", list(ex.SHAPES))
def test_random_values_within_the_narrow_bound(dev, kv, shape):  # noqa: F811
    D, hq, hkv, ns, lens, s = ex.SHAPES[shape]
    b = Batch(dev, kv, D, hq, hkv, ns, lens, seed=11)
    b.run()
    at, want, tol = _bounds.attention_rows(b, s, ex.tokens_of(ns[s]))
    share = op.assert_within(b.out[at], want, tol, f"{shape} {kv}")
    print(f"{shape} {kv}: at most {share:.2f} of the bound")
