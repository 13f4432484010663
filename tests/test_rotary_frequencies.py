"""Rotary frequencies that have no meaning are refused. No GPU needed."""
import math

import pytest
import torch

import paged_kv_cache_252_gb300.api as api


@pytest.mark.parametrize("kw", [
    {"base": 1.0, "scaling": "ramp", "factor": 2.0, "original_context": 4096},     # no pair makes fewer turns than another
    {"base": 0.5, "scaling": "ramp", "factor": 2.0, "original_context": 4096},
    {"base": math.inf}, {"base": math.nan}, {"factor": math.inf, "scaling": "linear"}, {"factor": math.nan},
    {"scaling": "bands", "factor": 2.0, "original_context": math.inf},
    {"scaling": "ramp", "factor": 2.0, "original_context": math.nan},
    {"scaling": "bands", "factor": 2.0, "original_context": 4096, "high": math.inf},
    {"scaling": "base", "factor": 1e300, "base": 1e300}])
def test_refused(kw):
    with pytest.raises(api.PagedKVError):
        api.rotary_inv_freq(64, device="cpu", **kw)


@pytest.mark.parametrize("kw", [{"base": 1.0}, {"base": 1.5, "scaling": "ramp", "factor": 2.0, "original_context": 4096},
                                {"base": 0.5}, {"base": 0.5, "scaling": "bands", "factor": 2.0, "original_context": 4096}])
def test_numbers(kw):
    f, a = api.rotary_inv_freq(64, device="cpu", **kw)
    assert torch.isfinite(f).all() and (f > 0).all() and math.isfinite(a)
