"""Rotary angles at positions beyond 2^31, against whole-number arithmetic."""
import math

import pytest
import torch

import _operators as op

BITS = 256   # fraction bits of the reference's turns


def _arctan_inverse(x):
    """2^BITS arctan(1 / x) (whole numbers, off by a few units)."""
    total, term, k = 0, (1 << (BITS + 32)) // x, 1
    while term:
        total += term // k if k % 4 == 1 else -(term // k)
        term //= x * x
        k += 2
    return total >> 32


TWO_PI = 8 * (4 * _arctan_inverse(5) - _arctan_inverse(239))   # Machin: pi / 4 = 4 arctan 1/5 - arctan 1/239


def turn_of(p, f):
    """p f / 2 pi less its whole turns, in [-1/2, 1/2), correct to the double's last bit."""
    num, den = float(f).as_integer_ratio()
    whole = p * num * (1 << (2 * BITS)) // (den * TWO_PI)      # 2^BITS p f / 2 pi
    part = whole & ((1 << BITS) - 1)
    if part >> (BITS - 1):
        part -= 1 << BITS
    return part / (1 << BITS)


def test_the_reference_by_hand():
    assert abs(TWO_PI / (1 << BITS) - 2 * math.pi) < 1e-15
    assert abs(turn_of(1, 1.0) - 1 / (2 * math.pi)) < 1e-16
    assert abs(turn_of(-3, 0.25) + 0.75 / (2 * math.pi)) < 1e-16
    p = 123456
    assert abs(math.remainder(turn_of(p, 0.7) - math.fmod(p * 0.7 / (2 * math.pi), 1.0), 1.0)) < 1e-10


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    return torch.device("cuda:0")


@pytest.mark.gpu
@pytest.mark.parametrize("interleaved", [False, True], ids=["halves", "pairs"])
@pytest.mark.parametrize("first", [(1 << 31) - 2, 1 << 40, (1 << 45) + 12345, (1 << 50) - 77, (1 << 52) + 1, -(1 << 45),
                                   -(1 << 50) + 3])
def test_angles_far_out(dev, first, interleaved):
    """A step is a fraction of a turn to 2^-64, so position p's angle is off by at most |p| 2^-64 turns."""
    import paged_kv_cache_252_gb300 as pkv
    T, H, D = 6, 2, 128
    g = torch.Generator(device=dev)
    g.manual_seed(4)
    inv, _ = pkv.rotary_inv_freq(D, 10000.0, device=dev)
    inv[5], inv[9], inv[20] = 0.9999999, 3.7, -0.031      # frequencies of a user's own
    x = torch.randn((T, H, D), generator=g, device=dev).half()
    pos = [first + 3 * t for t in range(T)]
    out = torch.empty_like(x)
    pkv.rotary_embed(out, x, torch.tensor(pos, device=dev), inv, interleaved=interleaved)
    ang = torch.tensor([[2 * math.pi * turn_of(p, f) for f in inv.tolist()] for p in pos], dtype=torch.float64, device=dev)
    j = torch.arange(D // 2, device=dev)
    re, im = (2 * j, 2 * j + 1) if interleaved else (j, j + D // 2)
    xd, want = x.double(), torch.empty(x.shape, dtype=torch.float64, device=dev)
    c, s = ang.cos()[:, None], ang.sin()[:, None]
    want[..., re] = xd[..., re] * c - xd[..., im] * s
    want[..., im] = xd[..., re] * s + xd[..., im] * c
    size = torch.empty_like(want)
    size[..., re] = size[..., im] = xd[..., re].abs() + xd[..., im].abs()
    off = abs(first) * 2.0 ** -64 * 2 * math.pi + 2.0 ** -21          # the angle, and fp32's part
    op.assert_within(out, want, 2.0 ** -11 * want.abs() + off * size + 2.0 ** -25, f"position {first}")
