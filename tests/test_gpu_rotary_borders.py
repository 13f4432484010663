"""E5M2 keys chosen to lie beside the rounding borders of their type."""
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


def _beside_borders(pos, inv, factor, lo, hi, g, tries):
    """fp16 pairs [T, half, 2] whose turned real part lies lo to hi units of 2^-24 factor (|re| + |im|) from
    the middle between two E5M2 values (pairs for which no try did: zeros)."""
    ang = pos.double()[:, None] * inv
    c, s = ang.cos(), ang.sin()
    best = torch.zeros(ang.shape + (2,), dtype=torch.float16, device=pos.device)
    for _ in range(tries):
        x = torch.randn(ang.shape + (2,), generator=g, device=pos.device).half()
        re, im = x[..., 0].double(), x[..., 1].double()
        y = factor * (re * c - im * s)
        m, e = torch.frexp(y.abs())                       # m in [1/2, 1): E5M2 values are multiples of 1/8
        away = ((m * 8).frac() - 0.5).abs() * torch.exp2(e.double() - 3)
        units = away / (2.0 ** -24 * factor * (re.abs() + im.abs()))
        ok = (units >= lo) & (units <= hi) & (e > -13)
        best = torch.where(ok[..., None], x, best)
    return best


@pytest.mark.parametrize("inter", [False, True], ids=["halves", "pairs"])
@pytest.mark.parametrize("factor", [1.0, 1.1386294361119891])
@pytest.mark.parametrize("lo,hi", [(0.0, 3.0), (3.0, 9.0)])
def test_keys_beside_borders_round_to_the_nearest(dev, inter, factor, lo, hi):
    import paged_kv_cache_252_gb300 as pkv
    T, D = 1024, 128
    g = torch.Generator(device=dev)
    g.manual_seed(6)
    inv, _ = pkv.rotary_inv_freq(D, 10000.0, device=dev)
    pos = torch.arange(16384, 16384 + T, device=dev, dtype=torch.int32)
    # a pair lies in a band of one unit some 5 times in 10^6 tries
    x = _beside_borders(pos, inv, factor, lo, hi, g, 4000)
    found = (x != 0).any(-1).double().mean().item()
    print(f"{lo} to {hi} units from a border: {found:.3f} of the pairs")
    assert found > 0.02
    key = x.reshape(T, 1, D) if inter else torch.cat((x[..., 0], x[..., 1]), -1)[:, None].contiguous()
    kc = torch.zeros((T // 16, 1, 16, D), dtype=torch.uint8, device=dev)
    q = torch.zeros_like(key)
    pkv.rotary_write(torch.empty_like(q), q, key, key.clone(), pos, torch.arange(T, device=dev, dtype=torch.int32), kc,
                     kc.clone(), inv, interleaved=inter, attn_factor=factor)
    want = op.turn(key, pos, inv, inter, factor)
    step = torch.exp2(torch.frexp(want)[1].double().sub(3).clamp(min=-16))
    want = (want / step).round().mul(step).clamp(-57344, 57344)
    got = op.cache_rows(kc).transpose(1, 2).reshape(T, 1, D)
    assert int((got != want).sum()) == 0
