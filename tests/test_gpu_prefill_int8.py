"""Prefill over INT8 caches whose V scales are small, or differ widely, against 64 bits."""
import pytest
import torch

import _bounds
import _operators as op
from test_gpu_prefill import Batch, dev  # noqa: F401

pytestmark = pytest.mark.gpu


def _sink(dev, D, n, ctx, nats, v_scale):
    """Rows that give position 0, whose value is zero, `nats` more than each of the others."""
    b = Batch(dev, "int8", D, 2, 1, [n], [ctx])
    b.kc.fill_(-128)                      # code 0
    blk = int(b.bt[0, 0])
    b.kc[blk, :, 0] = 100 - 128
    b.vc[blk, :, 0] = -128
    b.sc[:, :, 0] = 0.0099945068359375    # an fp16 number
    b.q.fill_(nats / (D ** 0.5 * 100 * 0.0099945068359375))
    b.sc[:, :, 1] = torch.tensor(v_scale).half().float()
    b.vc[..., 0] = 127 - 128              # a dimension where nothing cancels
    b.vc[..., 1] = 1 - 128
    b.vc[blk, :, 0] = -128
    return b


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("nats,ctx", [(9.0, 4096), (11.0, 8192), (4.0, 700), (0.0, 300)])
@pytest.mark.parametrize("largest", [0.0025, 0.02, 0.127, 1.0, 60000.0])
def test_long_flat_tails_behind_a_sink(dev, D, nats, ctx, largest):  # noqa: F811
    """Weights far below the sink's keep their bits whatever the values' size (their largest is given)."""
    b = _sink(dev, D, 3, ctx, nats, largest / 127)
    b.run()
    _bounds.check_rows(b, f"{largest} {nats}")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("where", ["unseen", "weightless", "last", "every"])
def test_widely_differing_scales(dev, D, where):  # noqa: F811
    """V scales of 500 beside 1e-5: in later tokens of the chunk, at positions of no weight, in
    the last tile, in every tile at positions of no weight."""
    n, ctx = 40, 900
    b = Batch(dev, "int8", D, 2, 1, [n], [ctx], q_gain=0.3)
    b.sc[:, :, 1] = torch.tensor(1e-5).half().float()
    b.sc[:, :, 0] = 0.0099945068359375
    b.q.abs_()
    at = {"unseen": range(ctx - 8, ctx), "weightless": [3, 70], "last": [ctx - n - 1],
          "every": range(5, ctx - n, 128)}[where]
    for p in at:
        blk = int(b.bt[0, p // 16])
        b.sc[blk, :, 1, p % 16] = 500.0
        if where in ("weightless", "every"):
            b.kc[blk, :, p % 16] = -127 - 128 + 256     # code -127 ...
            b.sc[blk, :, 0, p % 16] = 4.0               # ... scaled so that its score is far below the others'
    b.run()
    _bounds.check_rows(b, where)


@pytest.mark.parametrize("D", [64, 128])
def test_rising_products_move_the_maximum(dev, D):  # noqa: F811
    """Scores and V scales that grow along the context, so that the maximum moves in every tile."""
    b = Batch(dev, "int8", D, 2, 1, [20], [3000])
    ids = b.bt[0].long()
    ramp = torch.linspace(0.0, 1.0, ids.numel() * 16, device=dev).view(-1, 1, 16)
    b.kc.fill_(100 - 128)
    b.sc[ids, :, 0] = (ramp * 0.02 + 1e-4).half().float()
    b.sc[ids, :, 1] = torch.exp2(ramp * 20 - 16).half().float()
    b.q.copy_(torch.where(torch.arange(20, device=dev)[:, None, None] % 2 == 0, 0.5, -0.5).expand_as(b.q))
    b.run()
    _bounds.check_rows(b, "rising")


@pytest.mark.parametrize("v_scale", [0.0, 2.0 ** -24, 1e-30, 2000.0])
def test_scales_outside_the_codecs_range(dev, v_scale):  # noqa: F811
    """Scales a user may set himself: zero, the least fp16 number, less, and more than fp16 rows give."""
    b = Batch(dev, "int8", 128, 2, 1, [5], [400], q_gain=6.0)
    b.sc[:, :, 1] = v_scale
    b.run()
    at, want, tol = _bounds.attention_rows(b, 0)
    fits = want.abs() < 65000
    g = b.out[at].double()
    assert ((g - want).abs() <= tol)[fits].all() and not torch.isnan(g).any()
    assert (g[want.abs() > 66000].abs() == float("inf")).all()
    assert torch.equal(g.sign()[~fits], want.sign()[~fits])


@pytest.mark.parametrize("D", [64, 128])
def test_negative_scales(dev, D):  # noqa: F811
    """V scales of either sign: right, and no slower for it (sums that leave fp16 would send every row through
    the plain row pass, some 100 times as long)."""
    from test_gpu_prefill_nonfinite import _time
    b = Batch(dev, "int8", D, 8, 2, [600], [2600], q_gain=2.0)
    plain = _time(b)
    b.sc[:, :, 1, ::3] *= -300.0
    b.sc[:, :, 1, 1::3] *= -1.0
    t = _time(b)
    print(f"{plain * 1e3:.0f} us, {t * 1e3:.0f} us with negative scales")
    at, want, tol = _bounds.attention_rows(b, 0, [0, 1, 63, 64, 300, 598, 599])
    op.assert_within(b.out[at], want, tol, "negative scales")
    assert t < 4 * plain + 0.02
