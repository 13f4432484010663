"""Rotary embedding and its fusion with the cache write, against 64 bits."""
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


def _gen(dev, seed):
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    return g


def _bound(x, y, pairs_abs, u):
    """u |y| for the rounding, and fp32's part: each product and the cosine (sincospif is within
    2 ulp, its argument within 1/2 ulp of at most pi) are off by at most 2^-21 of |re| + |im|."""
    return u * y.abs() + 2.0 ** -21 * pairs_abs + 2.0 ** -25   # 2^-25: half of fp16's least step


def _pairs_abs(x, half, interleaved, factor):
    y = x.double().abs()
    j = torch.arange(half, device=x.device)
    re, im = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
    out = torch.zeros_like(y)
    s = (y[..., re] + y[..., im]) * abs(factor)
    out[..., re], out[..., im] = s, s
    return out


POS = {"near": 0, "far": 1_000_003, "farthest": (1 << 31) - 300}


@pytest.mark.parametrize("interleaved", [False, True], ids=["halves", "pairs"])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=["fp16", "bf16"])
@pytest.mark.parametrize("T,H,D,rot", [(1, 1, 64, 16), (3, 5, 128, 128), (257, 32, 128, 96), (40, 3, 64, 64),
                                       (2000, 2, 64, 48)])
def test_embed_matches_64_bits(dev, T, H, D, rot, dtype, interleaved):
    import paged_kv_cache_252_gb300 as pkv
    g = _gen(dev, T + rot)
    inv, _ = pkv.rotary_inv_freq(rot, 10000.0, device=dev)
    x = torch.randn((T, H, D), generator=g, device=dev).to(dtype)
    for name, first in POS.items():
        pos = torch.arange(first, first + T, device=dev, dtype=torch.int64)
        if name == "near":
            pos = pos.to(torch.int32)
        out = torch.full_like(x, float("nan"))
        pkv.rotary_embed(out, x, pos, inv, interleaved=interleaved, attn_factor=1.25)
        want = op.turn(x, pos, inv, interleaved, 1.25)
        pa = _pairs_abs(x, rot // 2, interleaved, 1.25)
        # the 64-bit reference's own angle is rounded to 2^-53 of up to 2^31 rad
        op.assert_within(out, want, _bound(x, want, pa, op.HALF_STEP[dtype]) + pa * 2.0 ** -21, f"{name} {T}x{H}x{D}/{rot}")
        assert torch.equal(out[..., rot:], x[..., rot:])


def test_embed_in_place_strided_rows_negative_positions_and_inverse(dev):
    import paged_kv_cache_252_gb300 as pkv
    g = _gen(dev, 5)
    T, H, D = 33, 4, 128
    inv, _ = pkv.rotary_inv_freq(D, 500000.0, device=dev)
    wide = torch.randn((T, H * D + 64), generator=g, device=dev).half()
    x = wide[:, 8:8 + H * D].view(T, H, D)          # rows 64 elements apart, 16 bytes in
    before = wide.clone()
    pos = torch.arange(-T, 0, device=dev)
    out = torch.empty((T, H, D), dtype=torch.float16, device=dev)
    pkv.rotary_embed(out, x, pos, inv)
    op.assert_within(out, op.turn(x, pos, inv, False),
                     _bound(x, op.turn(x, pos, inv, False), _pairs_abs(x, D // 2, False, 1.0), 2.0 ** -11), "strided")
    pkv.rotary_embed(x, x, pos, inv)                # in place
    assert torch.equal(x, out)
    assert torch.equal(wide[:, :8], before[:, :8]) and torch.equal(wide[:, 8 + H * D:], before[:, 8 + H * D:])
    back = torch.empty_like(out)
    pkv.rotary_embed(back, out, pos, inv, inverse=True)
    x0 = before[:, 8:8 + H * D].reshape(T, H, D)
    pa = _pairs_abs(x0, D // 2, False, 1.0)
    # two roundings to fp16, the first turned with the row
    op.assert_within(back, x0.double(), 2.0 ** -11 * (x0.double().abs() + 1.5 * pa) + 2.0 ** -20 * pa + 2.0 ** -24, "back")


@pytest.mark.parametrize("interleaved", [False, True], ids=["halves", "pairs"])
def test_inverse_is_the_gradient(dev, interleaved):
    """<turn(x), w> = <x, turn_inverse(w)>: in 64 bits against autograd and against differences."""
    import paged_kv_cache_252_gb300 as pkv
    g = _gen(dev, 9)
    T, H, D, rot = 7, 2, 64, 32
    inv, _ = pkv.rotary_inv_freq(rot, device=dev)
    pos = torch.randint(0, 1 << 17, (T,), generator=g, device=dev)
    x = torch.randn((T, H, D), generator=g, device=dev).half()
    w = torch.randn((T, H, D), generator=g, device=dev).half()
    grad = torch.empty_like(w)
    pkv.rotary_embed(grad, w, pos, inv, interleaved=interleaved, attn_factor=1.5, inverse=True)
    half = rot // 2
    ang = pos.double()[:, None] * inv
    c, s = (ang.cos() * 1.5)[:, None], (ang.sin() * 1.5)[:, None]
    xd = x.double().requires_grad_()

    def f(v):
        re, im = (v[..., 0:rot:2], v[..., 1:rot:2]) if interleaved else (v[..., :half], v[..., half:rot])
        a, b = re * c - im * s, re * s + im * c
        y = torch.stack((a, b), -1).flatten(-2) if interleaved else torch.cat((a, b), -1)
        return (torch.cat((y, v[..., rot:]), -1) * w.double()).sum()
    f(xd).backward()
    pa = _pairs_abs(w, half, interleaved, 1.5)
    op.assert_within(grad, xd.grad, _bound(w, xd.grad, pa, 2.0 ** -11), "autograd")
    d = torch.randn(x.shape, generator=g, device=dev, dtype=torch.float64)
    slope = (f(x.double() + 1e-3 * d) - f(x.double() - 1e-3 * d)) / 2e-3
    got = (grad.double() * d).sum()
    assert abs(got - slope) <= ((2.0 ** -11 * xd.grad.abs() + 2.0 ** -20 * pa + 2.0 ** -25) * d.abs()).sum() + 1e-6


def _write_case(dev, kv, T, hq, hkv, D, seed, packed=True):
    g = _gen(dev, seed)
    blocks = -(-T // 16) + 2
    kc, vc, sc = op.make_cache(kv, blocks, hkv, D, g, dev)
    dt = op.src_dtype(kv)
    qkv = torch.randn((T, (hq + 2 * hkv) * D), generator=g, device=dev).to(dt)
    q = qkv[:, :hq * D].view(T, hq, D)
    key = qkv[:, hq * D:(hq + hkv) * D].view(T, hkv, D)
    value = qkv[:, (hq + hkv) * D:].view(T, hkv, D)
    if not packed:
        q, key, value = q.contiguous(), key.contiguous(), value.contiguous()
    slots = torch.randperm(blocks * 16, generator=g, device=dev)[:T].to(torch.int32)
    return q, key, value, slots, kc, vc, sc


@pytest.mark.parametrize("packed", [True, False], ids=["packed", "apart"])
@pytest.mark.parametrize("kv", ["fp16", "bf16", "e5m2", "int8"])
@pytest.mark.parametrize("T,hq,hkv,D,rot,inter", [(1, 4, 2, 64, 64, False), (64, 32, 8, 128, 128, True),
                                                  (513, 6, 2, 64, 16, False), (1500, 8, 1, 128, 64, True)])
def test_write_matches_64_bits(dev, kv, T, hq, hkv, D, rot, inter, packed):
    import paged_kv_cache_252_gb300 as pkv
    q, key, value, slots, kc, vc, sc = _write_case(dev, kv, T, hq, hkv, D, 100 + T, packed)
    slots[5::7] = -1                                         # padding: query turned, nothing written
    k0, v0, s0 = kc.clone(), vc.clone(), None if sc is None else sc.clone()
    inv, f = pkv.rotary_inv_freq(rot, 10000.0, scaling="ramp", factor=4.0, original_context=4096, device=dev)
    pos = torch.arange(4090, 4090 + T, device=dev)
    q_out = torch.full((T, hq, D), float("nan"), dtype=q.dtype, device=dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    pkv.rotary_write(q_out, q, key, value, pos, slots, kc, vc, inv, interleaved=inter, attn_factor=f, scales=sc,
                     device_status=status)
    assert status.item() == 0
    u = op.HALF_STEP[q.dtype]
    wq, wk = op.turn(q, pos, inv, inter, f), op.turn(key, pos, inv, inter, f)
    op.assert_within(q_out, wq, _bound(q, wq, _pairs_abs(q, rot // 2, inter, f), u), "q")
    used = slots >= 0
    at = slots[used].long()
    pk = _pairs_abs(key, rot // 2, inter, f)[used]
    wk, wv = wk[used], value[used].double()

    def rows(c):
        return c.transpose(1, 2).reshape(-1, hkv, D)
    if kv == "int8":
        got_k, got_v = (rows(op.cache_rows(c, sc, w))[at] for w, c in enumerate((kc, vc)))
        for got, want, which, fp in ((got_k, wk, 0, pk), (got_v, wv, 1, torch.zeros_like(wv))):
            scale = sc[:, :, which].transpose(1, 2).reshape(-1, hkv)[at].double()[..., None]
            amax = want.abs().amax(-1, keepdim=True)
            # max / 127 rounded up to fp16 (at most 2^-10 more, 2^-24 where subnormal); a code is half a scale off
            err = fp.amax(-1, keepdim=True) * 2.0 ** -21
            assert ((scale >= (amax - err) / 127 * (1 - 2.0 ** -23)) &
                    (scale <= (amax + err) / 127 * (1 + 2.0 ** -9) + 2.0 ** -24)).all()
            assert ((got - want).abs() <= 0.5 * scale * (1 + 2.0 ** -20) + 2.0 ** -21 * fp).all()
    else:
        uk = op.HALF_STEP[torch.float8_e5m2] if kv == "e5m2" else u
        tiny = 2.0 ** -17 if kv == "e5m2" else 2.0 ** -25    # half of the type's least step
        op.assert_within(rows(op.cache_rows(kc))[at], wk, _bound(key, wk, pk, uk) + tiny, "k")
    # values, and every row no token maps to, exactly as the plain cache write leaves them
    k1, v1, s1 = k0.clone(), v0.clone(), None if s0 is None else s0.clone()
    if kv == "int8":
        pkv.kv_cache_write_int8(key.contiguous(), value.contiguous(), slots, k1, v1, s1)
        assert torch.equal(s1[:, :, 1], sc[:, :, 1])
    else:
        pkv.kv_cache_write(key.contiguous(), value.contiguous(), slots, k1, v1)
    assert torch.equal(v1, vc)
    rest = torch.ones(kc.shape[0] * 16, dtype=torch.bool, device=dev)
    rest[at] = False
    assert torch.equal(rows(kc)[rest], rows(k0)[rest])


@pytest.mark.parametrize("inter", [False, True], ids=["halves", "pairs"])
@pytest.mark.parametrize("scaling", [None, "ramp"])
def test_e5m2_keys_are_the_nearest_to_the_64_bit_value(dev, inter, scaling):
    """8.4 million keys, of which fp32 would place several on the wrong side of a rounding border: codes
    equal those of the 64-bit value (its own error, 2^-53 of an angle of 2e4 rad, reaches a border
    in fewer than one of 10^9)."""
    import paged_kv_cache_252_gb300 as pkv
    T, hkv, D = 8192, 8, 128
    q, key, value, slots, kc, vc, _ = _write_case(dev, "e5m2", T, 1, hkv, D, 77)
    inv, f = pkv.rotary_inv_freq(D, 10000.0, scaling=scaling, factor=4.0, original_context=4096, device=dev)
    pos = torch.arange(16384, 16384 + T, device=dev, dtype=torch.int32)
    pkv.rotary_write(torch.empty_like(q, memory_format=torch.contiguous_format), q, key, value, pos, slots, kc, vc, inv,
                     interleaved=inter, attn_factor=f)
    want = op.turn(key, pos, inv, inter, f)
    # nearest E5M2 value: two fraction bits, steps of 2^-16 below 2^-14, at most 57344
    step = torch.exp2(torch.frexp(want)[1].double().sub(3).clamp(min=-16))
    want = (want / step).round().mul(step).clamp(-57344, 57344)
    got = op.cache_rows(kc).transpose(1, 2).reshape(-1, hkv, D)[slots.long()]
    assert int((got != want).sum()) == 0


@pytest.mark.parametrize("kv", ["e5m2", "int8"])
def test_zero_angle_writes_what_the_cache_write_writes(dev, kv):
    """At position 0 nothing turns: bit for bit the plain cache write, extreme values included."""
    import paged_kv_cache_252_gb300 as pkv
    q, key, value, slots, kc, vc, sc = _write_case(dev, kv, 40, 4, 2, 128, 3, packed=False)
    key[0, 0, :9] = torch.tensor([0.0, -0.0, 65504.0, -65504.0, 57344.0, 61440.0, 6e-8, -1e-5, 1.0], device=dev)
    key[1] = 0.0
    if kv == "e5m2":
        key[2, 0, :64] = torch.linspace(-3e-5, 3e-5, 64, device=dev)
    inv, _ = pkv.rotary_inv_freq(128, device=dev)
    k1, v1, s1 = kc.clone(), vc.clone(), None if sc is None else sc.clone()
    pkv.rotary_write(torch.empty_like(q), q, key, value, torch.zeros(40, dtype=torch.int32, device=dev), slots, kc, vc,
                     inv, scales=sc)
    if kv == "int8":
        pkv.kv_cache_write_int8(key, value, slots, k1, v1, s1)
        assert torch.equal(s1, sc)
    else:
        pkv.kv_cache_write(key, value, slots, k1, v1)
    keep = lambda c: c.view(torch.uint8) & 0x7F if kv == "e5m2" else c   # 0 * sin may turn -0 into 0
    nz = k1.view(torch.uint8) & 0x7F != 0 if kv == "e5m2" else None
    assert torch.equal(keep(kc), keep(k1)) and torch.equal(vc, v1)
    if kv == "e5m2":
        assert torch.equal(kc[nz], k1[nz])


def test_not_a_number_is_the_caches_nan(dev):
    import paged_kv_cache_252_gb300 as pkv
    q, key, value, slots, kc, vc, _ = _write_case(dev, "e5m2", 4, 2, 1, 64, 8, packed=False)
    key[2, 0, 3] = float("nan")
    inv, _ = pkv.rotary_inv_freq(64, device=dev)
    pkv.rotary_write(torch.empty_like(q), q, key, value, torch.arange(4, device=dev), slots, kc, vc, inv)
    row = kc.transpose(1, 2).reshape(-1, 64)[slots[2].long()]
    nan = (row & 0x7F) > 0x7C
    assert nan.nonzero().flatten().tolist() == [3, 35] and ((row[nan] & 0x7F) == 0x7E).all()


def test_bad_slots_are_skipped_and_flagged(dev):
    import paged_kv_cache_252_gb300 as pkv
    q, key, value, slots, kc, vc, _ = _write_case(dev, "fp16", 20, 2, 2, 64, 4, packed=False)
    k0, v0 = kc.clone(), vc.clone()
    slots[:] = -1
    slots[3], slots[4] = kc.shape[0] * 16, -2
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    inv, _ = pkv.rotary_inv_freq(32, device=dev)
    pkv.rotary_write(torch.empty_like(q), q, key, value, torch.arange(20, device=dev), slots, kc, vc, inv,
                     device_status=status)
    assert status.item() == 1 and torch.equal(kc, k0) and torch.equal(vc, v0)


def test_replays_from_a_graph_on_another_stream(dev):
    import paged_kv_cache_252_gb300 as pkv
    q, key, value, slots, kc, vc, _ = _write_case(dev, "bf16", 30, 4, 2, 128, 6)
    inv, _ = pkv.rotary_inv_freq(128, device=dev)
    pos = torch.arange(30, device=dev)
    q_out, want = torch.empty((30, 4, 128), dtype=q.dtype, device=dev), torch.empty((30, 4, 128), dtype=q.dtype, device=dev)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        pkv.rotary_write(q_out, q, key, value, pos, slots, kc, vc, inv)
    for first in (7, 90000):
        pos.copy_(torch.arange(first, first + 30, device=dev))
        graph.replay()
        k1, v1 = kc.clone(), vc.clone()
        pkv.rotary_write(want, q, key, value, pos, slots, k1, v1, inv)
        assert torch.equal(q_out, want) and torch.equal(kc, k1) and torch.equal(vc, v1)


def test_no_tokens_is_a_no_op(dev):
    import paged_kv_cache_252_gb300 as pkv
    inv, _ = pkv.rotary_inv_freq(64, device=dev)
    x = torch.empty((0, 2, 64), dtype=torch.float16, device=dev)
    pkv.rotary_embed(torch.empty_like(x), x, torch.empty(0, dtype=torch.int32, device=dev), inv)
