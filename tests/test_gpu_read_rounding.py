"""The roundings of kv_cache_read, to the bit: INT8 values, and INT4 values read as bf16, to fp32 and then to the output's type; INT4
values read as fp16 once."""
import math

import pytest
import torch

import paged_kv_cache_252_gb300 as pkv
import _int4 as i4

pytestmark = pytest.mark.gpu
DEV = "cuda"
BITS = {torch.float16: (11, -24, 65504.0), torch.bfloat16: (8, -133, 255.0 * 2.0 ** 120),
        torch.float32: (24, -149, (2.0 ** 24 - 1) * 2.0 ** 104)}


def nearest(x, dtype):
    """x (64 bits) rounded to the type's numbers, halfway to the even one, beyond the largest by half a step to infinity."""
    bits, least, most = BITS[dtype]
    step = torch.exp2((torch.frexp(x)[1].double() - bits).clamp(min=least))
    y = torch.round(x / step) * step
    return torch.where(y.abs() > most, torch.copysign(torch.full_like(y, math.inf), y), y)


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _read(kv, kc, vc, sc, out):
    nb, hkv, _, d = kc.shape
    d *= 2 if kv == "int4" else 1
    slots = torch.arange(nb * 16, device=DEV, dtype=torch.int32)
    k, v = (torch.full((nb * 16, hkv, d), 7.0, dtype=out, device=DEV) for _ in range(2))
    pkv.kv_cache_read(k, v, slots, kc, vc, kv, scales=sc)
    return [x.view(nb, 16, hkv, d).transpose(1, 2).double() for x in (k, v)]


@pytest.mark.parametrize("out", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("size", [0.01, 2.0 ** -22, 700.0, 2.0 ** -140, 2.0 ** 121])
def test_int8(out, d, size):
    """Scales of 24 bits: the fp32 product lies on a border of fp16 about once in 2^13 elements, where one rounding might have gone
    the other way. Sizes down to where fp16 (2^-22), bf16 and fp32 (2^-140) are subnormal, and beyond the types' ranges."""
    g = _gen(d)
    nb, hkv = 512, 4
    codes = [torch.randint(-127, 128, (nb, hkv, 16, d), generator=g, device=DEV, dtype=torch.int16) for _ in range(2)]
    kc, vc = ((c - 128).to(torch.int8) for c in codes)
    sc = (torch.rand((nb, hkv, 2, 16), generator=g, device=DEV) + 0.5) * size
    for which, got in enumerate(_read("int8", kc, vc, sc, out)):
        want = nearest(nearest(codes[which].double() * sc[:, :, which, :, None].double(), torch.float32), out)
        assert torch.equal(got, want), f"{int((got != want).sum())} of {want.numel()}"


@pytest.mark.parametrize("out", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("sign", [1, -1])
def test_int4(out, d, sign):
    """Least values halfway between two bf16 (or on an fp16) number, and scales so small that fp32 drops
    z + s c's last bits; and least values and scales of every size."""
    g = _gen(d + 1)
    nb, hkv = 256, 4
    kc, vc = (torch.randint(0, 256, (nb, hkv, 16, d // 2), generator=g, device=DEV, dtype=torch.uint8) for _ in range(2))
    sc = torch.zeros((nb, hkv, 2, 16, d // 64, 2), dtype=torch.float16, device=DEV)
    shape = sc.shape[:-1]
    odd = 2 * torch.randint(128, 256, shape, generator=g, device=DEV) + 1          # 9 bits
    z = odd * torch.exp2(torch.randint(-12, 7, shape, generator=g, device=DEV).float())
    s = torch.exp2(torch.randint(-24, -10, shape, generator=g, device=DEV).float()) * torch.randint(1, 8, shape, generator=g, device=DEV)
    sc[..., 0], sc[..., 1] = s.half(), (sign * z).half()
    wild = torch.randint(0, 0x7BFF, (nb // 2, *shape[1:]), generator=g, device=DEV, dtype=torch.int16).view(torch.float16)
    sc[nb // 2:, ..., 0] = wild.clamp(max=8000)
    sc[nb // 2:, ..., 1] = sign * wild.flip(0)
    for which, got in enumerate(_read("int4", kc, vc, sc, out)):
        cache = (kc, vc)[which]
        exact = i4.stand_for(i4.unpack(cache), sc[:, :, which, ..., 0], sc[:, :, which, ..., 1])[0]
        want = nearest(exact if out == torch.float16 else nearest(exact, torch.float32), out)
        assert torch.equal(got, want), f"{int((got != want).sum())} of {want.numel()}"
