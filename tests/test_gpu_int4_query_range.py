"""INT4 decode with queries of bf16's whole range."""
import pytest
import torch

import _int4 as i4
from test_gpu_int4_attention import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("exponent", [-119, -116, -101, 60, 99, 100, 101, 104, 105, 106, 112, 114, 115, 120, 126])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("g,n", [(4, 1), (8, 1), (4, 4), (8, 4), (8, 8)])
def test_queries_of_the_whole_range(g, n, d, exponent):
    """Scaled back by `scale`: 2^exponent times a power of two leaves the bits of queries of size 1."""
    c = Case([max(n, x) for x in (3, 40, 300)], 2 * g, 2, d, torch.bfloat16, n=n, seed=g + n)
    c.q = c.q.clamp(-1.9, 1.9)
    small = c.q.double().abs() < 2.0 ** -6     # (bf16 holds the rest at its lower end)
    c.q[small] = 0
    i4.assert_within(c.fixed(), *c.want())
    c.scale = 1.0
    ordinary = c.fixed()
    c.q = (c.q.double() * 2.0 ** exponent).to(torch.bfloat16)
    c.scale = 2.0 ** -exponent
    assert torch.equal(c.fixed(), ordinary)
