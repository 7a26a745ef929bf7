"""fp32 weight gradients of more 256 x 256 tiles than the GPU has CTA pairs, so that every pair stores
several tiles from the same staging buffers, with right edges of every number of 32-column blocks, odd
and even: against float64 on the GPU, and the same bits call after call.

Bounds: a sum of n terms is within (n + 1) 2^-23 of the sum of magnitudes (any order, rounding toward
zero included); results over more than 4096 tokens are sums of parts of at most 4096, one more rounding
each; the scale is one more rounding of the result."""
from __future__ import annotations

import pytest
import torch

from test_linear_unit_wide import SUM, inside, kept, new8, randn, guarded, values, z  # noqa: F401

pytestmark = pytest.mark.gpu
DEV = "cuda"


def check(z, m, r, k, bits8, scale=0.25):  # noqa: F811
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert -(-r // 256) * -(-k // 256) > sms // 2  # a pair takes a second tile
    g, x = randn(m, r, 0.3, 21), randn(m, k, 1.0, 22)
    if bits8:
        c = new8(m, k)
        z.fsdp_checkpoint8_pack(x, *c)
        arg, v = {"x8": c}, values(z, c)
    else:
        arg, v = {"x": x}, x.double()
    buf, dw = guarded(r, k, torch.float32, 3.0)
    z.fsdp_linear_dw(g, dw, scale=scale, **arg)
    want, mag = scale * (g.double().T @ v), scale * (g.double().abs().T @ v.abs())
    inside(dw, want, (min(m, 4096) + 1 + m // 4096) * SUM * mag + SUM * want.abs(), "dW")
    assert kept(buf, 3.0)
    again = torch.empty_like(dw)
    for _ in range(4):
        again.fill_(float("nan"))
        z.fsdp_linear_dw(g, again, scale=scale, **arg)
        assert torch.equal(again, dw)
    z.zero_device_status()


# live 32-column blocks of the last tile column: 4104 one, 1080 two, 4184 three, 1144 four, 1160 and 1440
# five, 1208 six, 4312 seven, 1280 eight
@pytest.mark.parametrize("bits8", [False, True])
@pytest.mark.parametrize("m", [1, 65, 4097])
@pytest.mark.parametrize("k", [1160, 1440])
def test_right_edges_of_five_blocks(z, m, k, bits8):  # noqa: F811
    check(z, m, 14336, k, bits8)


@pytest.mark.parametrize("m", [8, 300])
@pytest.mark.parametrize("k", [1080, 1144, 1208, 1280, 4104, 4184, 4312])
def test_right_edges_of_every_number_of_blocks(z, m, k):  # noqa: F811
    check(z, m, 5128, k, m == 300)


# outputs of one tile column, which is the right edge of every tile: an odd number of blocks each time
@pytest.mark.parametrize("k", [8, 72, 136, 200])
def test_every_tile_at_the_right_edge(z, k):  # noqa: F811
    check(z, 40, 256 * 400 + 8, k, False)
