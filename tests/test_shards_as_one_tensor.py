"""Row shards given as one [n, rows, cols] tensor instead of a list: the linear unit's calls take them as
fsdp_unit_forward and fsdp_gather_rows do."""
from __future__ import annotations

import pytest
import torch

BF = torch.bfloat16


@pytest.fixture(scope="module")
def z():
    import __graft_entry__ as g
    g.build()
    import fsdp_sharded_optimizer_zero_gb300 as z
    return z


@pytest.mark.parametrize("n", [1, 2, 16])
def test_refused_for_its_device_alone(z, n):
    """Host tensors: the argument is looked at as shards, and refused as host memory."""
    w, x, y = torch.zeros(n, 8, 16, dtype=BF), torch.zeros(4, 16, dtype=BF), torch.zeros(4, 8 * n, dtype=BF)
    for call in (lambda: z.fsdp_unit_forward(w, x, y.float()), lambda: z.fsdp_linear_forward(w, x, y),
                 lambda: z.fsdp_linear_dx(w, y, x)):
        with pytest.raises(ValueError, match="must be a CUDA tensor"):
            call()


@pytest.mark.parametrize("empty", [[], (), torch.zeros(0, 8, 16, dtype=BF)])
def test_no_shards(z, empty):
    x = torch.zeros(4, 16, dtype=BF)
    with pytest.raises(ValueError, match="w_shards is empty"):
        z.fsdp_linear_forward(empty, x, x)
    with pytest.raises(ValueError, match="w_shards is empty"):
        z.fsdp_linear_dx(empty, x, x)


@pytest.mark.gpu
@pytest.mark.parametrize("m,r,k,n", [(5, 240, 136, 5), (300, 1160, 264, 1), (700, 4608, 264, 16)])
def test_same_bits_as_a_list(z, m, r, k, n):
    gen = torch.Generator(device="cuda").manual_seed(m)
    w = torch.randn(n, r // n, k, generator=gen, device="cuda").to(BF)
    x, dz = torch.randn(m, k, generator=gen, device="cuda").to(BF), torch.randn(m, r, generator=gen, device="cuda").to(BF)
    out = []
    for shards in (w, list(w.unbind())):
        y, dx = torch.empty_like(dz), torch.empty_like(x)
        z.fsdp_linear_forward(shards, x, y)
        z.fsdp_linear_dx(shards, dz, dx)
        out.append((y, dx))
    z.zero_device_status()
    assert torch.equal(out[0][0], out[1][0]) and torch.equal(out[0][1], out[1][1])
