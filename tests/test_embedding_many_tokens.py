"""The embedding's gradient of so many tokens that the sort's counts are added up by a launch of their own (more than
64 blocks of 2048), and where the offsets of sorted rows and of the table pass 2^31."""
from __future__ import annotations

import pytest
import torch

from test_embedding import BF, DEV, U, check_backward, gen_of, tokens_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def z():
    import __graft_entry__ as g
    g.build()
    import fsdp_sharded_optimizer_zero_gb300 as z
    yield z
    z.zero_device_status()
    torch.cuda.empty_cache()


@pytest.mark.parametrize("kind", ["uniform", "one", "text", "falling", "none"])
@pytest.mark.parametrize("m", [131072, 131073, 300001])  # 64 blocks, the first 65, many
@pytest.mark.parametrize("vocab", [400, 50257, 300007])  # one pass, two, three
def test_counts_added_up_by_one_block(z, m, vocab, kind):
    rows = (vocab + 7) // 8 * 8
    check_backward(z, m, vocab, rows, 8, kind, torch.int64, True)
    check_backward(z, m, vocab, rows, 8, kind, torch.int32, False, scale=2.5)
    check_backward(z, m, vocab, rows, 8, kind, torch.int64, True, add=True)


def test_wide_rows(z):
    """Several warps to a row beside the scan."""
    check_backward(z, 140001, 1000, 1000, 520, "text", torch.int64, True)
    check_backward(z, 140001, 1000, 1000, 520, "uniform", torch.int32, False, add=True)


def test_offsets_past_2_31(z):
    """Both dY and dE of 2.2e9 elements, sorted: all rows, in some columns."""
    m, vocab, rows, cols = 270001, 269900, 270000, 8200
    t = tokens_of("text", m, vocab, torch.int64)
    t[-3:] = vocab - 1
    dy = torch.empty(m, cols, dtype=BF, device=DEV).normal_(generator=gen_of(1))
    de = torch.empty(rows, cols, device=DEV)
    z.fsdp_embedding_backward(dy, t, de, vocab=vocab)
    z.zero_device_status()
    real = (t >= 0) & (t < vocab)
    at = t[real]
    count = torch.bincount(at, minlength=rows).double()[:, None]
    pick = torch.tensor([0, 7, 255, 256, 4095, 8191, 8192, 8199], device=DEV)
    g = dy[:, pick][real].double()
    want = torch.zeros(rows, pick.numel(), dtype=torch.float64, device=DEV).index_add_(0, at, g)
    mag = torch.zeros_like(want).index_add_(0, at, g.abs())
    assert bool(((de[:, pick].double() - want).abs() <= (count + 2) * U * mag * 1.01).all())
    unused = count[:, 0] == 0
    assert int(unused.sum()) > 1000
    assert sum(int(de[a:a + 8192][unused[a:a + 8192]].count_nonzero()) for a in range(0, rows, 8192)) == 0
