"""The loss over the vocabulary where a word's weights or a token's loss are not finite."""
from __future__ import annotations

import math

import pytest
import torch

from test_vocab_loss import Case, U, gen_of

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


@pytest.fixture(scope="module")
def z():
    import __graft_entry__ as g
    g.build()
    import fsdp_sharded_optimizer_zero_gb300 as z
    yield z
    z.zero_device_status()


@pytest.mark.parametrize("m", [40, 300, 16384, 16385, 20000, 50000])
def test_an_infinite_loss_makes_the_total_infinite(z, m):
    """However many tokens there are: a label with a logit of -inf, anywhere in the batch."""
    w = torch.randn(64, 8, generator=gen_of(m, 1), device=DEV).to(BF)
    w[5, 0] = -math.inf
    x = torch.rand(m, 8, generator=gen_of(m, 2), device=DEV).add(0.5).to(BF)
    labels = torch.full((m,), 3, dtype=torch.int64, device=DEV)
    loss, lse, total = torch.empty(m, device=DEV), torch.empty(m, device=DEV), torch.empty(2, device=DEV)
    for at in (0, m // 2, m - 1):
        labels.fill_(3)
        labels[at] = 5
        z.fsdp_vocab_loss_forward([w], x, labels, loss, lse, total=total)
        rest = torch.arange(m, device=DEV) != at
        assert float(loss[at]) == math.inf and bool(loss[rest].isfinite().all()) and bool(lse.isfinite().all())
        assert total.tolist() == [math.inf, float(m)]
    z.zero_device_status()


@pytest.mark.parametrize("m", [16384, 16385, 20000, 70001])
def test_total_of_many_tokens(z, m):
    """A thread adds several blocks' totals: 5 additions in a warp of tokens, two roundings in a thread that keeps what it rounds
    off, 5 and 15 over the threads."""
    c = Case(m, 500, 504, 72, 1)
    loss, _, total = c.forward(z)
    d = loss.double()
    assert abs(float(total[0]) - float(d.sum())) <= 28 * U * float(d.abs().sum())
    assert float(total[1]) == float(c.real.sum())


@pytest.mark.parametrize("factors", [False, True])
@pytest.mark.parametrize("m,vocab,k,piece", [(200, 60, 72, 0), (20, 60, 72, 0), (200, 5000, 264, 0), (200, 5000, 264, 1024), (20, 5000, 1096, 0)])
def test_padded_tokens_have_no_gradient_beside_words_that_are_not_finite(z, m, vocab, k, piece, factors):
    """dX of a token that is not counted is 0, whatever W holds: in one part and in several, in one piece and in more."""
    rows = (vocab + 7) // 8 * 8
    c = Case(m, vocab, rows, k, 1)
    g = torch.rand(m, generator=gen_of(m, 9), device=DEV) if factors else None
    _, lse, total = c.forward(z)
    want, _ = c.backward(z, lse, 2.0, g, total, piece, dw=False)
    w = c.shards[0]
    w[11, 3], w[vocab // 2, 5], w[vocab - 1, 7] = math.nan, math.inf, -math.inf
    _, lse1, total1 = c.forward(z)
    assert bool((~c.real).any()) and bool(lse1[c.real].isnan().all()) and float(total1[1]) == float(total[1])
    dX, _ = c.backward(z, lse1, 2.0, g, total1, piece, dw=False)
    assert not bool(dX[~c.real].any()) and bool(dX[c.real].isnan().any(1).all())
    # with the finite words' lse the rows of counted tokens are not finite where W is not, and the others' are 0 still
    dX, _ = c.backward(z, lse, 2.0, g, total, piece, dw=False)
    assert not bool(dX[~c.real].any())
