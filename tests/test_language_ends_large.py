"""Embedding, layer norm and the loss over the vocabulary where an element's offset passes 2^31 and 2^32:
sampled against float64."""
from __future__ import annotations

import pytest
import torch

from test_layernorm import backward64, forward64, inside
from test_vocab_loss import B16, SUM, U

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
    torch.cuda.empty_cache()


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def test_layernorm(z):
    rows, cols = 264000, 16384  # 4.3e9 elements
    x = torch.empty(rows, cols, dtype=BF, device=DEV).normal_(generator=gen(1))
    y, mean, rstd = torch.empty_like(x), torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    z.fsdp_layernorm_forward(x, y, mean=mean, rstd=rstd)
    pick = torch.tensor([0, 1, 131071, 131072, 131073, 262143, 262144, rows - 2, rows - 1], device=DEV)
    m64, r64, y64, em, er, ey = forward64(x[pick], None, None, 1e-5)
    inside(mean[pick], m64, em + U * m64.abs(), "mean")
    inside(rstd[pick], r64, er, "rstd")
    inside(y[pick], y64, ey + B16 * (y64.abs() + ey), "Y")
    dg, db = torch.empty(cols, device=DEV), torch.empty(cols, device=DEV)
    dy = y  # any gradient will do
    want = backward64(dy[pick], x[pick], mean[pick], rstd[pick], None, None)
    sums = torch.zeros(cols, dtype=torch.float64, device=DEV)
    size = torch.zeros_like(sums)
    for a in range(0, rows, 8192):
        part = dy[a:a + 8192].double()
        sums += part.sum(0)
        size += part.abs().sum(0)
    z.fsdp_layernorm_backward(dy, x, mean, rstd, dy, dgamma=dg, dbeta=db)  # in place
    inside(dy[pick], want[0], want[1] + B16 * (want[0].abs() + want[1]), "dX")
    inside(db, sums, (rows / 100) * U * size, "dbeta")  # a block adds at most rows / 152 of them, then the blocks


def test_embedding(z):
    rows, cols = 70000, 65536  # 4.6e9 elements
    t = torch.tensor([rows - 1, 0, 32768, 65535, 65536, 65537, rows - 1, -100, rows], device=DEV)
    table = torch.empty(rows, cols, dtype=BF, device=DEV).normal_(generator=gen(2))
    y = torch.empty(t.numel(), cols, dtype=BF, device=DEV)
    z.fsdp_embedding_forward([table], t, y)
    assert torch.equal(y[:7], table[t[:7]]) and not bool(y[7:].any())
    de = table  # overwritten: every row
    z.fsdp_embedding_backward(y, t, de)
    assert torch.equal(de[rows - 1].float(), (2.0 * y[0].float()).to(BF).float())
    for i in (1, 2, 3, 4, 5):
        assert torch.equal(de[t[i]], y[i])
    used = torch.zeros(rows, dtype=torch.bool, device=DEV)
    used[t[:7]] = True
    rest = [int(de[a:a + 4096][~used[a:a + 4096]].count_nonzero()) for a in range(0, rows, 4096)]
    assert sum(rest) == 0


def test_vocab_loss(z):
    m, vocab, k = 20000, 131000, 64  # dZ of one piece: 2.6e9 elements
    x = torch.randn(m, k, generator=gen(3), device=DEV).to(BF)
    w = (torch.randn(131072, k, generator=gen(4), device=DEV) * 0.2).to(BF)
    w[vocab:] = float("nan")
    labels = torch.randint(0, vocab, (m,), generator=gen(5), device=DEV)
    loss, lse, total = torch.empty(m, device=DEV), torch.empty(m, device=DEV), torch.empty(2, device=DEV)
    z.fsdp_vocab_loss_forward([w], x, labels, loss, lse, total=total, vocab=vocab)
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    z.fsdp_vocab_loss_backward([w], x, labels, lse, dx, dw, vocab=vocab, piece=131072)
    z.zero_device_status()
    x64, w64 = x.double(), w[:vocab].double()
    pick = torch.tensor([0, 255, 8191, 16383, 16384, 16385, m - 1], device=DEV)
    t = x64[pick] @ w64.t()
    ez = (k + 1) * SUM * (x64[pick].abs() @ w64.abs().t())
    want = torch.logsumexp(t, 1)
    e = ez.amax(1) + 4 * U * (t.abs().amax(1) + 1) + 144 * 2.0 ** -20 + 4 * U * want.abs()
    inside(lse[pick], want, e, "lse")
    at = labels[pick]
    dz = torch.exp(t - lse[pick].double()[:, None])
    dz[torch.arange(7, device=DEV), at] -= 1.0
    # each term: its rounding to bf16, and before that the error of the exponential and of the logit (p is dz, but for
    # the label), then sums of vocab products
    hot = torch.zeros_like(dz)
    hot[torch.arange(7, device=DEV), at] = 1.0
    p = dz + hot
    off = p * (ez + 4 * U * (t.abs() + lse[pick].double().abs()[:, None] + 1) + 2.0 ** -20) * 1.1 + 4 * U * hot
    want = dz @ w64
    bound = (off + B16 * (dz.abs() + off)) @ w64.abs() + vocab * SUM * (dz.abs() @ w64.abs())
    inside(dx[pick], want, bound + B16 * want.abs(), "dX")
    cols = torch.tensor([0, 1, 65535, 65536, 107374, 107375, vocab - 2, vocab - 1], device=DEV)
    t = x64 @ w64[cols].t()
    dz = torch.exp(t - lse.double()[:, None]) - (labels[:, None] == cols[None]).double()
    hot = (labels[:, None] == cols[None]).double()
    ez = (k + 1) * SUM * (x64.abs() @ w64[cols].abs().t())
    off = (dz + hot) * (ez + 4 * U * (t.abs() + lse.double().abs()[:, None] + 1) + 2.0 ** -20) * 1.1 + 4 * U * hot
    want = dz.t() @ x64
    bound = (off + B16 * (dz.abs() + off)).t() @ x64.abs() + m * SUM * (dz.abs().t() @ x64.abs())
    inside(dw[cols], want, bound + B16 * want.abs(), "dW")
    assert not bool(dw[vocab:].any())
