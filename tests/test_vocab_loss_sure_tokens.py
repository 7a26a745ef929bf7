"""Losses and gradients of tokens whose label has nearly all of the probability. X is 0 but for its first column, so each
logit is one product of two bf16 values, exact in fp32, and the losses' last digits are the softmax's own.

U is half a step of fp32, B16 of bf16, EX the relative error of ex2.approx."""
from __future__ import annotations

import pytest
import torch

import synth

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16
U, B16, EX, SUM = 2.0 ** -24, 2.0 ** -8, 2.0 ** -22, 2.0 ** -23
WORD = 7  # the label of most tokens: its logits are the largest
# m, vocab, k: both kernels, their contraction in one part and in several, one token, one tile
SHAPES = [(1, 1000, 72), (5, 300, 8), (20, 4000, 1096), (300, 5000, 72), (300, 5000, 1096), (1500, 9001, 264)]


@pytest.fixture(scope="module")
def z():
    import __graft_entry__ as g
    g.build()
    import fsdp_sharded_optimizer_zero_gb300 as z
    yield z
    z.zero_device_status()


class Sure:
    def __init__(self, z, m, vocab, k):
        gen = torch.Generator(device=DEV).manual_seed(synth.derive_seed(98, m, vocab, k))
        self.m, self.vocab = m, vocab
        a = torch.exp2(-7 * torch.rand(m, generator=gen, device=DEV))  # 2^-7 .. 1: from torn to sure
        a[0] = 1.0
        self.x = torch.zeros(m, k, dtype=BF, device=DEV)
        self.x[:, 0] = a
        b = torch.rand(vocab, generator=gen, device=DEV) * 80 - 20
        b[WORD] = 96.0
        self.w = torch.randn(vocab, k, generator=gen, device=DEV).to(BF)
        self.w[:, 0] = b
        rows = (vocab + 7) // 8 * 8
        self.shard = torch.zeros(rows, k, dtype=BF, device=DEV)
        self.shard[:vocab] = self.w
        self.labels = torch.where(torch.arange(m, device=DEV) % 4 == 3, torch.randint(0, vocab, (m,), generator=gen, device=DEV), WORD)
        self.z = self.x[:, :1].double() * self.w[:, 0].double()  # exact
        self.loss, self.lse, self.total = torch.empty(m, device=DEV), torch.empty(m, device=DEV), torch.empty(2, device=DEV)
        z.fsdp_vocab_loss_forward([self.shard], self.x, self.labels, self.loss, self.lse, total=self.total, vocab=vocab)
        z.zero_device_status()


@pytest.mark.parametrize("shape", SHAPES)
def test_losses(z, shape):
    c = Sure(z, *shape)
    top = c.z.amax(1)
    d = top[:, None] - c.z
    e = torch.exp(-d)
    tail = e.sum(1) - 1.0  # the largest is one word's alone
    of_label = top - c.z.gather(1, c.labels[:, None])[:, 0]
    log = torch.log1p(tail)
    want = of_label + log
    # a term: its argument is a difference and a product by a rounded log2 e, taken apart in up to as many steps as there are
    # joins (whose differences add up to d), an exponential each; additions: 16 of a thread, 4 groups, parts in turns
    # of 8 and joined. The largest term is exactly 1 throughout, and what is far below it changes no sum
    parts = -(-c.vocab // 128)
    each = (e * 4 * U * d).sum(1) + tail * (6 + parts / 128) * (EX + U)
    adds = torch.where(tail < 2.0 ** -30, 0.0, (40 + parts / 16) * U * (1 + tail))
    off = (each + adds) / (1 + tail) + 2 * EX * log + 2 * U * want
    got = c.loss.double()
    assert bool((got >= 0).all()), float(got.min())
    bad = (got - want).abs() - off - tail * (tail < 2.0 ** -30)
    assert bool((bad <= 0).all()), float(bad.max())
    sure = (tail < 2.0 ** -30) & (c.labels == WORD)
    assert bool(sure[0]) and not bool(c.loss[sure].any())
    lse = top + log
    assert bool(((c.lse.double() - lse).abs() <= off + U * lse.abs() + 2.0 ** -30).all())


@pytest.mark.parametrize("piece", [0, 256])
@pytest.mark.parametrize("shape", SHAPES)
def test_gradients(z, shape, piece):
    """dX's first column, the sum of dZ times W's first."""
    c = Sure(z, *shape)
    dX = torch.empty_like(c.x)
    z.fsdp_vocab_loss_backward([c.shard], c.x, c.labels, c.lse, dX, None, vocab=c.vocab, piece=piece)
    z.zero_device_status()
    d = c.z - c.lse.double()[:, None]
    p = torch.exp(d)
    hot = torch.zeros_like(p).scatter_(1, c.labels[:, None], 1.0)
    dz, w = p - hot, c.w[:, 0].double()
    # the argument's difference, product and rounded log2 e, the exponential, the label's subtraction, then bf16; fp32 sums
    e = p * (4 * U * d.abs() + EX) + U * dz.abs() * hot
    e = e + B16 * (dz.abs() + e)
    want = dz @ w
    bound = e @ w.abs() + (c.vocab + 32) * SUM * (dz.abs() @ w.abs())
    off = (dX[:, 0].double() - want).abs()
    bad = off - bound - B16 * (want.abs() + bound)
    assert bool((bad <= 0).all()), (float(bad.max()), int((bad > 0).sum()))
