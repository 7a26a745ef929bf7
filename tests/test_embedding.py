"""Token embedding and its gradient against float64 on the GPU, with derived bounds: U is half a step of
fp32, B16 of bf16."""
from __future__ import annotations

import pytest
import torch

import synth

DEV = "cuda"
BF = torch.bfloat16
U, B16 = 2.0 ** -24, 2.0 ** -8


@pytest.fixture(scope="module")
def z():
    import __graft_entry__ as g
    g.build()
    import fsdp_sharded_optimizer_zero_gb300 as z
    yield z
    if torch.cuda.is_available():
        z.zero_device_status()


def gen_of(*key):
    return torch.Generator(device=DEV).manual_seed(synth.derive_seed(96, *key))


def randn(*shape, std=1.0, key=0):
    return torch.randn(*shape, generator=gen_of(*shape, key), device=DEV) * std


def tokens_of(kind, m, vocab, dtype):
    gen = gen_of(m, vocab, 3)
    if kind == "uniform":
        t = torch.randint(0, vocab, (m,), generator=gen, device=DEV)
    elif kind == "one":  # every token the same
        t = torch.full((m,), vocab // 2, device=DEV)
    elif kind == "text":  # few tokens often, most seldom
        u = torch.rand(m, generator=gen, device=DEV, dtype=torch.float64)
        t = ((vocab + 1.0) ** u).long().sub(1).clamp(0, vocab - 1)
    elif kind == "falling":
        t = torch.arange(m - 1, -1, -1, device=DEV) * vocab // m
    else:  # "none": padding and ids past the vocabulary only
        t = torch.where(torch.rand(m, generator=gen, device=DEV) < 0.5, -100, vocab)
    if kind in ("uniform", "text"):  # some of each, and the type's lowest and highest value
        r = torch.rand(m, generator=gen, device=DEV)
        t = torch.where(r < 0.05, -100, torch.where(r < 0.08, vocab, t))
        lim = torch.iinfo(dtype)
        t = torch.where(r > 0.995, lim.max, torch.where(r > 0.99, lim.min, t))
    return t.to(dtype)


def guarded(*shape, dtype):
    n = shape[0] * shape[1]
    flat = torch.full((n + 64,), 3.0, dtype=dtype, device=DEV)
    flat[:n] = float("nan")
    return flat[:n].view(*shape), lambda: bool((flat[n:] == 3.0).all())


@pytest.mark.gpu
@pytest.mark.parametrize("m,vocab,rows,cols,n", [(1, 1, 8, 8, 1), (1, 50257, 50264, 768, 1), (37, 100, 120, 264, 5),
                                                 (1000, 1157, 1160, 1032, 5), (300, 33, 48, 4104, 16),
                                                 (9000, 500, 512, 40, 8), (3, 70000, 70000, 2048, 2)])
@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
def test_forward(z, m, vocab, rows, cols, n, dtype):
    table = randn(rows, cols).to(BF)
    table[vocab:] = float("nan")  # padding is never read
    shards = [s.clone() for s in table.chunk(n)]
    t = tokens_of("text", m, vocab, dtype)
    real = (t >= 0) & (t < vocab)
    want = table[torch.where(real, t, 0).long()].double()
    for scale in (1.0, cols ** 0.5):
        y, ok = guarded(m, cols, dtype=BF)
        z.fsdp_embedding_forward(shards, t, y, vocab=vocab, scale=scale)
        w = torch.where(real[:, None], want * scale, 0.0)
        assert ok() and bool(((y.double() - w).abs() <= (B16 + 2 * U) * w.abs()).all())  # scale to fp32, product, bf16
        if scale == 1.0:
            assert torch.equal(y.double(), w)


def check_backward(z, m, vocab, rows, cols, kind, dtype, wide, scale=1.0, add=False):
    t = tokens_of(kind, m, vocab, dtype)
    dy = randn(m, cols, key=1).to(BF)
    real = (t >= 0) & (t < vocab)
    at, g = t[real].long(), dy[real].double()
    want = torch.zeros(rows, cols, dtype=torch.float64, device=DEV).index_add_(0, at, g) * scale
    mag = torch.zeros(rows, cols, dtype=torch.float64, device=DEV).index_add_(0, at, g.abs()) * abs(scale)
    count = torch.zeros(rows, dtype=torch.float64, device=DEV).index_add_(0, at, torch.ones_like(at, dtype=torch.float64))
    de, ok = guarded(rows, cols, dtype=torch.float32 if wide else BF)
    old = randn(rows, cols, key=2).to(de.dtype)
    if add:
        de.copy_(old)
        want = want + old.double()
    z.fsdp_embedding_backward(dy, t, de, vocab=vocab, scale=scale, accumulate=add)
    # a sum passes through at most as many additions as it has terms; scale, product and the joining sum
    e = ((count + 2)[:, None] * U * mag + (U * want.abs() if add else 0.0)) * 1.01
    if not wide:
        e = e + B16 * (want.abs() + e)
    off = (de.double() - want).abs()
    assert ok() and bool((off <= e).all()), float((off - e).max())
    untouched = count == 0
    assert torch.equal(de[untouched], old[untouched] if add else torch.zeros_like(de[untouched]))
    again = old.clone() if add else torch.full_like(de, float("nan"))
    z.fsdp_embedding_backward(dy, t, again, vocab=vocab, scale=scale, accumulate=add)
    assert torch.equal(again, de)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["uniform", "one", "text", "falling", "none"])
@pytest.mark.parametrize("m,vocab,rows,cols", [(1, 1, 8, 8), (31, 5, 8, 264), (32, 40, 40, 256), (33, 3, 16, 520), (64, 2, 8, 8),
                                               (65, 1000, 1008, 768), (1003, 1157, 1160, 520), (2048, 60, 64, 1032),
                                               (4096, 3000, 3008, 264), (4097, 90, 96, 520), (8192, 3000, 3008, 264),
                                               (16384, 700, 704, 40), (700, 1200000, 1200000, 8)])
def test_backward(z, m, vocab, rows, cols, kind):
    check_backward(z, m, vocab, rows, cols, kind, torch.int64, True)
    check_backward(z, m, vocab, rows, cols, kind, torch.int32, False, scale=cols ** 0.5)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["uniform", "one", "text", "falling", "none"])
@pytest.mark.parametrize("m,vocab,rows,cols", [(16385, 50257, 50264, 64), (20000, 1, 8, 264), (40961, 300, 304, 264),
                                               (70001, 600, 600, 520), (33000, 300000, 300000, 8)])
def test_backward_sorted_in_passes(z, m, vocab, rows, cols, kind):
    """Tokens that take one, two and three passes of the sort."""
    check_backward(z, m, vocab, rows, cols, kind, torch.int32, True)
    check_backward(z, m, vocab, rows, cols, kind, torch.int64, False)


@pytest.mark.gpu
@pytest.mark.parametrize("wide", [True, False])
def test_backward_stretches_of_every_length(z, wide):
    """Tokens that come 1, 2, .. 40 runs of 16 positions often, each with every offset in its run and among the
    runs, added to a gradient: none is summed twice or left out."""
    for pad in (0, 1, 15, 16, 100, 255, 256, 257):
        lengths = [16 * n + d for n in (1, 2, 15, 16, 17, 31, 32, 33, 34, 40, 48) for d in (-1, 0, 1)]
        t = torch.cat([torch.full((pad,), 0, device=DEV)]
                      + [torch.full((n,), 1 + i, device=DEV) for i, n in enumerate(lengths)]).long()
        rows, cols = len(lengths) + 9, 8
        dy = torch.ones(t.numel(), cols, dtype=BF, device=DEV)
        de = torch.full((rows, cols), 1.0, dtype=torch.float32 if wide else BF, device=DEV)
        z.fsdp_embedding_backward(dy, t, de, accumulate=True)
        want = torch.bincount(t, minlength=rows).double() + 1.0
        assert torch.equal(de[:, 0].double(), want if wide else want.to(BF).double())
        assert torch.equal(de, de[:, :1].expand(-1, cols))


@pytest.mark.gpu
@pytest.mark.parametrize("m,vocab,rows,cols,kind", [(1003, 1157, 1160, 520, "text"), (20000, 50, 56, 264, "text"), (7, 9, 16, 8, "none")])
def test_backward_added_to_a_gradient(z, m, vocab, rows, cols, kind):
    check_backward(z, m, vocab, rows, cols, kind, torch.int64, True, scale=3.0, add=True)
    check_backward(z, m, vocab, rows, cols, kind, torch.int64, False, scale=3.0, add=True)


@pytest.mark.gpu
def test_gradient_against_differences(z):
    """L = sum G . Y is linear in the table: its difference along a direction is exact."""
    m, vocab, cols = 500, 60, 264
    t = tokens_of("text", m, vocab, torch.int64)
    g, v = randn(m, cols, key=4).to(BF), randn(vocab + 4, cols, key=5).to(BF)
    de, y = torch.empty(vocab + 4, cols, device=DEV), torch.empty(m, cols, dtype=BF, device=DEV)
    z.fsdp_embedding_backward(g, t, de, vocab=vocab, scale=2.0)
    z.fsdp_embedding_forward([v], t, y, vocab=vocab, scale=2.0)  # a power of two: exact
    slope, size = (g.double() * y.double()).sum(), (g.double() * y.double()).abs().sum()
    assert abs(float(slope - (de.double() * v.double()).sum())) <= m * U * float(size)


@pytest.mark.gpu
def test_infinities_stay_with_their_tokens(z):
    """A NaN row of dY under a padded token reaches nothing; under a token, that row alone."""
    t = torch.tensor([3, -100, 5, 3, 7], device=DEV)
    dy = randn(5, 264).to(BF)
    dy[1] = float("nan")
    de = torch.empty(8, 264, device=DEV)
    z.fsdp_embedding_backward(dy, t, de)
    assert bool(de.isfinite().all())
    dy[2] = float("inf")
    z.fsdp_embedding_backward(dy, t, de)
    assert [i for i in range(8) if not bool(de[i].isfinite().all())] == [5]


@pytest.mark.gpu
@pytest.mark.parametrize("m", [700, 6000, 20000])
def test_streams_and_graph(z, m):
    """Another stream than the current one; captured and replayed with other tokens; two graphs that share a
    workspace, one after the other."""
    vocab, cols = 300, 520
    dy, t = randn(m, cols).to(BF), tokens_of("text", m, vocab, torch.int64)
    want, got = torch.empty(304, cols, device=DEV), torch.empty(304, cols, device=DEV)
    z.fsdp_embedding_backward(dy, t, want, vocab=vocab)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    z.fsdp_embedding_backward(dy, t, got, vocab=vocab, stream=side)
    side.synchronize()
    assert torch.equal(want, got)
    ws = torch.empty(z.fsdp_embedding_backward_workspace(m, vocab, cols), dtype=torch.uint8, device=DEV)
    t2, outs, graphs = tokens_of("uniform", m, vocab, torch.int64), [], []
    for tok in (t, t2):
        outs.append(torch.empty(304, cols, device=DEV))
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            z.fsdp_embedding_backward(dy, tok, outs[-1], vocab=vocab, workspace=ws)
    t.copy_(tokens_of("falling", m, vocab, torch.int64))
    for g in (*graphs, *graphs):
        g.replay()
    for tok, out in zip((t, t2), outs):
        z.fsdp_embedding_backward(dy, tok, want, vocab=vocab)
        assert torch.equal(want, out)
