"""The loss over the vocabulary and its gradients against float64 on the GPU, with derived bounds.

SUM bounds the tensor cores' fp32 sums (a term's share per addition), U is half a step of fp32, B16 of
bf16. dZ is rounded to bf16 inside: its bounds are carried through the rounding, so that an element whose
rounding is certain is known exactly."""
from __future__ import annotations

import pytest
import torch

import synth

DEV = "cuda"
BF = torch.bfloat16
SUM, U, B16 = 2.0 ** -23, 2.0 ** -24, 2.0 ** -8

# m, vocab, rows, k, shards: one token, one word, sizes inside a tile, shards cut inside tiles (at multiples
# of 8, 16, 64, 128 rows), a shard that is padding throughout
SHAPES = [(1, 1, 8, 8, 1), (1, 1000, 1000, 72, 1), (5, 129, 144, 64, 2), (130, 255, 256, 136, 1), (256, 256, 256, 256, 1),
          (300, 257, 264, 264, 1), (257, 513, 640, 520, 5), (1003, 1157, 1160, 520, 5), (64, 5000, 5120, 768, 8),
          (700, 2100, 2560, 328, 4), (31, 1400, 2048, 136, 8), (2049, 3000, 3008, 128, 2), (20, 4100, 4224, 1032, 3),
          (520, 640, 640, 2056, 16), (4400, 2900, 2944, 192, 1), (600, 700, 704, 8200, 2), (300, 5000, 5120, 1096, 8),
          (4400, 2900, 2944, 1096, 2),
          # few tokens or few words, and rows long enough for several accumulators
          (7, 3000, 3008, 2056, 1), (33, 2000, 2048, 8200, 2), (64, 5100, 5120, 4104, 8), (32, 1000, 1024, 16392, 1),
          (500, 2000, 2048, 4104, 1), (300, 260, 320, 1288, 5),
          # many long shards cut at multiples of 8 rows
          (300, 5001, 5248, 264, 16), (700, 4900, 4992, 1096, 16), (20, 4000, 4400, 520, 10)]


@pytest.fixture(scope="module")
def z():
    import __graft_entry__ as g
    g.build()
    import fsdp_sharded_optimizer_zero_gb300 as z
    yield z
    if torch.cuda.is_available():
        z.zero_device_status()


def gen_of(*key):
    return torch.Generator(device=DEV).manual_seed(synth.derive_seed(97, *key))


def randn(*shape, std=1.0, key=0):
    return torch.randn(*shape, generator=gen_of(*shape, key), device=DEV) * std


def inside(got, want, bound, what):
    off = (got.double() - want).abs()
    bad = ~(off <= bound)
    assert not bool(bad.any()), (what, int(bad.sum()), float(off[bad].max()), float((off / bound)[bad].max()))


class Case:
    def __init__(self, m, vocab, rows, k, n, dtype=torch.int64, std=2.0, apart=True):
        self.m, self.vocab, self.rows, self.k = m, vocab, rows, k
        self.x = randn(m, k).to(BF)
        w = randn(rows, k, std=std * k ** -0.5, key=1).to(BF)
        w[vocab:] = float("nan")  # padding is never read
        self.shards = [s.clone() if apart else s for s in w.chunk(n)]
        lab = torch.randint(0, vocab, (m,), generator=gen_of(m, vocab, 2), device=DEV)
        r = torch.rand(m, generator=gen_of(m, 3), device=DEV)
        lim = torch.iinfo(dtype)
        lab = torch.where(r < 0.1, -100, torch.where(r > 0.98, lim.max, torch.where(r > 0.96, vocab, lab)))
        lab[0] = vocab - 1
        self.labels = lab.to(dtype)
        self.real = (lab >= 0) & (lab < vocab)
        self.at = torch.where(self.real, lab, 0)
        self.x64, self.w64 = self.x.double(), w[:vocab].double()
        self.z = self.x64 @ self.w64.t()
        self.ez = (k + 1) * SUM * (self.x64.abs() @ self.w64.abs().t())
        # the forward's logits are summed in parts of 1024 products, which are added with rounding to nearest
        ef = (min(k, 1024) + k // 1024 + 1) / (k + 1) * self.ez
        self.lse = torch.logsumexp(self.z, 1)
        # the sum's terms: exponential 2^-21, its argument 2 U of z and of the maximum (up to z's size), then
        # additions: 16 in a thread's two lanes, 4 groups, and the parts, in eight turns and joined; each join
        # scales by an exponential
        parts = -(-vocab // 128)
        top = self.z.abs().amax(1)
        self.e_lse = ef.amax(1) + 4 * U * (top + 1) + (parts / 8 + 16) * 2.0 ** -20 + 4 * U * self.lse.abs()
        self.loss = torch.where(self.real, self.lse - self.z.gather(1, self.at[:, None])[:, 0], 0.0)
        self.e_loss = torch.where(self.real, self.e_lse + ef.gather(1, self.at[:, None])[:, 0] + U * self.loss.abs(), 0.0)

    def forward(self, z, total=True, **kw):
        out = [torch.full((self.m + 16,), 3.0, device=DEV) for _ in range(2)] + [torch.full((4,), 3.0, device=DEV)]
        z.fsdp_vocab_loss_forward(self.shards, self.x, self.labels, out[0][:self.m], out[1][:self.m],
                                  total=out[2][:2] if total else None, vocab=self.vocab, **kw)
        for t, n in zip(out, (self.m, self.m, 2 if total else 0)):
            assert bool((t[n:] == 3.0).all())
        z.zero_device_status()
        return out[0][:self.m], out[1][:self.m], out[2][:2]

    def check_forward(self, z):
        loss, lse, total = self.forward(z)
        inside(lse, self.lse, self.e_lse, "lse")
        inside(loss, self.loss, self.e_loss, "loss")
        assert bool((loss[~self.real] == 0).all())
        assert float(total[1]) == float(self.real.sum())
        # summed with what is rounded off kept, then over the threads
        d = loss.double()
        inside(total[0], d.sum(), 16 * U * d.abs().sum(), "total")
        again = self.forward(z)
        assert all(torch.equal(a, b) for a, b in zip((loss, lse, total), again))
        assert torch.equal(self.forward(z, total=False)[0], loss)
        return loss, lse, total

    def weights(self, dloss):
        w = torch.ones(self.m, dtype=torch.float64, device=DEV) if dloss is None else dloss.double()
        return torch.where(self.real, w, 0.0)

    def backward(self, z, lse, scale=1.0, dloss=None, total=None, piece=0, dx=True, dw=True, **kw):
        dX = torch.full((self.m * self.k + 64,), 3.0, dtype=BF, device=DEV) if dx else None
        dW = torch.full((self.rows * self.k + 64,), 3.0, dtype=BF, device=DEV) if dw else None
        z.fsdp_vocab_loss_backward(self.shards, self.x, self.labels, lse,
                                   dX[:-64].view(self.m, self.k) if dx else None,
                                   dW[:-64].view(self.rows, self.k) if dw else None, vocab=self.vocab, dloss=dloss, total=total,
                                   scale=scale, piece=piece, **kw)
        for t in (dX, dW):
            assert t is None or bool((t[-64:] == 3.0).all())
        z.zero_device_status()
        return dX[:-64].view(self.m, self.k) if dx else None, dW[:-64].view(self.rows, self.k) if dw else None

    def check_backward(self, z, lse, dX, dW, scale, dloss, total, pieces):
        c = torch.tensor(scale, device=DEV) / (1.0 if total is None else total[1].clamp(min=1.0))
        cg = (c * self.weights(dloss).float()).double()[:, None]  # rounded twice, as it is there, and where it multiplies
        p = torch.exp(self.z - lse.double()[:, None])
        hot = torch.zeros_like(p).scatter_(1, self.at[:, None], 1.0) * self.real[:, None]
        dz = (p - hot) * self.real[:, None]
        # z, the argument's roundings (of z, lse and their difference), the exponential
        size = self.z.abs() + lse.double().abs()[:, None] + 1
        e = (p * (self.ez + 4 * U * size + 2.0 ** -20) * 1.1 + 4 * U * hot) * self.real[:, None] + 4 * U * dz.abs()
        lo, hi = ((dz + s * e).float().to(BF).double() for s in (-1.0, 1.0))
        mid, rad = (lo + hi) / 2, (hi - lo) / 2
        want = cg * (mid @ self.w64)
        bound = cg.abs() * (rad @ self.w64.abs() + (self.vocab + 32 + pieces) * SUM * (mid.abs() @ self.w64.abs())) + 3 * U * want.abs()
        if dX is not None:
            inside(dX, want, bound + B16 * (want.abs() + bound), "dX")
            assert not bool(dX[~self.real].any())
        # with factors of the tokens, X times them is rounded to bf16; else c multiplies the sums
        x = self.x64 if dloss is None else (cg.float() * self.x.float()).to(BF).double()
        c = c.double() if dloss is None else torch.ones((), dtype=torch.float64, device=DEV)
        want = c * (mid.t() @ x)
        bound = c.abs() * (rad.t() @ x.abs() + (self.m + 1) * SUM * (mid.abs().t() @ x.abs())) + 3 * U * want.abs()
        if dW is not None:
            inside(dW[:self.vocab], want, bound + B16 * (want.abs() + bound), "dW")
            assert not bool(dW[self.vocab:].any())


@pytest.mark.gpu
@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_forward(z, i):
    Case(*SHAPES[i], dtype=torch.int64 if i % 2 else torch.int32, apart=i % 3 != 0).check_forward(z)


@pytest.mark.gpu
@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_backward(z, i):
    c = Case(*SHAPES[i], dtype=torch.int32 if i % 2 else torch.int64, apart=i % 3 != 0)
    _, lse, total = c.forward(z)
    dloss = torch.rand(c.m, generator=gen_of(c.m, 9), device=DEV)
    for scale, g, t, piece in ((1.0, None, total, 0), (0.5, dloss, None, 256), (3.0, dloss, total, 512)):
        dX, dW = c.backward(z, lse, scale, g, t, piece)
        c.check_backward(z, lse, dX, dW, scale, g, t, -(-c.vocab // (piece or c.vocab)))
        dX1, _ = c.backward(z, lse, scale, g, t, piece, dw=False)
        _, dW1 = c.backward(z, lse, scale, g, t, piece, dx=False)
        assert torch.equal(dX1, dX) and torch.equal(dW1, dW)


@pytest.mark.gpu
@pytest.mark.parametrize("std", [0.02, 30.0, 3000.0])
def test_flat_and_peaked_logits(z, std):
    """From all words alike to one word that takes all, whose exponentials underflow elsewhere."""
    c = Case(300, 1157, 1160, 264, 5, std=std)
    _, lse, total = c.check_forward(z)
    dX, dW = c.backward(z, lse, total=total)
    c.check_backward(z, lse, dX, dW, 1.0, None, total, 1)


@pytest.mark.gpu
@pytest.mark.parametrize("m,vocab", [(20, 300), (300, 5000)])
def test_padded_tokens_may_hold_anything_with_factors(z, m, vocab):
    c = Case(m, vocab, (vocab + 7) // 8 * 8, 264, 1)
    _, lse, total = c.forward(z)
    g = torch.rand(m, generator=gen_of(m, 9), device=DEV)
    dX, dW = c.backward(z, lse, 2.0, g, total)
    c.x[~c.real], g[~c.real] = float("nan"), float("inf")
    loss, lse1, total1 = c.forward(z)
    assert torch.equal(total1, total) and torch.equal(lse1[c.real], lse[c.real]) and not bool(loss[~c.real].any())
    dX1, dW1 = c.backward(z, lse1, 2.0, g, total)
    assert torch.equal(dX1, dX) and torch.equal(dW1, dW) and not bool(dX1[~c.real].any())


@pytest.mark.gpu
@pytest.mark.parametrize("m,k,piece", [(130, 776, 0), (130, 4104, 0), (130, 8200, 256), (20, 4104, 256), (1500, 4104, 512)])
def test_what_is_left_of_sure_tokens_adds_up_to_nothing(z, m, k, piece):
    """The gradients of a token's logits add up to 0. Column 0 of X is 0 and of W 1, so dX's is their sum: small
    where the label's probability is near 1, however large the logits, if the backward's logits are the forward's."""
    vocab = 600 if m < 1000 else 5000
    x = randn(m, k).abs().add(0.5).to(BF)
    w = (1.0 + 0.01 * randn(vocab, k, key=1)) * (26.0 / (1.3 * k))
    w[7] *= 40.0 / 26.0
    w = w.to(BF)
    x[:, 0], w[:, 0] = 0.0, 1.0
    labels = torch.full((m,), 7, dtype=torch.int64, device=DEV)
    loss, lse = torch.empty(m, device=DEV), torch.empty(m, device=DEV)
    dX = torch.empty(m, k, dtype=BF, device=DEV)
    z.fsdp_vocab_loss_forward([w], x, labels, loss, lse)
    z.fsdp_vocab_loss_backward([w], x, labels, lse, dX, None, piece=piece)
    z.zero_device_status()
    logits = x.double() @ w.double().t()
    p = torch.softmax(logits, 1)
    left = 1.0 - p[:, 7]
    assert 1e-5 < float(left.min()) and float(left.max()) < 0.05 and float(logits[:, 7].min()) > 30.0
    # dZ rounded to bf16, the label's and the others'; lse as in Case (without its logits' sums: they are the same
    # here), then the argument's roundings and the exponential's; dX's sum
    top, parts = logits.amax(1), -(-vocab // 128)
    e = 4 * U * (top + 1) + (parts / 8 + 16) * 2.0 ** -20 + 4 * U * top + 4 * U * (2 * top + 1) + 2.0 ** -20
    bound = B16 * 2 * left + e + (vocab + 32) * SUM * 2 * left
    inside(dX[:, 0], torch.zeros_like(top), bound * (1 + B16), "the sum of dZ")


@pytest.mark.gpu
def test_no_token_counts(z):
    c = Case(200, 600, 640, 136, 2)
    c.labels.fill_(-100)
    c.x[5] = float("inf")  # no logits to speak of, in a row that is not counted
    loss, lse, total = c.forward(z)
    assert not bool(loss.any()) and total.tolist() == [0.0, 0.0]
    c.x[5] = 0
    dX, dW = c.backward(z, lse, total=total)
    assert not bool(dX.any()) and not bool(dW.any())


@pytest.mark.gpu
def test_rows_that_are_not_finite(z):
    """A token whose logits are NaN or infinite: its own loss and dX alone; not counted, nothing at all."""
    c = Case(300, 1157, 1160, 136, 1)
    c.labels[7], c.labels[8], c.labels[9] = 5, 6, -100
    want = c.forward(z)
    rows = torch.ones(300, dtype=torch.bool, device=DEV)
    rows[7:10] = False
    c.x[7, 3], c.x[8, 4], c.x[9, 5] = float("nan"), float("inf"), float("nan")
    loss, lse, _ = c.forward(z)
    assert torch.equal(loss[rows], want[0][rows]) and torch.equal(lse[rows], want[1][rows])
    assert bool(loss[7].isnan()) and not bool(loss[8].isfinite()) and float(loss[9]) == 0.0
    dX, _ = c.backward(z, lse, dw=False)
    assert bool(dX[rows].isfinite().all()) and not bool(dX[9].any()) and not bool(dX[7].isfinite().any())


@pytest.mark.gpu
def test_mean_loss_against_differences(z):
    """The mean loss in float64 along directions of X and W: central differences."""
    c = Case(257, 700, 704, 136, 4)
    _, lse, total = c.forward(z)
    dX, dW = c.backward(z, lse, total=total)
    h = 1e-4

    def loss(x, w):
        t = x @ w.t()
        each = torch.logsumexp(t, 1) - t.gather(1, c.at[:, None])[:, 0]
        return float(each[c.real].mean())

    v, u = randn(c.m, c.k, key=5).double(), randn(c.vocab, c.k, key=6).double()
    # dZ and the result rounded to bf16, whose errors add up like independent ones at most in full
    slope = (loss(c.x64 + h * v, c.w64) - loss(c.x64 - h * v, c.w64)) / (2 * h)
    dz = (torch.exp(c.z - c.lse[:, None]) * c.real[:, None] / c.real.sum()).scatter_add(
        1, c.at[:, None], -(c.real / c.real.sum())[:, None].double())
    size = float((dz.abs() * (v @ c.w64.t()).abs()).sum()) + float((dX.double() * v).abs().sum())
    assert abs(slope - float((dX.double() * v).sum())) <= 1.1 * B16 * size + 1e-6
    slope = (loss(c.x64, c.w64 + h * u) - loss(c.x64, c.w64 - h * u)) / (2 * h)
    size = float((dz.abs() * (c.x64 @ u.t()).abs()).sum()) + float((dW[:c.vocab].double() * u).abs().sum())
    assert abs(slope - float((dW[:c.vocab].double() * u).sum())) <= 1.1 * B16 * size + 1e-6


@pytest.mark.gpu
def test_streams_and_graphs(z):
    """On another stream than the current one; two captured steps that share a workspace, replayed with other
    inputs."""
    c = Case(600, 1157, 1160, 264, 5)
    want = c.forward(z)
    grads = c.backward(z, want[1], total=want[2], piece=512)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = c.forward(z, stream=side)
        g2 = c.backward(z, got[1], total=got[2], piece=512, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((*want, *grads), (*got, *g2)))
    nbytes = max(z.fsdp_vocab_loss_forward_workspace(c.m, c.vocab), z.fsdp_vocab_loss_backward_workspace(c.m, c.vocab, c.k, 512))
    ws = torch.empty(nbytes, dtype=torch.uint8, device=DEV)
    x2 = randn(c.m, c.k, key=8).to(BF)
    outs, graphs = [], []
    for x in (c.x, x2):
        o = [torch.empty(c.m, device=DEV), torch.empty(c.m, device=DEV), torch.empty(2, device=DEV),
             torch.empty(c.m, c.k, dtype=BF, device=DEV), torch.empty(c.rows, c.k, dtype=BF, device=DEV)]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            z.fsdp_vocab_loss_forward(c.shards, x, c.labels, o[0], o[1], total=o[2], vocab=c.vocab, workspace=ws)
            z.fsdp_vocab_loss_backward(c.shards, x, c.labels, o[1], o[3], o[4], vocab=c.vocab, total=o[2], piece=512, workspace=ws)
        outs.append(o)
        graphs.append(graph)
    c.x.copy_(randn(c.m, c.k, key=10).to(BF))
    for g in (*graphs, *graphs):
        g.replay()
    for x, o in ((c.x, outs[0]), (x2, outs[1])):
        c.x = x
        want = c.forward(z)
        grads = c.backward(z, want[1], total=want[2], piece=512)
        assert all(torch.equal(a, b) for a, b in zip((*want, *grads), o))


@pytest.mark.gpu
def test_many_tiles_of_a_pair(z):
    """More tiles than pairs of SMs, several rounds, at the 768-wide model's vocabulary: against float64 in
    slices of the rows."""
    m, vocab, k = 1500, 50257, 72
    c = Case(m, vocab, 50304, k, 8)
    _, lse, total = c.check_forward(z)
    for piece in (0, 16384):
        dX, dW = c.backward(z, lse, total=total, piece=piece)
        c.check_backward(z, lse, dX, dW, 1.0, None, total, 4)
