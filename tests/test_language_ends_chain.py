"""Embedding, norms, linear units and the loss over the vocabulary run together, as the example does: each
result against float64 on the GPU's own inputs to it, captured in a graph, on two streams at once."""
from __future__ import annotations

import pytest
import torch

from test_layernorm import backward64, forward64, inside, rows_depth
from test_vocab_loss import Case

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16
U, B16, SUM = 2.0 ** -24, 2.0 ** -8, 2.0 ** -23


@pytest.fixture(scope="module")
def z():
    import __graft_entry__ as g
    g.build()
    import fsdp_sharded_optimizer_zero_gb300 as z
    yield z
    z.zero_device_status()


@pytest.fixture(scope="module")
def ex(z):
    from fsdp_sharded_optimizer_zero_gb300 import example_language as ex
    return ex


def loss_case(model, p, x, labels):
    """test_vocab_loss's reference on these tensors."""
    c = Case.__new__(Case)
    w = torch.cat(p["e"])
    c.m, c.vocab, c.rows, c.k = x.shape[0], model.vocab, w.shape[0], model.d
    c.x, c.shards, c.labels = x, p["e"], labels
    c.real = (labels >= 0) & (labels < c.vocab)
    c.at = torch.where(c.real, labels, 0)
    c.x64, c.w64 = x.double(), w[:c.vocab].double()
    c.z = c.x64 @ c.w64.t()
    c.ez = (c.k + 1) * SUM * (c.x64.abs() @ c.w64.abs().t())
    return c


def one_step(ex, model, p, s, r):
    ex.forward(model, p, *s["batches"][r], s["bufs"][r])
    ex.backward(model, p, *s["batches"][r], model.views(s["grads"][r][:model.psi]), s["bufs"][r])


@pytest.mark.parametrize("m,sizes", [(384, {}), (77, dict(vocab=517, d=136, f=264, shards=1)), (1, dict(vocab=64, d=64, f=128, shards=2))])
def test_each_result_of_a_step(z, ex, m, sizes):
    model = ex.Model(**sizes)
    s = ex.setup(model, 1, m, DEV, seed=3)
    p, b = model.params(s["param"][:model.psi]), s["bufs"][0]
    g = model.views(s["grads"][0][:model.psi])
    tokens, labels = s["batches"][0]
    one_step(ex, model, p, s, 0)
    z.zero_device_status()
    real = tokens >= 0
    table = torch.cat(p["e"])
    assert torch.equal(b["x0"], torch.where(real[:, None], table[torch.where(real, tokens, 0)], torch.zeros((), dtype=BF, device=DEV)))
    for x, y, stat, ga, be in (("x0", "h1", "stat1", "g1", "c1"), ("x1", "h2", "stat2", "g2", "c2")):
        m64, r64, y64, em, er, ey = forward64(b[x], p[ga], p[be], ex.EPS)
        inside(b[stat][0], m64, em + U * m64.abs(), "mean")
        # padding's rows of zeros have no variance: rstd is eps^-1/2 and the bound that divides by it exact
        inside(b[stat][1], r64, er, "rstd")
        inside(b[y], y64, ey + B16 * (y64.abs() + ey), y)
    c = loss_case(model, p, b["h2"], labels)
    lse = torch.logsumexp(c.z, 1)
    e = c.ez.amax(1) + 4 * U * (c.z.abs().amax(1) + 1) + 32 * 2.0 ** -20 + 4 * U * lse.abs()
    inside(b["lse"], lse, e, "lse")
    each = torch.where(c.real, lse - c.z.gather(1, c.at[:, None])[:, 0], 0.0)
    inside(b["loss"], each, e + c.ez.amax(1) + U * each.abs(), "loss")
    assert float(b["total"][1]) == float(c.real.sum())
    c.check_backward(z, b["lse"], b["dh2"], None, 1.0, None, b["total"], 1)
    for dy, x, stat, ga, res, dx, dgamma, dbeta in (("dh2", "x1", "stat2", "g2", None, "dx1", 0, 1),
                                                    ("dh1", "x0", "stat1", "g1", "dx1", "dx0", 3, 4)):
        dx64, e, dg64, dga, db64, dba = backward64(b[dy], b[x], b[stat][0], b[stat][1], p[ga], b[res] if res else None)
        inside(b[dx], dx64, e + B16 * (dx64.abs() + e), dx)
        inside(b["small"][dgamma], dg64, (rows_depth(m) + 4) * U * dga, ga)
        inside(b["small"][dbeta], db64, rows_depth(m) * U * dba, "dbeta")
    # the table's gradient: as the output layer (one call's own dW, in bf16), and the embedding's on top
    head = torch.empty_like(g["e"])
    z.fsdp_vocab_loss_backward(p["e"], b["h2"], labels, b["lse"], None, head, vocab=model.vocab, total=b["total"])
    c.check_backward(z, b["lse"], None, head, 1.0, None, b["total"], 1)
    at, d = tokens[real], b["dx0"][real].double()
    want = head.double().index_add(0, at, d)
    mag = torch.zeros_like(want).index_add_(0, at, d.abs())
    count = torch.bincount(at, minlength=want.shape[0]).double()[:, None]
    e = (count + 2) * U * mag + U * want.abs()
    assert bool(((g["e"].double() - want).abs() <= e + B16 * (want.abs() + e)).all())
    untouched = count[:, 0] == 0
    assert torch.equal(g["e"][untouched], head[untouched]) and not bool(g["e"][model.vocab:].any())


def test_gradients_against_differences(z, ex):
    """The mean loss of the whole model in float64 along one direction of all parameters: a central difference against
    the gradients. Both passes round activations and gradients to bf16 between calls: eight roundings on the way
    from a parameter to the loss and back, each at most B16 of what it rounds."""
    model = ex.Model(vocab=203, d=64, f=128, shards=1)
    s = ex.setup(model, 1, 200, DEV, seed=5)
    p = model.params(s["param"][:model.psi])
    one_step(ex, model, p, s, 0)
    tokens, labels = s["batches"][0]
    real = tokens >= 0
    base = {k: v.double() for k, v in model.views(s["param"][:model.psi]).items()}
    grads = model.views(s["grads"][0][:model.psi])
    gen = torch.Generator(device=DEV).manual_seed(1)
    dirs = {k: torch.randn(v.shape, generator=gen, device=DEV, dtype=torch.float64) * v.std() if v.dim() == 2 else
            torch.randn(v.shape, generator=gen, device=DEV, dtype=torch.float64) * 0.1 for k, v in base.items()}
    dirs["e"][model.vocab:] = 0

    def norm(x, g, c):
        d = x - x.mean(1, keepdim=True)
        return d * (d.square().mean(1, keepdim=True) + ex.EPS).rsqrt() * g + c

    def loss(h):
        q = {k: base[k] + h * dirs[k] for k in base}
        x0 = torch.where(real[:, None], q["e"][torch.where(real, tokens, 0)], 0.0)
        a = norm(x0, q["g1"], q["c1"]) @ q["w1"].t() + q["b1"]
        x1 = x0 + (0.5 * a * torch.special.erfc(-a / 2.0 ** 0.5)) @ q["w2"].t() + q["b2"]
        t = norm(x1, q["g2"], q["c2"]) @ q["e"][:model.vocab].t()
        each = torch.logsumexp(t, 1) - t.gather(1, torch.where(real, labels, 0)[:, None])[:, 0]
        return float(each[real].mean())

    slope = (loss(1e-4) - loss(-1e-4)) / 2e-4
    got = {k: float((grads[k].double() * dirs[k]).sum()) for k in base}
    # a rounding's error times its share of the directional derivative adds up like independent errors; in full it is
    # at most this part of the norms
    size = sum(float(grads[k].double().norm() * dirs[k].norm()) for k in base)
    assert abs(slope - sum(got.values())) <= 8 * B16 * size, (slope, got)


def test_captured_step_equals_eager(z, ex):
    """Forward, backward and the optimizer's step of two ranks in one graph, replayed: the same bits as eager calls."""
    model = ex.Model()
    hp = {"lr": 3e-3, "beta1": 0.9, "beta2": 0.95, "eps": 1e-8, "weight_decay": 0.0}
    eager, graphed = (ex.setup(model, 2, 200, DEV, seed=7) for _ in range(2))

    def step(s):
        p = model.params(s["param"][:model.psi])
        for r in range(2):
            one_step(ex, model, p, s, r)
        z.zero_fused_step(s["plan"], z.ZERO_ALL_RANKS, s["grads"], s["master"], s["m"], s["v"], s["param"], hp, 1)

    state = {k: graphed[k].clone() for k in ("master", "m", "v", "param")}
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step(graphed)  # first use of every kernel outside the capture
    side.synchronize()
    for k, v in state.items():
        graphed[k].copy_(v)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(graphed)
    for k, v in state.items():
        graphed[k].copy_(v)
    for _ in range(3):
        step(eager)
        graph.replay()
    torch.cuda.synchronize()
    z.zero_device_status()
    for k in ("master", "m", "v", "param"):
        assert torch.equal(eager[k], graphed[k]), k
    for a, b in zip(eager["grads"], graphed["grads"]):
        assert torch.equal(a, b)


def test_ranks_on_streams_of_their_own(z, ex):
    """Two ranks' passes at once, each on its stream with its buffers: the same bits as one after the other."""
    model = ex.Model(vocab=4001, d=256, f=512, shards=2)
    s = ex.setup(model, 2, 700, DEV, seed=9)
    p = model.params(s["param"][:model.psi])
    for r in range(2):
        one_step(ex, model, p, s, r)
    torch.cuda.synchronize()
    want = [t.clone() for t in s["grads"]]
    side = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        for t in s["grads"]:
            t.zero_()
        torch.cuda.synchronize()
        for r in range(2):
            with torch.cuda.stream(side[r]):
                one_step(ex, model, p, s, r)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, s["grads"]))
    z.zero_device_status()


def test_example_runs(ex):
    losses = ex.main(steps=3, m=128)
    assert len(losses) == 3 and all(l == l and l < 1e3 for l in losses)
