"""Gradients of a language model's step and of the mean loss, along directions in which a missing term, a wrong sign or a wrong
scale shows: the gradients' own."""
from __future__ import annotations

import pytest
import torch

from test_language_ends_chain import B16, DEV, one_step
from test_vocab_loss import Case


@pytest.fixture(scope="module")
def z():
    import __graft_entry__ as g
    g.build()
    import fsdp_sharded_optimizer_zero_gb300 as z
    yield z
    if torch.cuda.is_available():
        z.zero_device_status()


# A gradient's way through the model rounds to bf16 eight times at most (the activations on the way to the loss among them), each
# by up to B16 of the value: relative to the tensor's norm, with all of them in line, 8 B16 = 3.1 %.
PART = 8 * B16
TERMS = ("skip", "embedding", "head")  # of X1's gradient from norm 2 past the MLP; the two of the tied table


def loss64(model, q, tokens, labels, eps, without=""):
    """The example's mean loss by torch's own differentiation; `without`: one term's gradient left out."""
    real = (tokens >= 0) & (tokens < model.vocab)

    def norm(x, g, c):
        d = x - x.mean(1, keepdim=True)
        return d * (d.square().mean(1, keepdim=True) + eps).rsqrt() * g + c

    def cut(t, term):
        return t.detach() if without == term else t

    table = q["e"][:model.vocab]
    x0 = torch.where(real[:, None], cut(table, "embedding")[torch.where(real, tokens, 0)], 0.0)
    a = norm(x0, q["g1"], q["c1"]) @ q["w1"].t() + q["b1"]
    x1 = cut(x0, "skip") + (0.5 * a * torch.special.erfc(-a / 2.0 ** 0.5)) @ q["w2"].t() + q["b2"]
    t = norm(x1, q["g2"], q["c2"]) @ cut(table, "head").t()
    each = torch.logsumexp(t, 1) - t.gather(1, torch.where(real, labels, 0)[:, None])[:, 0]
    return each[real].mean()


def gradients64(model, params, tokens, labels, eps, without=""):
    q = {k: v.double().clone().requires_grad_(True) for k, v in params.items()}
    loss64(model, q, tokens, labels, eps, without).backward()
    return {k: v.grad for k, v in q.items()}


def apart(got, want):
    """How far each tensor's gradient is, in parts of its norm."""
    return {k: float((got[k].double() - want[k]).norm() / want[k].norm()) for k in want}


def batch(model, m, dev, seed):
    """Parameters away from their symmetric start (norms' factors of 1, biases of 0), and a batch."""
    gen = torch.Generator(device=dev).manual_seed(seed)
    params = {}
    for name, s in model.sizes.items():
        r = torch.randn(*s, generator=gen, device=dev)
        params[name] = (r * s[1] ** -0.5 if len(s) == 2 else 1.0 + 0.3 * r if name[0] == "g" else 0.3 * r).to(torch.bfloat16)
    params["e"][model.vocab:] = 0
    tokens = torch.randint(0, model.vocab, (m,), generator=gen, device=dev)
    labels = torch.randint(0, model.vocab, (m,), generator=gen, device=dev)
    tokens[m - m // 8:], labels[m - m // 8:] = -100, -100
    return params, tokens, labels


SIZES = [(200, dict(vocab=203, d=64, f=128, shards=1)), (384, dict(vocab=1003, d=128, f=512, shards=4))]


@pytest.mark.gpu
@pytest.mark.parametrize("m,sizes", SIZES)
def test_each_tensor_of_a_step(z, m, sizes):
    from fsdp_sharded_optimizer_zero_gb300 import example_language as ex
    model = ex.Model(**sizes)
    s = ex.setup(model, 1, m, DEV, seed=5)
    params, tokens, labels = batch(model, m, DEV, 6)
    for name, view in model.views(s["param"][:model.psi]).items():
        view.copy_(params[name])
    s["batches"][0] = (tokens, labels)
    one_step(ex, model, model.params(s["param"][:model.psi]), s, 0)
    z.zero_device_status()
    got = model.views(s["grads"][0][:model.psi])
    off = apart(got, gradients64(model, params, tokens, labels, ex.EPS))
    assert all(v <= PART for v in off.values()), off


@pytest.mark.parametrize("m,sizes", SIZES)
@pytest.mark.parametrize("term", TERMS)
def test_a_missing_term_shows(m, sizes, term):
    """By the reference alone, on the CPU: a term left out takes the table's gradient more than twice what is allowed above away,
    so that a result that lacks it is outside whatever its roundings."""
    from fsdp_sharded_optimizer_zero_gb300 import example_language as ex
    model = ex.Model(**sizes)
    params, tokens, labels = batch(model, m, "cpu", 6)
    whole, cut = (gradients64(model, params, tokens, labels, ex.EPS, w) for w in ("", term))
    assert apart(cut, whole)["e"] > 2 * PART


@pytest.mark.gpu
@pytest.mark.parametrize("m,vocab,rows,k,n", [(257, 700, 704, 136, 4), (20, 1157, 1160, 264, 5)])
@pytest.mark.parametrize("factors", [False, True])
def test_mean_loss_along_its_gradients(z, m, vocab, rows, k, n, factors):
    """Central differences in float64 along dX and along dW: the slope is the gradient's own square."""
    c = Case(m, vocab, rows, k, n)
    g = torch.rand(m, generator=torch.Generator(device=DEV).manual_seed(m), device=DEV).add(0.5) if factors else None
    _, lse, total = c.forward(z)
    dX, dW = (t.double() for t in c.backward(z, lse, dloss=g, total=total))
    dW = dW[:vocab]
    weight = c.weights(g) / c.real.sum()

    def loss(x, w):
        t = x @ w.t()
        return float(((torch.logsumexp(t, 1) - t.gather(1, c.at[:, None])[:, 0]) * weight).sum())

    dz = torch.exp(c.z - c.lse[:, None]) * weight[:, None]
    dz.scatter_add_(1, c.at[:, None], -weight[:, None])
    roundings = 2 if factors else 1  # of the products' operands: dZ, and with factors X
    for grad, along in ((dX, "x"), (dW, "w")):
        v = grad / grad.norm()
        h = 1e-4 * (c.x64 if along == "x" else c.w64).norm() / v.numel() ** 0.5
        ends = [loss(c.x64 + s * h * v, c.w64) if along == "x" else loss(c.x64, c.w64 + s * h * v) for s in (1, -1)]
        slope, got = (ends[0] - ends[1]) / (2 * float(h)), float((grad * v).sum())
        # each rounding by at most B16 of the element: dZ's (and X's) as the products pass it on, the result's
        passed = float((dz.abs() * (v @ c.w64.t() if along == "x" else c.x64 @ v.t()).abs()).sum())
        bound = 1.05 * B16 * (roundings * passed + float((grad * v).abs().sum()))
        assert bound < 0.05 * got, (bound, got)  # or a wrong scale would not show
        assert abs(slope - got) <= bound + 1e-6 * got, (slope, got, bound)
