"""The linear unit's calls together: the example trains; a chain of dependent calls without any
synchronisation, on its own stream and replayed from a CUDA graph, gives the bits of the same
calls one at a time; shards that lie back to back give the bits of separate ones."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import synth

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


def randn(rows, cols, std, key):
    g = torch.Generator().manual_seed(synth.derive_seed(92, rows, cols, key))
    return (torch.randn(rows, cols, generator=g) * std).to(BF).to(DEV)


def test_example_trains(z):
    from fsdp_sharded_optimizer_zero_gb300 import example_linear
    losses = example_linear.main(steps=30)
    assert all(np.isfinite(losses)) and losses[-1] < 0.5 * losses[0]
    assert example_linear.main(steps=3) == losses[:3]  # the same bits again


def test_example_gradients_against_autograd(z):
    """The example's backward against float64 autograd of the same block on the values the
    forward kept (X and Z in 8 bits): every bf16 rounding on the way (H, dZ, the gradients) is
    2^-8 of the terms it rounds, so the gradients' norms agree within 4 x 2^-8."""
    from fsdp_sharded_optimizer_zero_gb300 import example_linear as e
    m, d, f = 333, 136, 264
    x, dy = randn(m, d, 1.0, 1), randn(m, d, 0.1, 2)
    p = {"w1": list(randn(f, d, 0.08, 3).chunk(3)), "b1": randn(1, f, 0.2, 4)[0].contiguous(),
         "w2": [randn(d, f, 0.06, 5)], "b2": randn(1, d, 0.2, 6)[0].contiguous()}
    b = e.block_buffers(m, d, f, DEV)
    g = {"w1": torch.empty(f, d, dtype=BF, device=DEV), "b1": torch.empty(f, dtype=BF, device=DEV),
         "w2": torch.empty(d, f, dtype=BF, device=DEV), "b2": torch.empty(d, dtype=BF, device=DEV)}
    y = e.forward(p, x, b).double()
    dx = e.backward(p, dy, g, b)
    z.zero_device_status()
    kept = []
    for name, cols in (("x8", d), ("z8", f)):
        t = torch.empty(m, cols, dtype=BF, device=DEV)
        z.fsdp_checkpoint8_unpack(*b[name], t)
        kept.append(t.double())
    x64, w1, w2 = kept[0], torch.cat(p["w1"]).double(), torch.cat(p["w2"]).double()
    pre = kept[1].requires_grad_()
    h = torch.nn.functional.gelu(pre)
    (h @ w2.T).backward(dy.double())
    dz = pre.grad
    want = {"w2": dy.double().T @ h.detach(), "b2": dy.double().sum(0), "w1": dz.T @ x64, "b1": dz.sum(0)}
    for name, v in want.items():
        assert (g[name].double() - v).norm() <= 4 * 2.0 ** -8 * v.norm(), name
    v = dz @ w1 + dy.double()
    assert (dx.double() - v).norm() <= 4 * 2.0 ** -8 * v.norm()
    v = torch.nn.functional.gelu(x.double() @ w1.T + p["b1"].double()) @ w2.T + p["b2"].double() + x.double()
    assert (y - v).norm() <= 4 * 2.0 ** -8 * v.norm()


# sizes that take the narrow kernel, the wide one, and both in one chain
@pytest.mark.parametrize("m,d,f", [(48, 256, 512), (1500, 2048, 2304), (2100, 1024, 3328)])
def test_unsynchronised_chain_and_graph_give_the_same_bits(z, m, d, f):
    from fsdp_sharded_optimizer_zero_gb300 import example_linear as e
    x, dy = randn(m, d, 1.0, 7), randn(m, d, 0.1, 8)
    p = {"w1": list(randn(f, d, 0.03, 9).chunk(2)), "b1": randn(1, f, 0.2, 10)[0].contiguous(),
         "w2": list(randn(d, f, 0.03, 11).chunk(2)), "b2": randn(1, d, 0.2, 12)[0].contiguous()}

    def fresh():
        b = e.block_buffers(m, d, f, DEV)
        g = {k: torch.zeros(s, dtype=BF, device=DEV) for k, s in (("w1", (f, d)), ("b1", (f,)), ("w2", (d, f)),
                                                                   ("b2", (d,)))}
        return b, g

    def run(b, g):
        e.forward(p, x, b)
        return e.backward(p, dy, g, b)

    # one call at a time: every call of the chain synchronised
    b0, g0 = fresh()
    names = ("fsdp_checkpoint8_pack", "fsdp_checkpoint8_unpack", "fsdp_linear_forward", "fsdp_linear_dw",
             "fsdp_linear_dx", "fsdp_act_backward")
    saved = {k: getattr(z, k) for k in names}
    try:
        for k in names:
            def call(*a, _f=saved[k], **kw):
                _f(*a, **kw)
                torch.cuda.synchronize()
            setattr(z, k, call)
        run(b0, g0)
        torch.cuda.synchronize()
    finally:
        for k in names:
            setattr(z, k, saved[k])

    def same(b, g):
        for k in ("h", "y", "dz", "dx", "db1", "db2"):
            assert torch.equal(b[k], b0[k]), k
        for k in ("x8", "z8"):
            assert torch.equal(b[k][0], b0[k][0]) and torch.equal(b[k][1], b0[k][1]), k
        for k in g0:
            assert torch.equal(g[k], g0[k]), k

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b, g = fresh()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(3):
            run(b, g)
    side.synchronize()
    same(b, g)
    b, g = fresh()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(b, g)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    same(b, g)
    z.zero_device_status()


@pytest.mark.parametrize("m,r,k,n", [(40, 480, 264, 4), (700, 4608, 264, 16), (1030, 2400, 1096, 12)])
def test_joined_and_separate_shards_give_the_same_bits(z, m, r, k, n):
    w, x, dz = randn(r, k, 0.05, 13), randn(m, k, 1.0, 14), randn(m, r, 0.3, 15)
    joined = list(w.chunk(n))
    room = torch.empty(n, r // n * k + 64, dtype=BF, device=DEV)  # 128 bytes between the shards
    apart = [room[i, :r // n * k].view(r // n, k) for i in range(n)]
    for t, s in zip(apart, joined):
        t.copy_(s)
    out = []
    for shards in (joined, apart, [w]):
        y, dx = torch.empty(m, r, dtype=BF, device=DEV), torch.empty(m, k, dtype=BF, device=DEV)
        z.fsdp_linear_forward(shards, x, y, act=z.FSDP_ACT_SILU)
        z.fsdp_linear_dx(shards, dz, dx)
        out.append((y, dx))
    for y, dx in out[1:]:
        assert torch.equal(y, out[0][0]) and torch.equal(dx, out[0][1])
