"""Layer norm, forward and backward, against float64 on the GPU, with derived bounds.

U is half a step of fp32, B16 of bf16. A row's sums are fp32 sums whose terms pass through at most D
additions; a product or sum adds a rounding each."""
from __future__ import annotations

import pytest
import torch

import synth

DEV = "cuda"
BF = torch.bfloat16
U, B16 = 2.0 ** -24, 2.0 ** -8

# every number of warps to a row and of pieces to a lane, rows wider than the registers, cut last pieces
SHAPES = [(1, 8), (3, 16), (700, 24), (33, 248), (1, 256), (9, 264), (5000, 768), (2, 768), (1100, 1024), (3000, 1032),
          (17, 2304), (1300, 2304), (1, 4096), (2500, 4096), (777, 5128), (40, 8192), (1300, 8200), (200, 12296),
          (65, 16384), (3, 16392), (70, 40008)]


@pytest.fixture(scope="module")
def z():
    import __graft_entry__ as g
    g.build()
    import fsdp_sharded_optimizer_zero_gb300 as z
    yield z
    if torch.cuda.is_available():
        z.zero_device_status()


def randn(*shape, std=1.0, key=0):
    gen = torch.Generator(device=DEV).manual_seed(synth.derive_seed(95, *shape, key))
    return torch.randn(*shape, generator=gen, device=DEV) * std


def guarded(*shape, dtype=BF):
    """A tensor with 64 sentinels behind it, and the check that they are untouched."""
    n = 1
    for s in shape:
        n *= s
    flat = torch.full((n + 64,), 3.0, dtype=dtype, device=DEV)
    flat[:n] = float("nan")

    def check():
        assert bool((flat[n:] == 3.0).all())
    return flat[:n].view(*shape), check


def depth(cols):
    return 48 + cols / 1024.0


def inside(got, want, bound, what):
    off = (got.double() - want).abs()
    bad = ~(off <= bound)
    assert not bool(bad.any()), (what, int(bad.sum()), float(off[bad].max()), float((off / bound)[bad].max()))


def forward64(x, gamma, beta, eps):
    x = x.double()
    mean = x.mean(1, keepdim=True)
    var = (x - mean).square().mean(1, keepdim=True)
    rstd = (var + eps).rsqrt()
    h = (x - mean) * rstd
    g = torch.ones_like(x[0]) if gamma is None else gamma.double()
    b = torch.zeros_like(x[0]) if beta is None else beta.double()
    e_mean = depth(x.shape[1]) * U * x.abs().mean(1, keepdim=True)
    # the variance: its terms two roundings each, and the square of the mean's error
    e_rel = 0.5 * (depth(x.shape[1]) + 4) * U + 0.5 * e_mean.square() / (var + eps) + 4 * U
    y = h * g + b
    e_y = (g.abs() * (h.abs() * (e_rel + 4 * U) + rstd * e_mean) + 2 * U * y.abs()) * 1.01
    return mean[:, 0], rstd[:, 0], y, e_mean[:, 0], e_rel[:, 0] * rstd[:, 0], e_y


@pytest.mark.gpu
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_forward(z, rows, cols):
    x = (randn(rows, cols) * torch.exp(randn(rows, 1, key=1)) + randn(rows, 1, std=2.0, key=2)).to(BF)
    gamma, beta = randn(cols, key=3).to(BF), randn(cols, key=4).to(BF)
    for g, b, eps in ((gamma, beta, 1e-5), (None, None, 0.5), (gamma, None, 1e-12), (None, beta, 0.0)):
        y, ok_y = guarded(rows, cols)
        mean, ok_m = guarded(rows, dtype=torch.float32)
        rstd, ok_r = guarded(rows, dtype=torch.float32)
        z.fsdp_layernorm_forward(x, y, gamma=g, beta=b, eps=eps, mean=mean, rstd=rstd)
        m64, r64, y64, em, er, ey = forward64(x, g, b, eps)
        inside(mean, m64, em + U * m64.abs(), "mean")
        if eps == 0.0 and cols == 8:
            continue  # a row of 8 may have nearly no variance
        inside(rstd, r64, er, "rstd")
        inside(y, y64, ey + B16 * (y64.abs() + ey), "Y")
        for ok in (ok_y, ok_m, ok_r):
            ok()
    again = torch.empty_like(y)
    z.fsdp_layernorm_forward(x, again, beta=beta, eps=0.0)  # without the statistics: the same Y
    assert torch.equal(again.view(torch.int16), y.view(torch.int16))


def backward64(dy, x, mean, rstd, gamma, res):
    dy, x, m, r = dy.double(), x.double(), mean.double()[:, None], rstd.double()[:, None]
    n = x.shape[1]
    g = dy * (1.0 if gamma is None else gamma.double())
    h = (x - m) * r
    dx = r * (g - g.mean(1, keepdim=True) - h * (g * h).mean(1, keepdim=True))
    # h: two roundings. Its sums: D more
    d = depth(n)
    e = r * (3 * U * g.abs() + d * U * g.abs().mean(1, keepdim=True) + h.abs() * (d + 8) * U * (g * h).abs().mean(1, keepdim=True)
             + 4 * U * (g.abs() + g.mean(1, keepdim=True).abs() + (h * (g * h).mean(1, keepdim=True)).abs()))
    if res is not None:
        dx = dx + res.double()
        e = e + U * dx.abs()
    return dx, e * 1.01, (dy * h).sum(0), (dy * h).abs().sum(0), dy.sum(0), dy.abs().sum(0)


def rows_depth(rows):
    return rows + 4  # a column's sum passes through at most as many additions as there are rows


@pytest.mark.gpu
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_backward(z, rows, cols):
    x = (randn(rows, cols) * torch.exp(randn(rows, 1, key=1)) + randn(rows, 1, std=2.0, key=2)).to(BF)
    gamma, dy, res = randn(cols, key=3).to(BF), randn(rows, cols, std=0.1, key=5).to(BF), randn(rows, cols, std=0.1, key=6).to(BF)
    mean, rstd = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    z.fsdp_layernorm_forward(x, torch.empty_like(x), mean=mean, rstd=rstd)
    for g, r in ((gamma, res), (None, None), (gamma, None)):
        dx, ok = guarded(rows, cols)
        dg, ok_g = guarded(cols, dtype=torch.float32)
        db, ok_b = guarded(cols, dtype=torch.float32)
        z.fsdp_layernorm_backward(dy, x, mean, rstd, dx, gamma=g, residual=r, dgamma=dg, dbeta=db)
        dx64, e, dg64, dga, db64, dba = backward64(dy, x, mean, rstd, g, r)
        inside(dx, dx64, e + B16 * (dx64.abs() + e), "dX")
        inside(dg, dg64, (rows_depth(rows) + 4) * U * dga, "dgamma")
        inside(db, db64, rows_depth(rows) * U * dba, "dbeta")
        for c in (ok, ok_g, ok_b):
            c()
        # one of the two, or neither: the same bits
        one = torch.empty_like(dg)
        z.fsdp_layernorm_backward(dy, x, mean, rstd, torch.empty_like(dx), gamma=g, residual=r, dgamma=one)
        assert torch.equal(one, dg)
        z.fsdp_layernorm_backward(dy, x, mean, rstd, torch.empty_like(dx), gamma=g, residual=r, dbeta=one)
        assert torch.equal(one, db)
        plain = torch.empty_like(dx)
        z.fsdp_layernorm_backward(dy, x, mean, rstd, plain, gamma=g, residual=r)
        assert torch.equal(plain, dx)
        # in place of dY, and of the residual
        inplace = dy.clone()
        z.fsdp_layernorm_backward(inplace, x, mean, rstd, inplace, gamma=g, residual=r, dgamma=dg, dbeta=one)
        assert torch.equal(inplace, dx) and torch.equal(one, db)
        if r is not None:
            skip = r.clone()
            z.fsdp_layernorm_backward(dy, x, mean, rstd, skip, gamma=g, residual=skip)
            assert torch.equal(skip, dx)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,cols", [(5, 264), (300, 2304), (4, 16392)])
def test_gradients_against_differences(z, rows, cols):
    """Along random directions of X, gamma and beta: central differences of L = sum dY . Y in float64."""
    eps = 1e-5
    x, gamma, beta = randn(rows, cols).to(BF), (1 + 0.2 * randn(cols, key=1)).to(BF), randn(cols, key=2).to(BF)
    dy = randn(rows, cols, std=0.1, key=3).to(BF)
    mean, rstd = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    z.fsdp_layernorm_forward(x, torch.empty_like(x), gamma=gamma, beta=beta, eps=eps, mean=mean, rstd=rstd)
    dx, dg, db = torch.empty_like(x), torch.empty(cols, device=DEV), torch.empty(cols, device=DEV)
    z.fsdp_layernorm_backward(dy, x, mean, rstd, dx, gamma=gamma, dgamma=dg, dbeta=db)
    x64, g64, b64 = x.double(), gamma.double(), beta.double()

    def loss(a, g, b):
        c = a - a.mean(1, keepdim=True)
        return float((dy.double() * (c * (c.square().mean(1, keepdim=True) + eps).rsqrt() * g + b)).sum())

    h = 1e-4
    v = randn(rows, cols, key=4).double()
    slope = (loss(x64 + h * v, g64, b64) - loss(x64 - h * v, g64, b64)) / (2 * h)
    # differences: third derivatives of order h^2; dX is rounded to bf16
    size = float((dx.double() * v).abs().sum())
    assert abs(slope - float((dx.double() * v).sum())) <= (B16 + 1e-5) * size + 1e-6 * float(dy.double().abs().sum())
    for grad, at in ((dg, 1), (db, 2)):
        v = randn(cols, key=5).double()
        lo, hi = [x64, g64, b64], [x64, g64, b64]
        lo[at], hi[at] = lo[at] - h * v, hi[at] + h * v
        slope = (loss(*hi) - loss(*lo)) / (2 * h)  # linear in both
        size = float((grad.double() * v).abs().sum()) + float(dy.double().abs().sum())
        assert abs(slope - float((grad.double() * v).sum())) <= 1e-5 * size


@pytest.mark.gpu
@pytest.mark.parametrize("rows,cols", [(6, 768), (6, 4096), (6, 20000)])
def test_a_row_that_is_not_finite_leaves_the_others(z, rows, cols):
    x = randn(rows, cols).to(BF)
    want, wm, wr = torch.empty_like(x), torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    z.fsdp_layernorm_forward(x, want, mean=wm, rstd=wr)
    x[1, 3], x[4, cols - 1] = float("inf"), float("nan")
    y, m, r = torch.empty_like(x), torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    z.fsdp_layernorm_forward(x, y, mean=m, rstd=r)
    for i in (1, 4):
        assert bool(y[i].isnan().any()) and not bool(r[i].isfinite())
    for i in (0, 2, 3, 5):
        assert torch.equal(y[i], want[i]) and bool(m[i] == wm[i]) and bool(r[i] == wr[i])


@pytest.mark.gpu
def test_constant_rows(z):
    """No variance: rstd = eps^-1/2, Y = beta, and the gradient is that of a shift and a scale by rstd."""
    x = torch.full((3, 1032), 7.0, dtype=BF, device=DEV)
    beta = randn(1032, key=1).to(BF)
    y, m, r = torch.empty_like(x), torch.empty(3, device=DEV), torch.empty(3, device=DEV)
    z.fsdp_layernorm_forward(x, y, beta=beta, eps=2.0 ** -16, mean=m, rstd=r)
    inside(m, torch.full((3,), 7.0, device=DEV).double(), torch.tensor(depth(1032) * U * 7.0, device=DEV), "mean")
    # x - mean may be the mean's rounding, times rstd = 2^8
    inside(y, beta.double().expand(3, -1), depth(1032) * U * 7.0 * 256 + B16 * beta.double().abs() + 1e-9, "Y")


@pytest.mark.gpu
def test_row_views_and_alignment(z):
    """Rows of a larger buffer; a base that is not 16-byte aligned is refused."""
    big = randn(40, 264).to(BF)
    y = torch.zeros(40, 264, dtype=BF, device=DEV)
    z.fsdp_layernorm_forward(big[10:20], y[10:20])
    want = torch.empty(10, 264, dtype=BF, device=DEV)
    z.fsdp_layernorm_forward(big[10:20].clone(), want)
    assert torch.equal(y[10:20], want) and not bool(y[:10].any()) and not bool(y[20:].any())
    off = torch.zeros(8 * 264 + 4, dtype=BF, device=DEV)[4:].view(8, 264)
    with pytest.raises(z.ZeroError, match="16-byte"):
        z.fsdp_layernorm_forward(off, y[:8])


@pytest.mark.gpu
def test_streams_and_graph(z):
    """On another stream than the current one, and captured and replayed with new inputs."""
    rows, cols = 500, 1160
    x, dy, gamma = randn(rows, cols).to(BF), randn(rows, cols, key=1).to(BF), randn(cols, key=2).to(BF)
    new = lambda: [torch.empty(rows, cols, dtype=BF, device=DEV), torch.empty(rows, device=DEV),  # noqa: E731
                   torch.empty(rows, device=DEV), torch.empty(rows, cols, dtype=BF, device=DEV),
                   torch.empty(cols, device=DEV), torch.empty(cols, device=DEV)]
    ws = torch.empty(z.fsdp_layernorm_backward_workspace(rows, cols), dtype=torch.uint8, device=DEV)

    def call(o, **kw):
        z.fsdp_layernorm_forward(x, o[0], gamma=gamma, mean=o[1], rstd=o[2], **kw)
        z.fsdp_layernorm_backward(dy, x, o[1], o[2], o[3], gamma=gamma, dgamma=o[4], dbeta=o[5], **kw)

    want, got = new(), new()
    call(want)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    call(got, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    out = new()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        z.fsdp_layernorm_forward(x, out[0], gamma=gamma, mean=out[1], rstd=out[2])
        z.fsdp_layernorm_backward(dy, x, out[1], out[2], out[3], gamma=gamma, dgamma=out[4], dbeta=out[5], workspace=ws)
    x.copy_(randn(rows, cols, key=7).to(BF))
    for _ in range(2):
        graph.replay()
    call(want)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, out))
