"""The linear unit at sizes of many 256 x 256 tiles with ragged edges in every dimension (the wide
kernel, with operands that need one copy a stage and with ones that need several), every
epilogue, against float64 on the GPU (torch). Bounds as in test_linear_unit."""
from __future__ import annotations

import math

import pytest
import torch

import synth

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16
G = 32
ACTS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}
SUM, B16 = 2.0 ** -23, 2.0 ** -8


@pytest.fixture(scope="module")
def z():
    import __graft_entry__ as g
    g.build()
    import fsdp_sharded_optimizer_zero_gb300 as z
    yield z
    z.zero_device_status()


def randn(rows, cols, std, key):
    gen = torch.Generator(device=DEV).manual_seed(synth.derive_seed(93, rows, cols, key))
    return (torch.randn(rows, cols, generator=gen, device=DEV) * std).to(BF)


def act64(x, act):
    if act == "relu":
        return x.clamp(min=0)
    if act == "gelu":
        return 0.5 * x * torch.special.erfc(-x / math.sqrt(2.0))
    if act == "gelu_tanh":
        return x * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (x + 0.044715 * x ** 3))
    return x * torch.sigmoid(x) if act == "silu" else x


def dact64(x, act):
    if act == "none":
        return torch.ones_like(x)
    if act == "relu":  # 0 at 0, where autograd's clamp takes 1
        return (x > 0).double()
    x = x.clone().requires_grad_()
    act64(x, act).sum().backward()
    return x.grad


def act_err(v, act):
    a = v.abs().clamp(max=90.0)
    rel = 2.0 ** -20 + a * 2.0 ** -21
    if act in ("none", "relu"):
        return 0.0 * a, 0.0 * a
    return rel * act64(v, act).abs() + 2.0 ** -120, rel * (1.0 + a) + 2.0 ** -120


def inside(got, want, bound, what):
    assert got.shape == want.shape
    bad = ~((got.double() - want).abs() <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} outside; first at {bad.nonzero()[0].tolist()}"


def new8(rows, cols):
    return (torch.empty(rows, cols, dtype=torch.int8, device=DEV),
            torch.empty(rows, -(-cols // G), dtype=torch.uint8, device=DEV))


def values(z, c):
    t = torch.empty(c[0].shape, dtype=BF, device=DEV)
    z.fsdp_checkpoint8_unpack(*c, t)
    return t.double()


def guarded(rows, cols, dtype, fill):
    buf = torch.full((rows * cols + 512,), fill, dtype=dtype, device=DEV)
    return buf, buf[256:256 + rows * cols].view(rows, cols)


def kept(buf, fill):
    return bool((buf[:256] == fill).all()) and bool((buf[-256:] == fill).all())


def apart(w, n):
    """n row shards with 128 bytes between them."""
    r, k = w.shape[0] // n, w.shape[1]
    room = torch.empty(n, r * k + 64, dtype=BF, device=DEV)
    out = [room[i, :r * k].view(r, k) for i in range(n)]
    for i, t in enumerate(out):
        t.copy_(w[i * r:(i + 1) * r])
    return out


# (m, r, k, shards, rows of a shard: copies of 8, 16, 32, 64 or 128 rows, or one matrix)
SHAPES = [(1030, 2400, 1096, 12), (2053, 2312, 264, 1), (1281, 2560, 2312, 16), (1800, 2304, 2368, 8),
          (2300, 1544, 1544, 1), (1100, 4096, 2048, 8), (2500, 1160, 1288, 5), (1537, 2816, 1672, 11)]


def forward_case(i):
    act = sorted(ACTS)[i % 5]
    return act, ("z", "z8", "none")[i % 3], i % 2 == 0, i % 4 in (0, 3)


def check_forward(z, m, r, k, n, act, kind, has_bias, has_res):
    x, w = randn(m, k, 1.0, 1), randn(r, k, 0.04, 2)
    bias = randn(1, r, 0.5, 3)[0].contiguous() if has_bias else None
    res = randn(m, r, 2.0, 4) if has_res else None
    ybuf, y = guarded(m, r, BF, 3.0)
    zbuf, zk = guarded(m, r, BF, 3.0)
    cbuf, codes = guarded(m, r, torch.int8, 99)
    sbuf, scales = guarded(m, -(-r // G), torch.uint8, 77)
    keep = {"z": {"z": zk}, "z8": {"z8": (codes, scales)}, "none": {}}[kind]
    z.fsdp_linear_forward(apart(w, n), x, y, bias=bias, act=ACTS[act], residual=res, **keep)
    z.zero_device_status()
    x64, w64 = x.double(), w.double()
    pre, ez = x64 @ w64.T, (k + 1) * SUM * (x64.abs() @ w64.abs().T)
    if has_bias:
        pre = pre + bias.double()
        ez = ez + SUM * pre.abs()
    want, e = act64(pre, act), 1.2 * ez + act_err(pre, act)[0]
    if has_res:
        want = want + res.double()
        e = e + SUM * want.abs()
    inside(y, want, e + B16 * (want.abs() + e), f"Y {act}")
    if kind == "z":
        inside(zk, pre, ez + B16 * (pre.abs() + ez), "Z")
    if kind == "z8":
        step = torch.exp2(scales.double() - 127.0).repeat_interleave(G, 1)[:, :r]
        inside(values(z, (codes, scales)), pre, step / 2 + ez, "Z in 8 bits")
        pad = -r % G
        amax = torch.nn.functional.pad(pre.abs() + ez, (0, pad)).view(m, -1, G).amax(-1)
        assert (torch.exp2(scales.double() - 127.0) <= 2.0 * amax / 127.5 * (1 + 1e-12)).all()  # no byte larger than needed
    assert kept(ybuf, 3.0) and kept(zbuf, 3.0) and kept(cbuf, 99) and kept(sbuf, 77)
    again = torch.empty_like(y)
    z.fsdp_linear_forward([w], x, again, bias=bias, act=ACTS[act], residual=res)
    assert torch.equal(again, y)


@pytest.mark.parametrize("i", range(24))
def test_forward(z, i):
    m, r, k, n = SHAPES[i % len(SHAPES)]
    check_forward(z, m, r, k, n, *forward_case(i // len(SHAPES) + i))


def check_dx(z, m, r, k, n, act, has_res, bits8):
    g, w, pre = randn(m, r, 0.3, 5), randn(r, k, 0.04, 6), randn(m, k, 1.5, 7)
    res = randn(m, k, 0.5, 8) if has_res else None
    c = new8(m, k)
    z.fsdp_checkpoint8_pack(pre, *c)
    arg, v = ({"z8": c}, values(z, c)) if bits8 else ({"z": pre}, pre.double())
    buf, dx = guarded(m, k, BF, 3.0)
    z.fsdp_linear_dx(apart(w, n), g, dx, act=ACTS[act], residual=res, **arg)
    z.zero_device_status()
    g64, w64 = g.double(), w.double()
    acc, ea = g64 @ w64, (r + 1) * SUM * (g64.abs() @ w64.abs())
    d, ed = dact64(v, act), act_err(v, act)[1]
    want = acc * d
    e = ea * (d.abs() + ed) + acc.abs() * ed + SUM * want.abs()
    if has_res:
        want = want + res.double()
        e = e + SUM * want.abs()
    inside(dx, want, e + B16 * (want.abs() + e), f"dX {act}")
    assert kept(buf, 3.0)


@pytest.mark.parametrize("i", range(16))
def test_dx(z, i):
    m, r, k, n = SHAPES[i % len(SHAPES)]
    act, _, has_res, bits8 = forward_case(i // len(SHAPES) + i)
    check_dx(z, m, r, k, n, act, has_res, bits8)


def check_dw(z, m, r, k, wide):
    """fp32 results over more than 4096 tokens are summed in parts: their error stays below the
    4096-term bound (4097 2^-23 of the magnitudes) plus a rounding per part."""
    g, x = randn(m, r, 0.3, 9), randn(m, k, 1.0, 10)
    c = new8(m, k)
    z.fsdp_checkpoint8_pack(x, *c)
    for arg, v in (({"x": x}, x.double()), ({"x8": c}, values(z, c))):
        buf, dw = guarded(r, k, torch.float32 if wide else BF, 3.0)
        z.fsdp_linear_dw(g, dw, scale=0.25, **arg)
        z.zero_device_status()
        want, mag = 0.25 * (g.double().T @ v), 0.25 * (g.double().abs().T @ v.abs())
        terms = min(m, 4096) if wide else m
        e = (terms + 1 + m // 4096) * SUM * mag + SUM * want.abs()
        inside(dw, want, e if wide else e + B16 * (want.abs() + e), "dW")
        assert kept(buf, 3.0)


@pytest.mark.parametrize("wide", [True, False])
@pytest.mark.parametrize("m,r,k", [(300, 2312, 1096), (1, 2304, 1544), (4097, 1544, 2312), (9001, 2560, 1160),
                                   (5000, 2048, 2048), (65, 2048, 2112)])
def test_dw(z, m, r, k, wide):
    check_dw(z, m, r, k, wide)


def test_dw_workspace_and_streams(z):
    """A workspace of the caller's, one from the allocator, a side stream as an object and as a
    handle: the same bits."""
    m, r, k = 500, 264, 328
    g, x = randn(m, r, 0.3, 11), randn(m, k, 1.0, 12)
    c = new8(m, k)
    z.fsdp_checkpoint8_pack(x, *c)
    out = [torch.empty(r, k, device=DEV) for _ in range(4)]
    ws = torch.empty(z.fsdp_linear_dw_workspace(m, k), dtype=torch.uint8, device=DEV)
    z.fsdp_linear_dw(g, out[0], x8=c, workspace=ws)
    z.fsdp_linear_dw(g, out[1], x8=c)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    z.fsdp_linear_dw(g, out[2], x8=c, stream=side)
    z.fsdp_linear_dw(g, out[3], x8=c, stream=side.cuda_stream)
    side.synchronize()
    torch.cuda.synchronize()
    assert all(torch.equal(t, out[0]) for t in out[1:])
    with pytest.raises(z.ZeroError):
        z.fsdp_linear_dw(g, out[0], x8=c, workspace=ws[:-256])


@pytest.mark.parametrize("kind", ["z", "z8", "none"])
@pytest.mark.parametrize("rows,cols", [(4100, 1032), (531, 8200), (9, 524296), (70001, 64), (4106, 4104),
                                       (8200, 2056), (33, 524296), (16385, 1536), (401, 10248), (16401, 1032)])
def test_act_backward_large(z, rows, cols, kind):
    """Large matrices: past 2^24 elements, from 1024 columns on, the column sums go through a workspace,
    the caller's or the allocator's; without one, and else, they are summed in strips of any width."""
    act = {"z": "gelu_tanh", "z8": "silu", "none": "none"}[kind]
    dy, pre = randn(rows, cols, 0.3, 13), randn(rows, cols, 1.5, 14)
    arg, v = {}, pre.double()
    if kind == "z":
        arg = {"z": pre}
    elif kind == "z8":
        c = new8(rows, cols)
        z.fsdp_checkpoint8_pack(pre, *c)
        arg, v = {"z8": c}, values(z, c)
    zbuf, dz = guarded(rows, cols, BF, 3.0)
    bbuf, db = guarded(1, cols, torch.float32, 3.0)
    z.fsdp_act_backward(dy, dz, db=db[0], act=ACTS[act], **arg)
    z.zero_device_status()
    g = dy.double()
    want = g * dact64(v, act)
    e = g.abs() * act_err(v, act)[1] + SUM * want.abs()
    inside(dz, want, e + B16 * (want.abs() + e) + 2.0 ** -133, "dZ")
    inside(db[0], want.sum(0), e.sum(0) + (rows + 1) * SUM * want.abs().sum(0), "db")
    assert kept(zbuf, 3.0) and kept(bbuf, 3.0)
    nbytes = z.fsdp_act_backward_workspace(rows, cols)
    ws = torch.full((nbytes + 64,), 7, dtype=torch.uint8, device=DEV)
    db2 = torch.empty(cols, device=DEV)
    z.fsdp_act_backward(dy, db=db2, act=ACTS[act], workspace=ws[:nbytes] if nbytes else None, **arg)
    assert torch.equal(db2, db[0]) and bool((ws[nbytes:] == 7).all())
    # dZ alone, and dZ in dY's place
    dz2 = torch.empty_like(dz)
    z.fsdp_act_backward(dy, dz2, act=ACTS[act], **arg)
    assert torch.equal(dz2, dz)
    # through the C ABI without a workspace: the strips, another fixed order
    z.library().fsdp_act_backward(dy.data_ptr(), arg["z"].data_ptr() if "z" in arg else None,
                                  *([t.data_ptr() for t in arg["z8"]] if "z8" in arg else [None, None]), rows, cols,
                                  ACTS[act], dz2.data_ptr(), db2.data_ptr(), None, 0,
                                  torch.cuda.current_stream().cuda_stream)
    assert torch.equal(dz2, dz)
    inside(db2, want.sum(0), e.sum(0) + (rows + 1) * SUM * want.abs().sum(0), "db, strips")
    z.fsdp_act_backward(dy, dy, db=db2, act=ACTS[act], **arg)
    assert torch.equal(dy, dz) and torch.equal(db2, db[0])
    z.zero_device_status()
