"""The linear unit with its epilogue and the 8-bit activation checkpoints on the GPU, against
plain 64-bit implementations written here.

Bounds (derived, u = 2^-24 the unit roundoff of fp32, b = 2^-8 that of bf16):
  * a product's fp32 sum over K terms: (K + 1) 2^-23 sum |a b| (any order, rounding toward
    zero included), plus 2^-23 of the result for the bias, scale or residual operation;
  * an activation or derivative evaluated at v: the fast exponential's argument is rounded
    once more, so relative (2^-20 + |v| 2^-21) of the terms' magnitudes; the error of v itself
    passes through with the activation's slope (at most 1.2) or curvature (at most 1.2);
  * a bf16 output: b of its magnitude.
An 8-bit value is within half a step of the number it codes; pack and unpack are exact.
"""
from __future__ import annotations

import math

import numpy as np
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


# ---- plain 64-bit forms ----

def _sigmoid(x):
    """1 / (1 + exp(-x)), and so (1 + tanh(x / 2)) / 2 without its cancellation for x << 0."""
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-x))


GELU_A = 2.0 * math.sqrt(2.0 / math.pi)


def act64(x, act):
    if act == "relu":
        return np.where(x < 0, 0.0, x)
    if act == "gelu":
        return 0.5 * x * _erfc(-x / math.sqrt(2.0))
    if act == "gelu_tanh":
        return x * _sigmoid(GELU_A * (x + 0.044715 * x ** 3))
    if act == "silu":
        return x * _sigmoid(x)
    return x


def dact64(x, act):
    if act == "relu":
        return (x > 0).astype(np.float64)
    if act == "gelu":
        return 0.5 * _erfc(-x / math.sqrt(2.0)) + x * np.exp(-0.5 * x * x) / math.sqrt(2.0 * math.pi)
    if act == "gelu_tanh":
        u = GELU_A * (x + 0.044715 * x ** 3)
        s, q = _sigmoid(u), _sigmoid(-u)
        return s + x * s * q * GELU_A * (1.0 + 3 * 0.044715 * x * x)
    if act == "silu":
        return _sigmoid(x) * (1.0 + x * _sigmoid(-x))
    return np.ones_like(x)


def _erfc(x):
    return torch.erfc(torch.from_numpy(np.ascontiguousarray(x))).numpy()


def pack64(x):
    """(codes, scale bytes) of x [rows, cols], from the definition: the least byte in 1..248
    with amax < 127.5 * 2^(byte - 127), codes rounded to nearest, ties to even."""
    rows, cols = x.shape
    groups = -(-cols // G)
    p = np.zeros((rows, groups * G))
    p[:, :cols] = x
    p = p.reshape(rows, groups, G)
    finite = np.isfinite(p).all(-1)
    p = np.where(finite[..., None], p, 0.0)
    amax = np.abs(p).max(-1)
    byte = np.ones(amax.shape, dtype=np.int64)
    for b in range(1, 248):  # the least one that fits, by counting those that do not
        byte += amax >= 127.5 * 2.0 ** (b - 127)
    codes = np.clip(np.rint(p / 2.0 ** (byte[..., None] - 127.0)), -127, 127)
    byte = np.where(finite, byte, 255)
    return codes.reshape(rows, -1)[:, :cols].astype(np.int8), byte.astype(np.uint8)


def values64(codes, scales):
    s = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(np.float64) - 127.0))
    return codes.astype(np.float64) * np.repeat(s, G, axis=1)[:, :codes.shape[1]]


def f64(t):
    return t.detach().double().cpu().numpy()


def act_err(v, act):
    """Bound of |act_gpu(v) - act(v)| and of |act'_gpu(v) - act'(v)| (fp32 evaluation)."""
    a = np.abs(v)
    rel = 2.0 ** -20 + np.minimum(a, 90.0) * 2.0 ** -21
    if act in ("none", "relu"):
        return 0.0 * a, 0.0 * a
    return rel * np.abs(act64(v, act)) + 2.0 ** -120, rel * (1.0 + np.minimum(a, 90.0)) * np.exp(-np.clip(-v, 0, 80)) + 2.0 ** -120


def inside(got, want, bound, what):
    err = np.abs(got - want)
    bad = ~(err <= bound)
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} outside the bound; worst {np.nanmax(err - bound)} over at "
                           f"{np.unravel_index(np.nanargmax(np.where(bad, err, -1)), err.shape)}")


# ---- inputs ----

def randn(rows, cols, std, key, outliers=False):
    g = torch.Generator().manual_seed(synth.derive_seed(91, rows, cols, key))
    t = torch.randn(rows, cols, generator=g) * std
    if outliers:
        t[:, torch.randint(0, cols, (max(1, cols // 64),), generator=g)] *= 20.0
    return t.to(BF).to(DEV)


def guarded(rows, cols, dtype, fill):
    """A [rows, cols] tensor with 256 guard elements before and after, all `fill`."""
    buf = torch.full((rows * cols + 512,), fill, dtype=dtype, device=DEV)
    return buf, buf[256:256 + rows * cols].view(rows, cols)


def guards_kept(buf, fill):
    return bool((buf[:256] == fill).all()) and bool((buf[-256:] == fill).all())


def new8(z, rows, cols):
    return (torch.empty(rows, cols, dtype=torch.int8, device=DEV),
            torch.empty(rows, -(-cols // G), dtype=torch.uint8, device=DEV))


def checkpoint(z, t):
    c = new8(z, *t.shape)
    z.fsdp_checkpoint8_pack(t, *c)
    return c


# ---- 8-bit checkpoints ----

SHAPES8 = [(1, 8), (1, 32), (3, 40), (5, 72), (64, 96), (33, 1160), (257, 2304), (7, 4096)]


@pytest.mark.parametrize("rows,cols", SHAPES8)
def test_pack_and_unpack_are_exact(z, rows, cols):
    x = randn(rows, cols, 1.3, 1, outliers=True)
    x[:, ::7] *= 1e-3
    if rows > 2:
        x[1] = 0
    cbuf, codes = guarded(rows, cols, torch.int8, 99)
    sbuf, scales = guarded(rows, -(-cols // G), torch.uint8, 77)
    z.fsdp_checkpoint8_pack(x, codes, scales)
    want_c, want_s = pack64(f64(x))
    assert np.array_equal(codes.cpu().numpy(), want_c) and np.array_equal(scales.cpu().numpy(), want_s)
    assert guards_kept(cbuf, 99) and guards_kept(sbuf, 77)
    obuf, out = guarded(rows, cols, BF, 5.0)
    z.fsdp_checkpoint8_unpack(codes, scales, out)
    assert np.array_equal(f64(out), values64(want_c, want_s)) and guards_kept(obuf, 5.0)
    amax = np.abs(f64(x)).reshape(-1).max()
    assert np.abs(f64(out) - f64(x)).max() <= amax / 127.5


@pytest.mark.parametrize("act", sorted(ACTS))
@pytest.mark.parametrize("rows,cols", [(1, 8), (33, 1160), (70, 96)])
def test_unpack_with_activation(z, rows, cols, act):
    c = checkpoint(z, randn(rows, cols, 2.0, 2, outliers=True))
    out = torch.empty(rows, cols, dtype=BF, device=DEV)
    z.fsdp_checkpoint8_unpack(*c, out, act=ACTS[act])
    v = values64(c[0].cpu().numpy(), c[1].cpu().numpy())
    want = act64(v, act)
    e = act_err(v, act)[0]
    inside(f64(out), want, e + B16 * (np.abs(want) + e) + 2.0 ** -133, f"unpack {act}")


def test_checkpoint_extremes(z):
    """Every power of two of bf16, its largest numbers, subnormals, ties, and groups that hold
    an infinity or a NaN."""
    big = 3.3895313892515355e38  # the largest finite bf16
    rows = []
    for e in range(-133, 128):
        rows.append([math.ldexp(1.0, e) * f for f in (1.0, -1.0, 0.5, 0.75, 1.9921875, -1.9921875, 1.984375, 0.0)] * 8)
    x = torch.tensor(rows, dtype=torch.float64).clamp(-big, big).to(BF)
    extra = torch.zeros(6, 64, dtype=BF)
    extra[0, 3], extra[1, 40], extra[2, 63] = float("inf"), float("-inf"), float("nan")
    extra[2, 5] = 3.0
    extra[3, :] = torch.tensor(big, dtype=BF)
    extra[4, :] = torch.arange(64).to(BF) * 0.25 + 96.0  # ties at a step of 1
    x = torch.cat([x, extra]).to(DEV)
    c = checkpoint(z, x)
    want_c, want_s = pack64(f64(x))
    assert np.array_equal(c[1].cpu().numpy(), want_s)
    assert np.array_equal(c[0].cpu().numpy(), want_c)
    out = torch.empty_like(x)
    z.fsdp_checkpoint8_unpack(*c, out)
    want = values64(want_c, want_s)
    assert np.array_equal(f64(out), want, equal_nan=True)
    nan = torch.isnan(out).cpu()
    assert nan[-6, :32].all() and not nan[-6, 32:].any() and nan[-5, 32:].all() and nan[-4, 32:].all()
    assert not nan[:-6].any() and not nan[-3:].any() and torch.isfinite(out[-3:]).all()
    # the NaN groups stay NaN through every activation and derivative
    for act in ACTS.values():
        z.fsdp_checkpoint8_unpack(*c, out, act=act)
        assert torch.isnan(out[-6, :32]).all() and torch.isnan(out[-4, 32:]).all()
        if act:
            dy, dz = torch.ones_like(x), torch.empty_like(x)
            z.fsdp_act_backward(dy, dz, z8=c, act=act)
            assert torch.isnan(dz[-6, :32]).all() and not torch.isnan(dz[:-6]).any()


# ---- activation backward ----

@pytest.mark.parametrize("kind", ["z", "z8"])
@pytest.mark.parametrize("act", sorted(ACTS))
@pytest.mark.parametrize("rows,cols", [(1, 8), (2, 136), (31, 40), (1003, 264), (300, 1160)])
def test_act_backward(z, rows, cols, act, kind):
    dy, pre = randn(rows, cols, 0.3, 3), randn(rows, cols, 1.7, 4, outliers=True)
    kept = {"z": pre} if kind == "z" else {"z8": checkpoint(z, pre)}
    v = f64(pre) if kind == "z" else values64(*[t.cpu().numpy() for t in kept["z8"]])
    zbuf, dz = guarded(rows, cols, BF, 3.0)
    bbuf, db = guarded(1, cols, torch.float32, 3.0)
    z.fsdp_act_backward(dy, dz, db=db[0], act=ACTS[act], **kept)
    g = f64(dy)
    want = g * dact64(v, act)
    e = np.abs(g) * act_err(v, act)[1] + 2.0 ** -23 * np.abs(want)
    inside(f64(dz), want, e + B16 * (np.abs(want) + e) + 2.0 ** -133, f"dZ {act} {kind}")
    inside(f64(db[0]), want.sum(0), e.sum(0) + (rows + 1) * SUM * np.abs(want).sum(0), f"db {act} {kind}")
    assert guards_kept(zbuf, 3.0) and guards_kept(bbuf, 3.0)
    # either output alone, dZ in dY's place, and a second call: the same bits
    dz2, db2 = torch.empty_like(dz), torch.empty(cols, device=DEV)
    z.fsdp_act_backward(dy, db=db2, act=ACTS[act], **kept)
    z.fsdp_act_backward(dy, dz2, act=ACTS[act], **kept)
    assert torch.equal(db2, db[0]) and torch.equal(dz2, dz)
    z.fsdp_act_backward(dy, dy, db=db2, act=ACTS[act], **kept)
    assert torch.equal(db2, db[0]) and torch.equal(dy, dz)


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
def test_act_backward_against_differences(z, act):
    """Central differences of the 64-bit activation, h = 1e-4: off by h^2 / 6 times the third
    derivative (below 4 for these), and by the cancellation 1e-16 |act| / h."""
    x = torch.linspace(-9, 9, 4096).view(64, 64).to(BF).to(DEV)
    dz = torch.empty_like(x)
    z.fsdp_act_backward(torch.ones_like(x), dz, z=x, act=ACTS[act])
    v, h = f64(x), 1e-4
    diff = (act64(v + h, act) - act64(v - h, act)) / (2 * h)
    e = act_err(v, act)[1] + 4 * h * h / 6 + 1e-15 * np.abs(v) / h
    inside(f64(dz), diff, e + B16 * (np.abs(diff) + e), f"difference {act}")


@pytest.mark.parametrize("act", sorted(ACTS))
def test_act_extreme_arguments(z, act):
    """Large finite pre-activations (where x^3, exp or x^2 overflow) keep finite, right
    gradients and outputs."""
    vals = [1e4, 1e10, 1e20, 3e38, 60.0, 100.0, 88.5, 1e-30, 1e-40, 0.0, 20.0, 12.0]
    x = torch.tensor(vals + [-a for a in vals], dtype=torch.float64).to(BF).to(DEV).view(1, 24)
    dz = torch.empty_like(x)
    z.fsdp_act_backward(torch.ones_like(x), dz, z=x, act=ACTS[act])
    with np.errstate(over="ignore", invalid="ignore"):
        want = dact64(np.clip(f64(x), -100, 100), act)
    assert torch.isfinite(dz).all()
    inside(f64(dz), want, 1e-5 + B16 * np.abs(want), f"grad {act}")
    # the forward on the same numbers: X W^T with W the identity
    eye = torch.eye(24, dtype=BF, device=DEV)
    y = torch.empty(1, 24, dtype=BF, device=DEV)
    z.fsdp_linear_forward([eye], x, y, act=ACTS[act])
    with np.errstate(over="ignore", invalid="ignore"):
        want = np.where(f64(x) > 50, f64(x), act64(np.clip(f64(x), -100, 50), act))
        if act == "none":
            want = f64(x)
    assert torch.isfinite(y).all()
    inside(f64(y), want, 1e-5 + 2.0 ** -7 * np.abs(want), f"value {act}")


# ---- forward ----

def shards_of(r, k, n, key):
    return [randn(r // n, k, 0.05, key + 7 * i) for i in range(n)]


# (m, r, k, n): ragged in every dimension; shards of 8 .. 296 rows; one token to several tiles
SHAPES = [(1, 8, 8, 1), (1, 1024, 512, 8), (3, 136, 72, 1), (5, 40, 520, 5), (17, 128, 64, 16), (64, 256, 128, 2),
          (127, 264, 200, 1), (128, 512, 256, 8), (129, 768, 320, 8), (130, 2304, 96, 8), (255, 1160, 136, 5),
          (300, 320, 1032, 4), (520, 592, 264, 2), (1, 2048, 4096, 8), (33, 264, 2056, 3), (770, 1184, 72, 4)]


def product64(x, shards):
    xa, w = f64(x), np.concatenate([f64(s) for s in shards])
    return xa @ w.T, (xa.shape[1] + 1) * SUM * (np.abs(xa) @ np.abs(w).T)


@pytest.mark.parametrize("kind", ["z", "z8", "none"])
@pytest.mark.parametrize("m,r,k,n", SHAPES)
def test_forward(z, m, r, k, n, kind):
    i = SHAPES.index((m, r, k, n))
    act = sorted(ACTS)[(i + {"z": 0, "z8": 1, "none": 2}[kind]) % 5]
    has_bias, has_res = i % 2 == 0 or kind == "z8", i % 3 != 0
    x, shards = randn(m, k, 1.0, 5), shards_of(r, k, n, 6)
    bias = randn(1, r, 0.5, 8)[0].contiguous() if has_bias else None
    res = randn(m, r, 2.0, 9) if has_res else None
    ybuf, y = guarded(m, r, BF, 3.0)
    zbuf, zk = guarded(m, r, BF, 3.0)
    cbuf, codes = guarded(m, r, torch.int8, 99)
    sbuf, scales = guarded(m, -(-r // G), torch.uint8, 77)
    keep = {"z": {"z": zk}, "z8": {"z8": (codes, scales)}, "none": {}}[kind]
    z.fsdp_linear_forward(shards, x, y, bias=bias, act=ACTS[act], residual=res, **keep)
    z.zero_device_status()
    pre, ez = product64(x, shards)
    if has_bias:
        pre = pre + f64(bias)
        ez = ez + SUM * np.abs(pre)
    want = act64(pre, act)
    e = 1.2 * ez + act_err(pre, act)[0]
    if has_res:
        want = want + f64(res)
        e = e + SUM * np.abs(want)
    inside(f64(y), want, e + B16 * (np.abs(want) + e) + 2.0 ** -133, f"Y {act}")
    assert guards_kept(ybuf, 3.0) and guards_kept(zbuf, 3.0) and guards_kept(cbuf, 99) and guards_kept(sbuf, 77)
    if kind == "z":
        inside(f64(zk), pre, ez + B16 * (np.abs(pre) + ez) + 2.0 ** -133, "Z")
    if kind == "z8":
        s = scales.cpu().numpy()
        pad = -r % G
        mag = np.pad(np.abs(pre), ((0, 0), (0, pad))).reshape(m, -1, G)
        slack = np.pad(ez, ((0, 0), (0, pad))).reshape(m, -1, G)
        step = 2.0 ** (s.astype(np.float64) - 127.0)
        # the byte of a largest magnitude within the sums' error: it fits, and a smaller one would not
        assert np.all((mag - slack).max(-1) < 127.5 * step)
        assert np.all((s == 1) | ((mag + slack).max(-1) >= 127.5 * step / 2))
        half = np.repeat(step / 2, G, axis=1)[:, :r]
        inside(values64(codes.cpu().numpy(), s), pre, half + ez, "Z in 8 bits")
    # the same bits again, and on another stream
    y2 = torch.empty_like(y)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    z.fsdp_linear_forward(shards, x, y2, bias=bias, act=ACTS[act], residual=res, stream=side)
    side.synchronize()
    assert torch.equal(y, y2)


def test_forward_non_finite_inputs_stay_in_their_rows(z):
    """A token row with a NaN, or with infinities, changes no other row; a NaN weight row no
    other column; the checkpoint marks exactly the groups that hold one."""
    m, r, k = 200, 328, 136
    x, shards = randn(m, k, 1.0, 10), shards_of(r, k, 1, 11)
    clean = torch.empty(m, r, dtype=BF, device=DEV)
    z.fsdp_linear_forward(shards, x, clean, act=ACTS["silu"])
    bad = x.clone()
    bad[7, 135], bad[130, 0] = float("nan"), float("inf")
    w = shards[0].clone()
    w[40, 3] = float("nan")
    y, c = torch.empty_like(clean), new8(z, m, r)
    z.fsdp_linear_forward([w], bad, y, act=ACTS["silu"], z8=c)
    z.zero_device_status()
    rows = [i for i in range(m) if i not in (7, 130)]
    cols = [j for j in range(r) if j != 40]
    assert torch.equal(y[rows][:, cols], clean[rows][:, cols])
    assert not torch.isfinite(y[130]).any()
    s = c[1].cpu()
    assert (s[7] == 255).all() and (s[130] == 255).all() and (s[:, 1] == 255).all()
    assert (s[rows][:, [0] + list(range(2, s.shape[1]))] != 255).all()
    assert torch.isnan(y[7]).all() and torch.isnan(y[:, 40]).all()


# ---- input gradient ----

@pytest.mark.parametrize("kind", ["z", "z8"])
@pytest.mark.parametrize("m,r,k,n", SHAPES)
def test_dx(z, m, r, k, n, kind):
    i = SHAPES.index((m, r, k, n))
    act = sorted(ACTS)[(i + (kind == "z8")) % 5]
    dzv, shards = randn(m, r, 0.3, 12), shards_of(r, k, n, 13)
    pre = randn(m, k, 1.5, 14)
    kept = {"z": pre} if kind == "z" else {"z8": checkpoint(z, pre)}
    res = randn(m, k, 0.5, 15) if i % 2 else None
    buf, dx = guarded(m, k, BF, 3.0)
    z.fsdp_linear_dx(shards, dzv, dx, act=ACTS[act], residual=res, **kept)
    z.zero_device_status()
    v = f64(pre) if kind == "z" else values64(*[t.cpu().numpy() for t in kept["z8"]])
    w, g = np.concatenate([f64(s) for s in shards]), f64(dzv)
    acc, ea = g @ w, (r + 1) * SUM * (np.abs(g) @ np.abs(w))
    d, ed = dact64(v, act), act_err(v, act)[1]
    want = acc * d
    e = ea * (np.abs(d) + ed) + np.abs(acc) * ed + SUM * np.abs(want)
    if res is not None:
        want = want + f64(res)
        e = e + SUM * np.abs(want)
    inside(f64(dx), want, e + B16 * (np.abs(want) + e) + 2.0 ** -133, f"dX {act} {kind}")
    assert guards_kept(buf, 3.0)


def test_dx_against_differences(z):
    """dX . V against the central difference of the 64-bit loss sum(dY * act(X W^T + b)) along
    V, the two calls (activation backward, input gradient) as a user chains them. The loss is
    smooth: h^2 and cancellation are far below the bf16 roundings of dZ and dX, each b of the
    terms they round."""
    m, r, k, n = 37, 96, 72, 2
    x, shards = randn(m, k, 1.0, 16), shards_of(r, k, n, 17)
    bias, dy = randn(1, r, 0.5, 18)[0].contiguous(), randn(m, r, 1.0, 19)
    y, pre = torch.empty(m, r, dtype=BF, device=DEV), torch.empty(m, r, dtype=BF, device=DEV)
    z.fsdp_linear_forward(shards, x, y, bias=bias, act=ACTS["gelu_tanh"], z=pre)
    dzv, dx, db = torch.empty_like(dy), torch.empty_like(x), torch.empty(r, device=DEV)
    z.fsdp_act_backward(dy, dzv, db=db, z=pre, act=ACTS["gelu_tanh"])
    z.fsdp_linear_dx(shards, dzv, dx)
    w = np.concatenate([f64(s) for s in shards])
    g, xa, b = f64(dy), f64(x), f64(bias)

    def loss(xx, bb):
        return (g * act64(xx @ w.T + bb, "gelu_tanh")).sum()

    rng = np.random.default_rng(3)
    v, vb, h = rng.standard_normal(xa.shape), rng.standard_normal(b.shape), 1e-4
    d64 = g * dact64(xa @ w.T + b, "gelu_tanh")
    # Z was kept in bf16: its rounding moves act' by at most 1.2 b |Z|; then dZ and dX round
    zr = 2 * B16 * np.abs(xa @ w.T + b)
    ez = np.abs(g) * (1.2 * zr + 1e-5) + B16 * np.abs(d64)
    diff = (loss(xa + h * v, b) - loss(xa - h * v, b)) / (2 * h)
    bound = ((ez @ np.abs(w) + B16 * np.abs(d64 @ w) + r * SUM * (np.abs(d64) @ np.abs(w))) * np.abs(v)).sum() + 1e-3
    assert abs((f64(dx) * v).sum() - diff) <= bound
    diff = (loss(xa, b + h * vb) - loss(xa, b - h * vb)) / (2 * h)
    assert abs((f64(db) * vb).sum() - diff) <= (ez.sum(0) * np.abs(vb)).sum() + 1e-3


# ---- weight gradient ----

@pytest.mark.parametrize("wide", [True, False])
@pytest.mark.parametrize("kind", ["x", "x8"])
@pytest.mark.parametrize("m,r,k,n", SHAPES)
def test_dw(z, m, r, k, n, kind, wide):
    dzv, x = randn(m, r, 0.3, 20), randn(m, k, 1.0, 21, outliers=True)
    kept = {"x": x} if kind == "x" else {"x8": checkpoint(z, x)}
    v = f64(x) if kind == "x" else values64(*[t.cpu().numpy() for t in kept["x8"]])
    scale = 1.0 / 3.0 if wide else 0.125
    buf, dw = guarded(r, k, torch.float32 if wide else BF, 3.0)
    z.fsdp_linear_dw(dzv, dw, scale=scale, **kept)
    z.zero_device_status()
    g, s = f64(dzv), float(np.float32(scale))
    want = s * (g.T @ v)
    e = (m + 1) * SUM * s * (np.abs(g).T @ np.abs(v)) + SUM * np.abs(want)
    inside(f64(dw), want, e if wide else e + B16 * (np.abs(want) + e) + 2.0 ** -133, f"dW {kind}")
    assert guards_kept(buf, 3.0)
    again = torch.empty_like(dw)
    z.fsdp_linear_dw(dzv, again, scale=scale, **kept)
    assert torch.equal(dw, again)


def test_dw_long_sum_stays_accurate(z):
    """fp32 weight gradients over many tokens: the error stays at fp32's level (2^-16 of the
    result's norm is 256 roundings' worth) however long the sum over tokens."""
    m, r, k = 16384, 136, 264
    dzv, x = randn(m, r, 0.3, 22), randn(m, k, 1.0, 23)
    for kept, v in (({"x": x}, f64(x)), ({"x8": checkpoint(z, x)}, None)):
        if v is None:
            v = values64(*[t.cpu().numpy() for t in kept["x8"]])
        dw = torch.empty(r, k, device=DEV)
        z.fsdp_linear_dw(dzv, dw, **kept)
        want = f64(dzv).T @ v
        assert np.linalg.norm(f64(dw) - want) <= 2.0 ** -16 * np.linalg.norm(want)


def test_dw_non_finite_tokens(z):
    """A NaN in one column of dZ or X reaches its row or column of dW and nothing else."""
    m, r, k = 70, 136, 72
    dzv, x = randn(m, r, 0.3, 24), randn(m, k, 1.0, 25)
    dzv[69, 135], x[0, 71] = float("nan"), float("nan")
    dw = torch.empty(r, k, device=DEV)
    z.fsdp_linear_dw(dzv, dw, x=x)
    nan = torch.isnan(dw).cpu()
    assert nan[135].all() and nan[:, 71].all() and not nan[:135, :71].any()
    c = checkpoint(z, x)
    z.fsdp_linear_dw(dzv, dw, x8=c)
    nan = torch.isnan(dw).cpu()
    assert nan[135].all() and nan[:, 64:].all() and not nan[:135, :64].any()


# ---- large offsets, a tile band at full size ----

def test_offsets_past_32_bits(z):
    """More than 2^31 elements in every streaming call, and more than 2^31 outputs of a
    forward: the last rows equal a small call on the same rows."""
    rows, cols, tail = 262_200, 8_208, 40
    gen = torch.Generator(device=DEV).manual_seed(5)
    x = torch.empty(rows, cols, dtype=BF, device=DEV)
    x[:64] = 1.0
    x[-tail:] = torch.randn(tail, cols, generator=gen, device=DEV).to(BF)
    assert x.numel() > 2 ** 31
    last = x[-tail:].clone()
    c, small = new8(z, rows, cols), new8(z, tail, cols)
    z.fsdp_checkpoint8_pack(x, *c)
    z.fsdp_checkpoint8_pack(last, *small)
    assert torch.equal(c[0][-tail:], small[0]) and torch.equal(c[1][-tail:], small[1])
    out, o2 = torch.empty_like(x), torch.empty_like(last)
    z.fsdp_checkpoint8_unpack(*c, out, act=ACTS["silu"])
    z.fsdp_checkpoint8_unpack(*small, o2, act=ACTS["silu"])
    assert torch.equal(out[-tail:], o2)
    z.fsdp_act_backward(x, out, z8=c, act=ACTS["silu"])
    z.fsdp_act_backward(last, o2, z8=small, act=ACTS["silu"])
    assert torch.equal(out[-tail:], o2)
    del c
    w = randn(cols, 8, 0.1, 26)
    xs = randn(rows, 8, 1.0, 27)
    codes = new8(z, rows, cols)
    z.fsdp_linear_forward([w], xs, out, act=ACTS["gelu"], residual=x, z8=codes)
    small = new8(z, tail, cols)
    z.fsdp_linear_forward([w], xs[-tail:].clone(), o2, act=ACTS["gelu"], residual=last, z8=small)
    assert torch.equal(out[-tail:], o2)
    assert torch.equal(codes[0][-tail:], small[0]) and torch.equal(codes[1][-tail:], small[1])
    z.zero_device_status()


@pytest.mark.parametrize("m,r,k,n", [(2048, 4096, 1024, 8), (1000, 2304, 768, 8), (2041, 768, 768, 1)])
def test_several_tiles_against_float64_on_the_gpu(z, m, r, k, n):
    """Sizes with many tiles per block: every output of the three products against float64
    products on the GPU (torch), the same bounds."""
    x, shards = randn(m, k, 1.0, 28), shards_of(r, k, n, 29)
    w = torch.cat(shards).double()
    y = torch.empty(m, r, dtype=BF, device=DEV)
    z.fsdp_linear_forward(shards, x, y)
    want = x.double() @ w.T
    e = (k + 1) * SUM * (x.double().abs() @ w.abs().T)
    assert ((y.double() - want).abs() <= e + B16 * (want.abs() + e)).all()
    g = randn(m, r, 0.3, 30)
    dx = torch.empty(m, k, dtype=BF, device=DEV)
    z.fsdp_linear_dx(shards, g, dx)
    want = g.double() @ w
    e = (r + 1) * SUM * (g.double().abs() @ w.abs())
    assert ((dx.double() - want).abs() <= e + B16 * (want.abs() + e)).all()
    for kept, v in (({"x": x}, x.double()), ({"x8": checkpoint(z, x)}, None)):
        if v is None:
            vals = torch.empty_like(x)
            z.fsdp_checkpoint8_unpack(*kept["x8"], vals)
            v = vals.double()
        dw = torch.empty(r, k, device=DEV)
        z.fsdp_linear_dw(g, dw, **kept)
        want = g.double().T @ v
        e = (m + 2) * SUM * (g.double().abs().T @ v.abs())
        assert ((dw.double() - want).abs() <= e).all()
    z.zero_device_status()


def test_binding_refuses_wrong_tensors(z):
    """Wrong shapes, types, devices and strides are Python errors before anything is launched."""
    m, r, k = 16, 64, 32
    x, shards, y = randn(m, k, 1.0, 31), shards_of(r, k, 2, 32), torch.empty(m, r, dtype=BF, device=DEV)
    with pytest.raises(ValueError):
        z.fsdp_linear_forward(shards, x[:, :24], y)
    with pytest.raises(ValueError):
        z.fsdp_linear_forward(shards, x, y.t())
    with pytest.raises(ValueError):
        z.fsdp_linear_forward(shards, x, torch.empty(m - 1, r, dtype=BF, device=DEV))
    with pytest.raises(TypeError):
        z.fsdp_linear_forward(shards, x.float(), y)
    with pytest.raises(ValueError):
        z.fsdp_linear_forward(shards, x.cpu(), y)
    with pytest.raises(ValueError):
        z.fsdp_linear_forward(shards, x, y, bias=torch.zeros(r - 1, dtype=BF, device=DEV))
    with pytest.raises(ValueError):
        z.fsdp_checkpoint8_pack(x, torch.empty(m, k, dtype=torch.int8, device=DEV),
                                torch.empty(m, 2, dtype=torch.uint8, device=DEV))
    with pytest.raises(TypeError):
        z.fsdp_linear_dw(y, torch.empty(r, k, dtype=torch.float16, device=DEV), x=x)
    with pytest.raises(z.ZeroError):
        z.fsdp_linear_forward(shards, x, y, act=9)
    z.zero_device_status()
