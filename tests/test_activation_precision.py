"""How near the activations' derivatives come in fp32, at every finite bf16 pre-activation: db of one row of
dY = 1 is the unrounded derivative.

With a the argument of the exponential (SILU |x|, GELU_TANH the |2 u| of its tanh u, GELU x^2 / 2): it is
rounded up to four times, 2^-24 of it each, and twice that through h^2 in the sigmoid, so the exponential is
off by at most |a| 2^-22, and by 2^-20 from the fast exponential, reciprocal and the offset in its argument.
Below 0 the derivative is the gate g (1 / (1 + e^-x), .., Phi) times terms of at most 1 + 3 |a| that are off
by as much; from 0 on the gate's distance from 1 is off by at most 2^-23, times at most 1 + 3 |a| with |a| <
17.4 (past that the gate is 1): 2^-17. Below 2^-115 fp32 may have lost the number.

And what a value past the largest code of the largest scale byte becomes."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from test_linear_unit import ACTS, DEV, GELU_A, _erfc, _sigmoid, dact64, f64, z  # noqa: F401

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.mark.parametrize("kind", ["z", "z8"])
@pytest.mark.parametrize("act", ["relu", "gelu", "gelu_tanh", "silu"])
def test_derivative_in_fp32(z, act, kind):  # noqa: F811
    every = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16).view(BF)
    x = every[torch.isfinite(every)].to(DEV).view(1, -1)
    assert x.shape[1] == 255 * 256
    kept = {"z": x}
    if kind == "z8":  # codes -127 .. 127 at the scales 2^-12 .. 2^1
        codes = torch.arange(-127, 129).clamp(max=127).to(torch.int8).repeat(14).view(1, -1).to(DEV)
        scales = torch.arange(115, 129, dtype=torch.uint8).repeat_interleave(8).view(1, -1).to(DEV)
        kept = {"z8": (codes, scales)}
        x = torch.empty(codes.shape, dtype=BF, device=DEV)
        z.fsdp_checkpoint8_unpack(codes, scales, x)
    db = torch.full((x.shape[1],), float("nan"), device=DEV)
    z.fsdp_act_backward(torch.ones_like(x), db=db, act=ACTS[act], **kept)
    v = f64(x)[0]
    c = np.clip(v, -1e3, 1e3)  # past it every derivative is 0 or 1
    with np.errstate(over="ignore", under="ignore"):
        want = dact64(c, act)
        if act == "relu":
            assert np.array_equal(f64(db), want)
            return
        a = {"silu": np.abs(c), "gelu_tanh": np.abs(GELU_A * (c + 0.044715 * c ** 3)), "gelu": 0.5 * c * c}[act]
        g = {"silu": _sigmoid(c), "gelu_tanh": _sigmoid(GELU_A * (c + 0.044715 * c ** 3)),
             "gelu": 0.5 * _erfc(-c / np.sqrt(2.0))}[act]
    a = np.minimum(a, 90.0)
    bound = np.where(c < 0, (2.0 ** -20 + a * 2.0 ** -22) * (1 + 3 * a) * g + 2.0 ** -115, 2.0 ** -17)
    err = np.abs(f64(db) - want)
    i = int(np.argmax(err - bound))
    assert (err <= bound).all(), f"{act} at {v[i]}: off by {err[i]:.3e}, bound {bound[i]:.3e}"


@pytest.mark.parametrize("m", [1, 700])
def test_z_past_the_largest_code(z, m):  # noqa: F811
    """fp32 Z of 255.875 * 2^120, past 127.5 * 2^121: byte 248 is the largest, the code 127, so the value
    read back is 254 * 2^120, off by less than a whole step of 2^121 instead of half of one."""
    r, k = 40, 8
    x = torch.zeros(m, k, dtype=BF, device=DEV)
    x[:, 0] = 255.0 * 2.0 ** 120
    w = torch.zeros(r, k, dtype=BF, device=DEV)
    w[:, 0] = torch.tensor([1.0, -1.0] * (r // 2)).to(BF)
    bias = (w[:, 0].float() * 1.75 * 2.0 ** 119).to(BF)
    y = torch.empty(m, r, dtype=BF, device=DEV)
    c = torch.empty(m, r, dtype=torch.int8, device=DEV), torch.empty(m, 2, dtype=torch.uint8, device=DEV)
    z.fsdp_linear_forward([w], x, y, bias=bias, z8=c)
    z.zero_device_status()
    out = torch.empty_like(y)
    z.fsdp_checkpoint8_unpack(*c, out)
    assert (c[1] == 248).all() and torch.equal(c[0].float(), 127.0 * w[:, 0].float().expand(m, r))
    err = (out.double() - w[:, 0].double() * 255.875 * 2.0 ** 120).abs()
    assert (err == 1.875 * 2.0 ** 120).all() and (err < 2.0 ** 121).all()
