"""The activation's backward through the C ABI without a workspace, at sizes where one would be used: the
column sums are summed in strips. Outputs start as NaN, and the call's code is looked at, so a call that
does nothing fails. Bounds as in test_linear_unit."""
from __future__ import annotations

import pytest
import torch

from test_linear_unit_wide import ACTS, B16, BF, DEV, SUM, act_err, dact64, guarded, inside, new8, randn, values, z  # noqa: F401

pytestmark = pytest.mark.gpu
NAN = float("nan")


def call(z, dy, arg, rows, cols, act, dz, db):  # noqa: F811
    codes = [t.data_ptr() for t in arg["z8"]] if "z8" in arg else [None, None]
    return z.library().fsdp_act_backward(dy.data_ptr(), arg["z"].data_ptr() if "z" in arg else None, *codes, rows, cols,
                                         ACTS[act], dz.data_ptr() if dz is not None else None,
                                         db.data_ptr() if db is not None else None, None, 0,
                                         torch.cuda.current_stream().cuda_stream)


def edges_are_nan(buf):
    return bool(torch.isnan(buf[:256]).all()) and bool(torch.isnan(buf[-256:]).all())


@pytest.mark.parametrize("kind,act", [("z", "gelu_tanh"), ("z", "relu"), ("z8", "silu"), ("z8", "gelu"), ("none", "none")])
@pytest.mark.parametrize("rows,cols", [(4106, 4104), (8200, 2056), (33, 524296), (16385, 1536), (16401, 1032),
                                       (2100, 8200)])
def test_without_a_workspace(z, rows, cols, kind, act):  # noqa: F811
    assert rows * cols > 1 << 24 and (z.fsdp_act_backward_workspace(rows, cols) > 0 or cols > 1 << 19)
    dy, pre = randn(rows, cols, 0.3, 41), randn(rows, cols, 1.5, 42)
    arg, v = {}, pre.double()
    if kind == "z":
        arg = {"z": pre}
    elif kind == "z8":
        c = new8(rows, cols)
        z.fsdp_checkpoint8_pack(pre, *c)
        arg, v = {"z8": c}, values(z, c)
    zbuf, dz = guarded(rows, cols, BF, NAN)
    bbuf, db = guarded(1, cols, torch.float32, NAN)
    assert call(z, dy, arg, rows, cols, act, dz, db[0]) == 0
    g = dy.double()
    want = g * dact64(v, act)
    e = g.abs() * act_err(v, act)[1] + SUM * want.abs()
    inside(dz, want, e + B16 * (want.abs() + e) + 2.0 ** -133, "dZ")
    inside(db[0], want.sum(0), e.sum(0) + (rows + 1) * SUM * want.abs().sum(0), "db")
    assert edges_are_nan(zbuf) and edges_are_nan(bbuf)
    # db alone, and again: the same bits
    for _ in range(2):
        alone = torch.full((cols,), NAN, device=DEV)
        assert call(z, dy, arg, rows, cols, act, None, alone) == 0
        assert torch.equal(alone, db[0])
    z.zero_device_status()
