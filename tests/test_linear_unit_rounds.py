"""The forward's wide kernel where every CTA pair takes many tiles: the biases that four epilogue warps
share, copied at each tile, are the right ones; and no wait for other warps of a role is open-ended."""
from __future__ import annotations

import re
from pathlib import Path

import pytest
import torch

from test_linear_unit_wide import B16, SUM, act_err, act64, apart, inside, randn, z  # noqa: F401

CSRC = Path(__file__).resolve().parents[1] / "fsdp_sharded_optimizer_zero_gb300" / "csrc"
DEV = "cuda"


@pytest.mark.parametrize("name", ["fsdp_linear.cu", "fsdp_gemm.cu", "tcgen05.cuh", "device_common.cuh"])
def test_warps_of_a_role_meet_only_where_they_agree_on_leaving(name):
    """A role's loops end when a bounded wait gives up, which its warps may see at different tiles: at a
    named barrier that only counts threads, one that goes on would wait for good for one that has left.
    (A GPU wait that never ends is not provoked to show it: the source has no such barrier.)"""
    code = re.sub(r"//[^\n]*", "", (CSRC / name).read_text())
    assert not re.findall(r'"[^"]*\b(?:bar|barrier)(?:\.cta)?\.(?:sync|arrive)\b[^"]*"', code)


@pytest.mark.gpu
@pytest.mark.parametrize("m,r,k,n,act,res", [(8192, 4112, 64, 1, "none", False), (8200, 4096, 128, 8, "silu", True),
                                             (6001, 5000, 72, 5, "relu", False)])
def test_biases_over_many_tiles_of_a_pair(z, m, r, k, n, act, res):  # noqa: F811
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert -(-m // 256) * -(-r // 256) >= 6 * (sms // 2)
    x, w = randn(m, k, 1.0, 31), randn(r, k, 0.04, 32)
    bias = randn(1, r, 4.0, 33)[0].contiguous()  # of a tile's columns: no two alike
    rs = randn(m, r, 2.0, 34) if res else None
    y = torch.empty(m, r, dtype=torch.bfloat16, device=DEV)
    code = {"none": z.FSDP_ACT_NONE, "relu": z.FSDP_ACT_RELU, "silu": z.FSDP_ACT_SILU}[act]
    z.fsdp_linear_forward(apart(w, n), x, y, bias=bias, act=code, residual=rs)
    z.zero_device_status()
    x64, w64 = x.double(), w.double()
    pre = x64 @ w64.T + bias.double()
    ez = (k + 1) * SUM * (x64.abs() @ w64.abs().T) + SUM * pre.abs()
    want, e = act64(pre, act), 1.2 * ez + act_err(pre, act)[0]
    if res:
        want = want + rs.double()
        e = e + SUM * want.abs()
    inside(y, want, e + B16 * (want.abs() + e), f"Y {act}")
    for _ in range(4):
        again = torch.full_like(y, float("nan"))
        z.fsdp_linear_forward(apart(w, n), x, again, bias=bias, act=code, residual=rs)
        assert torch.equal(again, y)
