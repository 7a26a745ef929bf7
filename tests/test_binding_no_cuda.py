"""The binding on a PyTorch without CUDA and on a machine without a driver: it imports, what needs no device
works, and tensors that are not on a GPU are refused by name, as they are where there is one. No GPU."""
from __future__ import annotations

import os
import subprocess
import sys

import pytest
import torch

BF = torch.bfloat16
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def z():
    import __graft_entry__ as g
    g.build()
    import fsdp_sharded_optimizer_zero_gb300 as z
    return z


def t(*shape, dtype=BF):
    return torch.zeros(*shape, dtype=dtype)


def z8(m, k):
    return t(m, k, dtype=torch.int8), t(m, -(-k // 32), dtype=torch.uint8)


CALLS = {
    "gather_rows": lambda z: z.fsdp_gather_rows([t(8, 16), t(8, 16)], t(16, 16)),
    "unit_forward": lambda z: z.fsdp_unit_forward([t(128, 64)], t(4, 64), t(4, 128, dtype=torch.float32)),
    "linear_forward": lambda z: z.fsdp_linear_forward([t(8, 16), t(8, 16)], t(4, 16), t(4, 16)),
    "linear_dx": lambda z: z.fsdp_linear_dx([t(8, 16)], t(4, 8), t(4, 16)),
    "linear_dw": lambda z: z.fsdp_linear_dw(t(4, 8), t(8, 16, dtype=torch.float32), x=t(4, 16)),
    "linear_dw from 8 bits": lambda z: z.fsdp_linear_dw(t(4, 8), t(8, 16), x8=z8(4, 16)),
    "act_backward": lambda z: z.fsdp_act_backward(t(4, 16), t(4, 16), z=t(4, 16), act=z.FSDP_ACT_RELU),
    "pack": lambda z: z.fsdp_checkpoint8_pack(t(4, 16), *z8(4, 16)),
    "unpack": lambda z: z.fsdp_checkpoint8_unpack(*z8(4, 16), t(4, 16)),
}


@pytest.mark.parametrize("name", sorted(CALLS))
def test_host_tensors_are_refused_by_name(z, name):
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        CALLS[name](z)


def test_imports_without_the_private_names(z):
    """A PyTorch built without CUDA has none of torch._C's _cuda_ functions."""
    code = """
import torch
for name in [n for n in dir(torch._C) if n.startswith("_cuda_")]:
    delattr(torch._C, name)
import fsdp_sharded_optimizer_zero_gb300 as z
assert z.zero_plan(1000, 4, "zero2", 1 << 20).layout["psi_padded"] >= 1000
assert z.fsdp_linear_dw_workspace(4, 16) == 256
x = torch.zeros(4, 16, dtype=torch.bfloat16)
for call in (lambda: z.fsdp_linear_forward([x], x, x), lambda: z.fsdp_gather_rows([x], x)):
    try:
        call()
    except ValueError as e:
        assert "must be a CUDA tensor" in str(e), e
    else:
        raise AssertionError("a host tensor was accepted")
print("fine")
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "fine" in r.stdout, r.stderr[-2000:]


def test_the_public_way_without_the_private_names(z, monkeypatch):
    """With CUDA but other private names: the current stream by torch.cuda, devices checked tensor by
    tensor."""
    monkeypatch.delattr(torch._C, "_cuda_getDevice")

    class Stream:
        cuda_stream = 4321

    monkeypatch.setattr(torch.cuda, "current_stream", Stream)
    assert z._lib._stream(None) == 4321 and z._lib._stream(7) == 7 and z._lib._stream(Stream()) == 4321
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        CALLS["linear_forward"](z)
