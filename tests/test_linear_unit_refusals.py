"""Argument errors of the linear-unit and 8-bit checkpoint calls through the C ABI: each is
ZERO_ERR_INVALID_ARG with a message, found on the host before anything is launched. No GPU:
the pointers are made up and never read."""
from __future__ import annotations

import ctypes as C

import pytest

P = 1 << 20  # a 16-byte-aligned address that is never dereferenced


@pytest.fixture(scope="module")
def z():
    import __graft_entry__ as g
    g.build()
    import fsdp_sharded_optimizer_zero_gb300 as z
    return z


def refused(z, rc, word):
    assert rc == -1
    msg = z.zero_last_error()
    assert word in msg, msg


def shards(n, p=P):
    return (C.c_void_p * n)(*[p] * n)


def forward(z, **kw):
    a = dict(n=2, w=shards(2), r=64, k=32, x=P, m=4, bias=None, act=0, res=None, y=P, zz=None, zc=None, zs=None)
    a.update(kw)
    return z.library().fsdp_linear_forward(a["n"], a["w"], a["r"], a["k"], a["x"], a["m"], a["bias"], a["act"],
                                           a["res"], a["y"], a["zz"], a["zc"], a["zs"], None)


def dx(z, **kw):
    a = dict(n=2, w=shards(2), r=64, k=32, dz=P, m=4, zz=P, zc=None, zs=None, act=1, res=None, dx=P)
    a.update(kw)
    return z.library().fsdp_linear_dx(a["n"], a["w"], a["r"], a["k"], a["dz"], a["m"], a["zz"], a["zc"], a["zs"],
                                      a["act"], a["res"], a["dx"], None)


def dw(z, **kw):
    a = dict(dz=P, x=P, xc=None, xs=None, m=4, r=64, k=32, scale=1.0, dw=P, dwb=None, ws=None, wsb=0)
    a.update(kw)
    return z.library().fsdp_linear_dw(a["dz"], a["x"], a["xc"], a["xs"], a["m"], a["r"], a["k"], a["scale"], a["dw"],
                                      a["dwb"], a["ws"], a["wsb"], None)


def actb(z, **kw):
    a = dict(dy=P, zz=P, zc=None, zs=None, m=4, k=32, act=4, dz=P, db=None, ws=None, wsb=0)
    a.update(kw)
    return z.library().fsdp_act_backward(a["dy"], a["zz"], a["zc"], a["zs"], a["m"], a["k"], a["act"], a["dz"], a["db"],
                                         a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,word", [
    (dict(m=0), "1..2^30"), (dict(r=0), "1..2^30"), (dict(k=0), "1..2^30"), (dict(m=1 << 31), "1..2^30"),
    (dict(k=36), "multiples of 8"), (dict(r=60), "multiples of 8"), (dict(n=0), "n_ranks"), (dict(n=17), "n_ranks"),
    (dict(n=3, w=shards(3)), "multiple of 8"), (dict(n=16, w=shards(16)), "multiple of 8"), (dict(w=None), "w_shards"),
    (dict(w=(C.c_void_p * 2)(P, None)), "missing rank"), (dict(w=shards(2, P + 8)), "16-byte"), (dict(x=None), "NULL"),
    (dict(y=None), "NULL"), (dict(act=5), "act 5"), (dict(act=-1), "act -1"), (dict(zc=P), "both"), (dict(zs=P), "both"),
    (dict(zz=P, zc=P, zs=P), "keep Z"), (dict(x=P + 2), "16-byte"), (dict(y=P + 8), "16-byte"),
    (dict(bias=P + 4), "16-byte"), (dict(res=P + 2), "16-byte"), (dict(zz=P + 8), "16-byte"),
    (dict(zc=P + 1, zs=P), "16-byte")])
def test_forward_refuses(z, kw, word):
    refused(z, forward(z, **kw), word)


@pytest.mark.parametrize("kw,word", [
    (dict(m=0), "1..2^30"), (dict(k=33), "multiples of 8"), (dict(n=17), "n_ranks"), (dict(w=None), "w_shards"),
    (dict(dz=None), "NULL"), (dict(dx=None), "NULL"), (dict(act=7), "act 7"), (dict(zz=None), "kept activation"),
    (dict(zc=P, zs=P), "kept activation"), (dict(zz=None, zc=P), "kept activation"), (dict(zz=P + 4), "16-byte"),
    (dict(res=P + 4), "16-byte"), (dict(dx=P + 8), "16-byte")])
def test_dx_refuses(z, kw, word):
    refused(z, dx(z, **kw), word)


@pytest.mark.parametrize("kw,word", [
    (dict(m=0), "1..2^30"), (dict(r=12), "multiples of 8"), (dict(dz=None), "NULL"), (dict(x=None), "pass X"),
    (dict(xc=P, xs=P), "pass X"), (dict(x=None, xc=P), "pass X"), (dict(dw=None), "one of dW"),
    (dict(dwb=P), "one of dW"), (dict(scale=float("nan")), "finite"), (dict(scale=float("inf")), "finite"),
    (dict(dz=P + 2), "16-byte"), (dict(dw=P + 4), "16-byte"), (dict(x=None, xc=P + 8, xs=P), "16-byte"),
    (dict(x=None, xc=P, xs=P), "workspace of 0"), (dict(x=None, xc=P, xs=P, ws=P, wsb=255), "workspace of 255"),
    (dict(x=None, xc=P, xs=P, ws=P + 4, wsb=256), "16-byte")])
def test_dw_refuses(z, kw, word):
    refused(z, dw(z, **kw), word)


@pytest.mark.parametrize("kw,word", [
    (dict(m=0), ">= 1"), (dict(k=0), ">= 1"), (dict(k=20), "multiple of 8"), (dict(dy=None), "dY"),
    (dict(dz=None), "both NULL"), (dict(act=5), "act 5"), (dict(zz=None), "kept activation"),
    (dict(zz=None, zs=P), "kept activation"), (dict(dz=P + 8), "16-byte"), (dict(db=P + 4), "16-byte"),
    (dict(m=1 << 41), "2^40"), (dict(ws=P + 8, wsb=1 << 30), "16-byte")])
def test_act_backward_refuses(z, kw, word):
    refused(z, actb(z, **kw), word)


def test_act_backward_refuses_a_small_workspace(z):
    m, k = 1 << 20, 4096
    need = C.c_uint64()
    assert z.library().fsdp_act_backward_workspace(m, k, C.byref(need)) == 0
    assert need.value > 64  # else the call would be accepted, and launched
    refused(z, actb(z, m=m, k=k, db=P, ws=P, wsb=64), "workspace of 64")


@pytest.mark.parametrize("args,word", [
    ((None, 4, 32, P, P), "NULL"), ((P, 4, 32, None, P), "NULL"), ((P, 4, 32, P, None), "NULL"),
    ((P, 0, 32, P, P), ">= 1"), ((P, 4, 0, P, P), ">= 1"), ((P, 4, 28, P, P), "multiple of 8"),
    ((P + 8, 4, 32, P, P), "16-byte"), ((P, 4, 32, P + 1, P), "16-byte"), ((P, 4, 32, P, P + 4), "16-byte")])
def test_pack_refuses(z, args, word):
    refused(z, z.library().fsdp_checkpoint8_pack(*args, None), word)


@pytest.mark.parametrize("args,word", [
    ((None, P, 4, 32, 0, P), "NULL"), ((P, None, 4, 32, 0, P), "NULL"), ((P, P, 4, 32, 0, None), "NULL"),
    ((P, P, -1, 32, 0, P), ">= 1"), ((P, P, 4, 4, 0, P), "multiple of 8"), ((P, P, 4, 32, 8, P), "act 8"),
    ((P, P, 4, 32, 0, P + 2), "16-byte")])
def test_unpack_refuses(z, args, word):
    refused(z, z.library().fsdp_checkpoint8_unpack(*args, None), word)


def test_act_backward_workspace(z):
    assert z.fsdp_act_backward_workspace(16, 4096) == 0
    b = z.fsdp_act_backward_workspace(1 << 20, 4096)
    assert b > 0 and b % (4 * 4096) == 0
    assert z.fsdp_act_backward_workspace(3, 1 << 21) == 0 or z.fsdp_act_backward_workspace(3, 1 << 21) >= 4 << 21
    with pytest.raises(z.ZeroError):
        z.fsdp_act_backward_workspace(4, 20)
    refused(z, z.library().fsdp_act_backward_workspace(4, 32, None), "NULL")


def test_dw_workspace(z):
    assert z.fsdp_linear_dw_workspace(3, 40) == 256 and z.fsdp_linear_dw_workspace(8192, 4096) == 2 * 8192 * 4096
    with pytest.raises(z.ZeroError):
        z.fsdp_linear_dw_workspace(0, 40)
    refused(z, z.library().fsdp_linear_dw_workspace(4, 32, None), "NULL")
