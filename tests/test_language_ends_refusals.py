"""Argument errors of the embedding, layer norm and vocabulary loss calls, found on the host before anything
is launched. Through the C ABI the pointers are made up and never read, so those tests run where there is no
GPU; the binding's own checks are tested with tensors."""
from __future__ import annotations

import ctypes as C
import re
from pathlib import Path

import pytest
import torch

P = 1 << 20  # a 16-byte-aligned address that is never dereferenced
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="made-up device addresses: only where there is no GPU")


@pytest.fixture(scope="module")
def z():
    import __graft_entry__ as g
    g.build()
    import fsdp_sharded_optimizer_zero_gb300 as z
    return z


def refused(z, rc, word, code=-1):
    assert rc == code, (rc, z.zero_last_error())
    assert word in z.zero_last_error(), z.zero_last_error()


def shards(n, p=P):
    return (C.c_void_p * n)(*[p] * n)


NAN, INF = float("nan"), float("inf")
CSRC = Path(__file__).resolve().parents[1] / "fsdp_sharded_optimizer_zero_gb300" / "csrc"


@pytest.mark.parametrize("name", ["linear_wide.cuh", "linear_narrow.cuh", "fsdp_vocab_loss.cu"])
def test_warps_of_the_products_meet_only_where_they_agree_on_leaving(name):
    """As in the linear unit: a role's loops end when a bounded wait gives up, which its warps may see at different
    tiles, so no named barrier counts them. (That wait is not provoked on a GPU: the source has no such barrier.)"""
    code = re.sub(r"//[^\n]*", "", (CSRC / name).read_text())
    assert not re.findall(r'"[^"]*\b(?:bar|barrier)(?:\.cta)?\.(?:sync|arrive)\b[^"]*"', code)


def embed(z, **kw):
    a = dict(n=2, e=shards(2), rows=64, v=60, k=32, t=P, tb=8, m=4, scale=1.0, y=P)
    a.update(kw)
    return z.library().fsdp_embedding_forward(a["n"], a["e"], a["rows"], a["v"], a["k"], a["t"], a["tb"], a["m"], a["scale"],
                                              a["y"], None)


def embed_grad(z, **kw):
    a = dict(dy=P, t=P, tb=8, m=5000, rows=64, v=60, k=32, scale=1.0, add=0, de=P, deb=None, ws=P, wsb=1 << 30)
    a.update(kw)
    return z.library().fsdp_embedding_backward(a["dy"], a["t"], a["tb"], a["m"], a["rows"], a["v"], a["k"], a["scale"], a["add"],
                                               a["de"], a["deb"], a["ws"], a["wsb"], None)


def norm(z, **kw):
    a = dict(x=P, rows=4, k=32, g=P, b=P, eps=1e-5, y=P, mean=P, rstd=P)
    a.update(kw)
    return z.library().fsdp_layernorm_forward(a["x"], a["rows"], a["k"], a["g"], a["b"], a["eps"], a["y"], a["mean"], a["rstd"],
                                              None)


def norm_grad(z, **kw):
    a = dict(dy=P, x=P, mean=P, rstd=P, rows=50000, k=32, g=P, res=P, dx=P, dg=P, db=P, ws=P, wsb=1 << 30)
    a.update(kw)
    return z.library().fsdp_layernorm_backward(a["dy"], a["x"], a["mean"], a["rstd"], a["rows"], a["k"], a["g"], a["res"], a["dx"],
                                               a["dg"], a["db"], a["ws"], a["wsb"], None)


def loss(z, **kw):
    a = dict(n=2, w=shards(2), r=64, v=60, k=32, x=P, m=4, t=P, tb=8, loss=P, lse=P, total=P, ws=P, wsb=1 << 30)
    a.update(kw)
    return z.library().fsdp_vocab_loss_forward(a["n"], a["w"], a["r"], a["v"], a["k"], a["x"], a["m"], a["t"], a["tb"], a["loss"],
                                               a["lse"], a["total"], a["ws"], a["wsb"], None)


def loss_grad(z, **kw):
    a = dict(n=2, w=shards(2), r=64, v=60, k=32, x=P, m=4, t=P, tb=8, lse=P, dloss=P, total=P, scale=1.0, dx=P, dw=P, piece=0,
             ws=P, wsb=1 << 30)
    a.update(kw)
    return z.library().fsdp_vocab_loss_backward(a["n"], a["w"], a["r"], a["v"], a["k"], a["x"], a["m"], a["t"], a["tb"], a["lse"],
                                                a["dloss"], a["total"], a["scale"], a["dx"], a["dw"], a["piece"], a["ws"],
                                                a["wsb"], None)


@no_gpu
@pytest.mark.parametrize("kw,word", [
    (dict(m=0), "1..2^30"), (dict(m=(1 << 30) + 1), "1..2^30"), (dict(rows=0), "1..2^30"), (dict(k=0), "2^20"),
    (dict(k=(1 << 20) + 8), "2^20"), (dict(k=12), "multiple of 8"), (dict(v=0), "vocab 0"), (dict(v=65), "vocab 65"),
    (dict(tb=2), "token_bytes"), (dict(n=0), "n_ranks"), (dict(n=17), "n_ranks"), (dict(n=3, e=shards(3)), "multiple of n_ranks"),
    (dict(e=None), "e_shards"), (dict(e=(C.c_void_p * 2)(P, None)), "missing rank"), (dict(e=shards(2, P + 8)), "16-byte"),
    (dict(t=None), "NULL"), (dict(y=None), "NULL"), (dict(y=P + 2), "16-byte"), (dict(t=P + 4), "8 bytes"),
    (dict(t=P + 2, tb=4), "4 bytes"), (dict(scale=NAN), "finite"), (dict(scale=-INF), "finite")])
def test_embedding_refuses(z, kw, word):
    refused(z, embed(z, **kw), word)


@no_gpu
@pytest.mark.parametrize("kw,word", [
    (dict(m=-1), "1..2^30"), (dict(k=20), "multiple of 8"), (dict(v=100), "vocab 100"), (dict(tb=0), "token_bytes"),
    (dict(dy=None), "NULL"), (dict(t=None), "NULL"), (dict(de=None), "one of dE"), (dict(deb=P), "one of dE"),
    (dict(scale=INF), "finite"), (dict(dy=P + 4), "16-byte"), (dict(de=P + 4), "16-byte"), (dict(t=P + 1), "8 bytes"),
    (dict(ws=None), "workspace of 0"), (dict(wsb=255), "workspace of 255"), (dict(ws=P + 8), "16-byte")])
def test_embedding_backward_refuses(z, kw, word):
    refused(z, embed_grad(z, **kw), word)


@no_gpu
def test_embedding_refuses_more_than_it_counts(z):
    refused(z, embed_grad(z, m=1 << 30, k=1 << 20), "2^42", code=-4)


@no_gpu
@pytest.mark.parametrize("kw,word", [
    (dict(rows=0), "1..2^30"), (dict(k=0), "1..2^30"), (dict(rows=(1 << 30) + 1), "1..2^30"), (dict(k=28), "multiple of 8"),
    (dict(x=None), "NULL"), (dict(y=None), "NULL"), (dict(mean=None), "both"), (dict(rstd=None), "both"), (dict(eps=-1e-5), "eps"),
    (dict(eps=NAN), "eps"), (dict(eps=INF), "eps"), (dict(x=P + 8), "16-byte"), (dict(g=P + 8), "16-byte"), (dict(b=P + 2), "16-byte"),
    (dict(y=P + 4), "16-byte"), (dict(mean=P + 2), "4-byte")])
def test_layernorm_refuses(z, kw, word):
    refused(z, norm(z, **kw), word)


@no_gpu
@pytest.mark.parametrize("kw,word", [
    (dict(rows=-2), "1..2^30"), (dict(k=4), "multiple of 8"), (dict(dy=None), "NULL"), (dict(x=None), "NULL"), (dict(mean=None), "NULL"),
    (dict(rstd=None), "NULL"), (dict(dx=None), "NULL"), (dict(dy=P + 8), "16-byte"), (dict(res=P + 8), "16-byte"),
    (dict(dx=P + 2), "16-byte"), (dict(dg=P + 2), "4-byte"), (dict(ws=None), "workspace of 0"), (dict(wsb=8), "workspace of 8"),
    (dict(ws=P + 4), "16-byte")])
def test_layernorm_backward_refuses(z, kw, word):
    refused(z, norm_grad(z, **kw), word)


LOSS = [(dict(m=0), "1..2^30"), (dict(r=0), "1..2^30"), (dict(k=0), "1..2^30"), (dict(k=36), "multiple of 8"), (dict(v=0), "vocab 0"),
        (dict(v=65), "vocab 65"), (dict(tb=1), "label_bytes"), (dict(n=0), "n_ranks"), (dict(n=17), "n_ranks"),
        (dict(n=3, w=shards(3)), "multiple of 8"), (dict(n=16, w=shards(16)), "multiple of 8"), (dict(w=None), "w_shards"),
        (dict(w=(C.c_void_p * 2)(None, P)), "missing rank"), (dict(w=shards(2, P + 8)), "16-byte"), (dict(x=None), "NULL"),
        (dict(t=None), "NULL"), (dict(lse=None), "NULL"), (dict(x=P + 8), "16-byte"), (dict(t=P + 4), "their elements"),
        (dict(lse=P + 2), "their elements"), (dict(total=P + 2), "their elements"), (dict(ws=None), "workspace of 0"),
        (dict(wsb=255), "workspace of 255"), (dict(ws=P + 4), "16-byte")]


@no_gpu
@pytest.mark.parametrize("kw,word", LOSS + [(dict(loss=None), "NULL"), (dict(loss=P + 1), "their elements")])
def test_vocab_loss_refuses(z, kw, word):
    refused(z, loss(z, **kw), word)


@no_gpu
@pytest.mark.parametrize("kw,word", LOSS + [
    (dict(dx=None, dw=None), "both NULL"), (dict(dx=P + 8), "16-byte"), (dict(dw=P + 8), "16-byte"), (dict(dloss=P + 2), "their elements"),
    (dict(scale=NAN), "finite"), (dict(piece=-256), "piece"), (dict(piece=100), "piece"), (dict(piece=1 << 31), "piece")])
def test_vocab_loss_backward_refuses(z, kw, word):
    refused(z, loss_grad(z, **kw), word)


@no_gpu
def test_vocab_loss_refuses_more_tiles_than_it_counts(z):
    refused(z, loss(z, m=1 << 30, r=1 << 30, v=1 << 30), "2^30 tiles", code=-4)


def test_workspaces(z):
    assert z.fsdp_embedding_backward_workspace(1, 1, 8) == 0  # few tokens: none is used
    small, large = z.fsdp_embedding_backward_workspace(5000, 500, 64), z.fsdp_embedding_backward_workspace(100000, 500, 64)
    assert 0 < small < large < 100000 * 64 * 2
    assert z.fsdp_layernorm_backward_workspace(4, 4096) == 0 and z.fsdp_layernorm_backward_workspace(50000, 4096) >= 8 * 4096
    assert z.fsdp_vocab_loss_forward_workspace(8192, 50257) < 8192 * 50257 // 8
    whole, piece = (z.fsdp_vocab_loss_backward_workspace(8192, 50257, 768, p) for p in (0, 4096))
    assert 2 * 8192 * 4096 <= piece < whole
    assert z.fsdp_vocab_loss_backward_workspace(1, 1, 8, 0) > 0
    for call in (lambda: z.fsdp_embedding_backward_workspace(0, 5, 8), lambda: z.fsdp_layernorm_backward_workspace(3, 12),
                 lambda: z.fsdp_vocab_loss_forward_workspace(4, 0), lambda: z.fsdp_vocab_loss_backward_workspace(4, 5, 8, 7)):
        with pytest.raises(z.ZeroError):
            call()
    for name, args in (("fsdp_embedding_backward_workspace", (4, 5, 8)), ("fsdp_layernorm_backward_workspace", (4, 8)),
                       ("fsdp_vocab_loss_forward_workspace", (4, 5)), ("fsdp_vocab_loss_backward_workspace", (4, 5, 8, 0))):
        refused(z, getattr(z.library(), name)(*args, None), "NULL")


def test_binding_checks(z):
    """Types, shapes and devices, before the library is called."""
    bf = torch.bfloat16
    x, ids = torch.zeros(4, 32, dtype=bf), torch.zeros(4, dtype=torch.int64)
    e = [torch.zeros(8, 32, dtype=bf)]
    with pytest.raises(TypeError, match="int32 or torch.int64"):
        z.fsdp_embedding_backward(x, ids.float(), e[0])
    with pytest.raises(ValueError, match="1-D"):
        z.fsdp_embedding_backward(x, ids[None], e[0])
    with pytest.raises(ValueError, match="CUDA"):
        z.fsdp_embedding_forward(e, ids, x)
    with pytest.raises(ValueError, match="2-D"):
        z.fsdp_layernorm_forward(ids, x)
    with pytest.raises(ValueError, match="empty"):
        z.fsdp_vocab_loss_forward([], x, ids, ids, ids)
    with pytest.raises(ValueError, match="CUDA"):
        z.fsdp_vocab_loss_backward(e, x, ids, torch.zeros(4), x, e[0])


@pytest.mark.gpu
def test_binding_checks_shapes(z):
    dev, bf = "cuda", torch.bfloat16
    x, y, ids = torch.zeros(4, 32, dtype=bf, device=dev), torch.zeros(4, 32, dtype=bf, device=dev), torch.zeros(4, dtype=torch.int64, device=dev)
    e, f = [torch.zeros(8, 32, dtype=bf, device=dev)], torch.zeros(4, device=dev)
    bad = [
        (ValueError, "Y", lambda: z.fsdp_embedding_forward(e, ids, y[:3])),
        (ValueError, "contiguous", lambda: z.fsdp_embedding_forward(e, torch.zeros(8, dtype=torch.int64, device=dev)[::2], y)),
        (TypeError, "Y", lambda: z.fsdp_embedding_forward(e, ids, y.float())),
        (ValueError, "dY", lambda: z.fsdp_embedding_backward(x[:2], ids, e[0])),
        (TypeError, "dE", lambda: z.fsdp_embedding_backward(x, ids, e[0].half())),
        (ValueError, "gamma", lambda: z.fsdp_layernorm_forward(x, y, gamma=e[0][0, :16].clone())),
        (ValueError, "mean", lambda: z.fsdp_layernorm_forward(x, y, mean=f[:3].clone(), rstd=f)),
        (TypeError, "dgamma", lambda: z.fsdp_layernorm_backward(x, x, f, f, y, dgamma=e[0][0].clone())),
        (ValueError, "loss", lambda: z.fsdp_vocab_loss_forward(e, x, ids, f[:2].clone(), f)),
        (ValueError, "X", lambda: z.fsdp_vocab_loss_forward(e, x[:, :16].contiguous(), ids, f, f)),
        (ValueError, "total", lambda: z.fsdp_vocab_loss_forward(e, x, ids, f, f, total=f)),
        (ValueError, "dW", lambda: z.fsdp_vocab_loss_backward(e, x, ids, f, y, x)),
        (z.ZeroError, "vocab", lambda: z.fsdp_vocab_loss_forward(e, x, ids, f, f, vocab=9)),
        (z.ZeroError, "workspace", lambda: z.fsdp_vocab_loss_backward(e, x, ids, f, y, e[0], workspace=torch.empty(16, dtype=torch.uint8, device=dev))),
        (z.ZeroError, "piece", lambda: z.fsdp_vocab_loss_backward(e, x, ids, f, y, e[0], piece=100)),
    ]
    for kind, word, call in bad:
        with pytest.raises(kind, match=word):
            call()
    z.zero_device_status()
