"""The workspace that the binding takes for a call which was given none belongs to the call's stream: no
other stream's queued work uses it, whatever that stream has freed."""
from __future__ import annotations

import contextlib

import pytest
import torch

DEV = "cuda"
BF = torch.bfloat16


@pytest.fixture(scope="module")
def z():
    import __graft_entry__ as g
    g.build()
    import fsdp_sharded_optimizer_zero_gb300 as z
    return z


class Handle:
    cuda_stream = 77


@pytest.mark.parametrize("stream,want", [(None, "current"), (0, "default"), (1234, 1234), (Handle(), 77)])
def test_allocated_on_the_stream_of_the_call(z, monkeypatch, stream, want):
    """No GPU: torch's stream context and allocation are replaced by ones that take notes."""
    now, seen = ["current"], []

    @contextlib.contextmanager
    def on(s):
        now.append(s)
        yield
        now.pop()

    class Block:
        def record_stream(self, s):
            pass

    def empty(n, dtype, device):
        seen.append((n, dtype, now[-1]))
        return Block()

    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda h: h)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda: "default")
    monkeypatch.setattr(torch, "empty", empty)
    assert isinstance(z._lib._call_workspace(512, "cuda", stream), Block)
    assert seen == [(512, torch.uint8, want)] and now == ["current"]


def randn(rows, cols, std, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn(rows, cols, generator=gen, device=DEV) * std).to(BF)


@pytest.mark.gpu
@pytest.mark.parametrize("op", ["dw", "act_backward"])
@pytest.mark.parametrize("as_handle", [False, True])
def test_not_a_block_that_the_current_stream_still_reads(z, op, as_handle):
    """The current stream has a read of a block queued behind a delay, and the block is freed: the
    allocator may hand it to that stream's next allocation. A call on another stream, which does not wait
    for the current one, leaves it alone."""
    if op == "dw":
        m, r, k = 4000, 264, 1032
        g, x = randn(m, r, 0.3, 1), randn(m, k, 1.0, 2)
        x8 = torch.empty(m, k, dtype=torch.int8, device=DEV), torch.empty(m, -(-k // 32), dtype=torch.uint8, device=DEV)
        z.fsdp_checkpoint8_pack(x, *x8)
        nbytes = z.fsdp_linear_dw_workspace(m, k)

        def call(out, **kw):
            z.fsdp_linear_dw(g, out, x8=x8, **kw)

        new = lambda: torch.empty(r, k, device=DEV)  # noqa: E731
    else:
        m, k = 9000, 2048
        g, x = randn(m, k, 0.3, 3), randn(m, k, 1.0, 4)
        nbytes = z.fsdp_act_backward_workspace(m, k)
        assert nbytes > 0

        def call(out, **kw):
            z.fsdp_act_backward(g, db=out, z=x, act=z.FSDP_ACT_SILU, **kw)

        new = lambda: torch.empty(k, device=DEV)  # noqa: E731
    want, got = new(), new()
    call(want)
    copy = torch.empty(nbytes, dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    block = torch.full((nbytes,), 7, dtype=torch.uint8, device=DEV)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)  # about 0.1 s
    copy.copy_(block)
    del block
    call(got, stream=side.cuda_stream if as_handle else side)
    side.synchronize()
    torch.cuda.synchronize()
    assert bool((copy == 7).all())
    assert torch.equal(got, want)
    z.zero_device_status()


@pytest.mark.gpu
def test_many_calls_on_two_streams(z):
    """Calls on two streams in turn, no workspace given, nothing synchronised between: the same bits as
    one at a time."""
    m, r, k = 3000, 264, 520
    g = [randn(m, r, 0.3, 5 + i) for i in range(2)]
    x8 = []
    for i in range(2):
        c = torch.empty(m, k, dtype=torch.int8, device=DEV), torch.empty(m, -(-k // 32), dtype=torch.uint8, device=DEV)
        z.fsdp_checkpoint8_pack(randn(m, k, 1.0, 7 + i), *c)
        x8.append(c)
    want = [torch.empty(r, k, device=DEV) for _ in range(2)]
    for i in range(2):
        z.fsdp_linear_dw(g[i], want[i], x8=x8[i])
    torch.cuda.synchronize()
    side = [torch.cuda.Stream() for _ in range(2)]
    got = [[torch.empty(r, k, device=DEV) for _ in range(2)] for _ in range(20)]
    torch.cuda.synchronize()
    for row in got:
        for i in range(2):
            z.fsdp_linear_dw(g[i], row[i], x8=x8[i], stream=side[i])
    torch.cuda.synchronize()
    assert all(torch.equal(row[i], want[i]) for row in got for i in range(2))
    z.zero_device_status()
