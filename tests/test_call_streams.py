"""The stream of a routing or clipping call: torch's stream object, or its
address as a number, 0 being the default stream."""

import contextlib

import numpy as np
import pytest
import torch

import fp8_fine_grained_quant_amd as fq
from fake_device import NO_MEMORY, current_device, hollow


class Recorder:
    """Stands for the bound native module; keeps the stream that was current."""

    def __init__(self, monkeypatch):
        self.current, self.seen = "none", []

        @contextlib.contextmanager
        def stream(s):
            before, self.current = self.current, s
            yield
            self.current = before

        monkeypatch.setattr(torch.cuda, "stream", stream)
        monkeypatch.setattr(torch.cuda, "default_stream", lambda *a: "default")
        # an external stream of address 0 is a stream of torch's pool
        monkeypatch.setattr(torch.cuda, "ExternalStream", lambda p: ("external", p) if p else "pool")
        monkeypatch.setattr(fq, "_bound", self, raising=False)

    def call(self, *args):
        self.seen.append((self.current, args))
        return "result"


@pytest.mark.parametrize("stream, want", [(0, "default"), (64, ("external", 64)), (np.int64(0), "default"),
                                          (np.int64(64), ("external", 64))], ids=str)
def test_number(stream, want, monkeypatch):
    r = Recorder(monkeypatch)
    assert fq._on_stream("call", (1, 2), stream) == "result"
    assert r.seen == [(want, (1, 2, None))]


def test_object(monkeypatch):
    r = Recorder(monkeypatch)
    s = type("Stream", (), {"cuda_stream": 0})()
    fq._on_stream("call", (), s)
    assert r.seen == [(s, (None,))]


def path(x, logits, grad, k, stream):
    """Every call that allocates, one after the other on `stream`."""
    ids, w = fq.moe_route(logits, k, stream=stream)
    off, dst, src = fq.moe_sort(ids, logits.shape[1], stream=stream)
    rows = fq.moe_dispatch(x, dst, stream=stream)
    _, q, s = fq.moe_dispatch_quant(x, dst, stream=stream)
    y = fq.moe_combine(rows, dst, w, stream=stream)
    dr, dw = fq.moe_combine_bwd(y, rows, dst, w, stream=stream)
    _, dq, ds, dw2 = fq.moe_combine_bwd_quant(y, rows, dst, w, stream=stream)
    dl = fq.moe_route_bwd(dw, logits, ids, stream=stream)
    dx = fq.moe_dispatch_bwd(dr, dst, stream=stream)
    norm = fq.grad_clip([grad], 1.0, stream=stream)
    return [ids, w, off, dst, src, rows, q, s, y, dr, dw, dq, ds, dw2, dl, dx, norm, grad]


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["zero", "zero from a side stream", "side", "side as a number"])
def test_order_on_the_stream(name):
    """Inputs that the stream's earlier work is still to write, outputs read by
    its next work: no wait of the host in between."""
    t, k, h, e = 1500, 6, 256, 40
    gen = torch.Generator(device="cuda").manual_seed(5)
    want_x = torch.randn(t, h, generator=gen, device="cuda").to(torch.bfloat16)
    want_l = torch.randn(t, e, generator=gen, device="cuda")
    want_g = torch.randn(70_000, generator=gen, device="cuda")
    side = torch.cuda.Stream()
    on = torch.cuda.default_stream() if name.startswith("zero") else side
    given = {"zero": 0, "zero from a side stream": 0, "side": side, "side as a number": side.cuda_stream}[name]
    assert torch.cuda.default_stream().cuda_stream == 0
    grad = want_g.clone()
    want = [v.clone() for v in path(want_x, want_l, grad, k, None)]
    x, logits, grad = (torch.zeros_like(v) for v in (want_x, want_l, want_g))
    torch.cuda.synchronize()
    with torch.cuda.stream(on):
        torch.cuda._sleep(50_000_000)
        x.copy_(want_x)
        logits.copy_(want_l)
        grad.copy_(want_g)
    with torch.cuda.stream(side if name == "zero from a side stream" else torch.cuda.default_stream()):
        got = path(x, logits, grad, k, given)
    with torch.cuda.stream(on):
        read = [v.clone() for v in got]
    torch.cuda.synchronize()
    for i, (a, b) in enumerate(zip(read, want)):
        assert torch.equal(a, b), i


class Address:
    def __init__(self, p):
        self.p = p

    def __int__(self):
        return self.p


@pytest.mark.parametrize("stream", [None, 0, 64, np.int64(0), np.uint64(64), Address(64)], ids=lambda s: type(s).__name__)
def test_kinds_of_numbers(stream):
    """Taken with given outputs: the call goes on to the tensors' memory."""
    x, ids, w = hollow(6, 32), hollow(6, 4, dt=torch.int32), hollow(6, 4)
    with current_device(0), pytest.raises(RuntimeError, match=NO_MEMORY):
        fq.fp8q_moe_route(x, ids, w, stream=stream)


def test_no_stream():
    x, ids, w = hollow(6, 32), hollow(6, 4, dt=torch.int32), hollow(6, 4)
    for bad, error in ((1 << 80, OverflowError), (object(), TypeError), ("now", ValueError)):
        with current_device(0), pytest.raises(error):
            fq.fp8q_moe_route(x, ids, w, stream=bad)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", [int, np.int64, Address])
def test_numbers_on_the_gpu(kind):
    """A stream's address as any number, with and without given outputs."""
    logits = torch.randn(50, 32, device="cuda")
    ids, w = fq.moe_route(logits, 4)
    torch.cuda.synchronize()
    for stream in (torch.cuda.default_stream(), torch.cuda.Stream()):
        made = fq.moe_route(logits, 4, stream=kind(stream.cuda_stream))
        out = torch.empty_like(ids), torch.empty_like(w)
        torch.cuda.synchronize()
        fq.fp8q_moe_route(logits, *out, stream=kind(stream.cuda_stream))
        torch.cuda.synchronize()
        for got in (made, out):
            assert torch.equal(got[0], ids) and torch.equal(got[1], w)
