"""Routing and clipping calls take tensors of one device, the current one, and
refuse others before any work: the library's kernels run on the current device,
which may have no access to another's memory."""

import pytest
import torch

import fp8_fine_grained_quant_amd as fq
from fake_device import NO_MEMORY, current_device, hollow

i32, u8, bf16 = torch.int32, torch.uint8, torch.bfloat16
T, K, H, E = 6, 4, 32, 8


def operands():
    """Every call with given outputs: name -> (function, its tensors)."""
    t = lambda *shape, dt=torch.float32: (shape, dt)
    x, rows, ids, w = t(T, H), t(T * K, H), t(T, K, dt=i32), t(T, K)
    q, s = t(T * K, H, dt=u8), t(T * K, 1)
    route = lambda logits, ids, w, bias: fq.fp8q_moe_route(logits, ids, w, bias=bias)
    sort = lambda ids, off, dst, src, ws: fq.fp8q_moe_sort(ids, E, off, dst, src, ws)
    clip = lambda a, b, oa, ob, norm, ws: fq.fp8q_grad_clip([a, b], [oa, ob], 1.0, norm, ws)
    return {
        "route": (route, [t(T, E), ids, w, t(E)]),
        "route_bwd": (fq.fp8q_moe_route_bwd, [w, t(T, E), ids, t(T, E)]),
        "sort": (sort, [ids, t(E + 1, dt=i32), ids, t(T * K, dt=i32), t(64, dt=u8)]),
        "dispatch": (fq.fp8q_moe_dispatch, [x, ids, rows, q, s]),
        "dispatch_bwd": (fq.fp8q_moe_dispatch_bwd, [rows, ids, x]),
        "combine": (fq.fp8q_moe_combine, [rows, ids, w, x]),
        "combine_bwd": (fq.fp8q_moe_combine_bwd, [x, rows, ids, w, w, rows, q, s]),
        "clip": (clip, [t(5), t(7), t(5), t(7), t(), t(1 << 20, dt=u8)]),
    }


@pytest.mark.parametrize("name", operands())
def test_one_device(name):
    fn, args = operands()[name]
    make = lambda other=-1: [hollow(*shape, dt=dt, device="cuda:1" if i == other else "cuda:0")
                             for i, (shape, dt) in enumerate(args)]
    with current_device(0):
        with pytest.raises(RuntimeError, match=NO_MEMORY):
            fn(*make())
        for i in range(len(args)):
            with pytest.raises(ValueError, match="tensors on cuda:[01] and cuda:[01]"):
                fn(*make(i))


@pytest.mark.parametrize("name", operands())
def test_current_device(name):
    fn, args = operands()[name]
    tensors = [hollow(*shape, dt=dt, device="cuda:1") for shape, dt in args]
    with current_device(0), pytest.raises(ValueError, match="tensors on cuda:1, but the current device is cuda:0"):
        fn(*tensors)
    with current_device(1), pytest.raises(RuntimeError, match=NO_MEMORY):
        fn(*tensors)


def test_given_stream():
    """A stream's address does not tell its device: the rule is the same."""
    x, ids, w = hollow(T, E), hollow(T, K, dt=i32), hollow(T, K)
    with current_device(1), pytest.raises(ValueError, match="tensors on cuda:0, but the current device is cuda:1"):
        fq.fp8q_moe_route(x, ids, w, stream=64)


def test_clip_of_other_places():
    a, b = hollow(5), hollow(7, device="cuda:1")
    with current_device(0):
        with pytest.raises(ValueError, match="tensors on cuda:0 and cuda:1"):
            fq.grad_clip([a, b], 1.0)
        with pytest.raises(ValueError, match="GPU tensors only"):
            fq.grad_clip([a, torch.zeros(7)], 1.0)
        with pytest.raises(ValueError, match="tensors on cuda:0 and cuda:1"):
            fq.grad_clip([a], 1.0, out=[hollow(5, device="cuda:1")])


class Emptying:
    """A bound whose reading empties the list of gradients."""

    def __init__(self, grads):
        self.grads = grads

    def __float__(self):
        self.grads.clear()
        return 1.0


def test_clip_keeps_its_tensors():
    a = [hollow(5), hollow(7)]
    with current_device(0), pytest.raises(RuntimeError, match=NO_MEMORY):
        fq.fp8q_grad_clip(a, a, Emptying(a), hollow(), hollow(1 << 20, dt=u8))
    assert a == []
