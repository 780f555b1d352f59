"""Calls up to the library's entry without a GPU: tensors that have a device and
a shape but no memory, and the native calls bound to a current device of the
test's choice.  Such a call passes every check and then stops where the first
tensor is asked for its memory."""

import contextlib
import ctypes

import torch

import fp8_fine_grained_quant_amd as fq

NO_MEMORY = "Cannot access data pointer"


class Hollow(torch.Tensor):
    """A tensor without storage: asking for its memory throws."""

    @staticmethod
    def __new__(cls, shape, dtype, device):
        return torch.Tensor._make_wrapper_subclass(cls, shape, dtype=dtype, device=device)

    @classmethod
    def __torch_dispatch__(cls, func, types, args=(), kwargs=None):
        raise NotImplementedError(func)


def hollow(*shape, dt=torch.float32, device="cuda:0"):
    t = Hollow(shape, dt, device)
    torch._C._set_throw_on_mutable_data_ptr(t)
    return t


@contextlib.contextmanager
def current_device(index):
    """The native calls take device `index` for the current one, and the address
    0 for its current stream."""
    lib, native = fq.load_library(), fq._native()
    names = [n for n in fq.EXPORTS if n.startswith(("fp8q_moe_", "fp8q_grad_"))]
    native.bind({n: ctypes.cast(getattr(lib, n), ctypes.c_void_p).value for n in names}, lambda: index, lambda d: 0,
                fq._check, fq._score, fq._on_stream)
    try:
        yield
    finally:
        fq._bind(lib)
