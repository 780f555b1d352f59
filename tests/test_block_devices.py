"""The training block's calls that allocate refuse tensors that are not of the
current device before they allocate or launch anything (without a GPU an allocation
fails with another error)."""

import pytest
import torch

import fp8_fine_grained_quant_amd as fq
from fake_device import current_device, hollow

U8, F32, BF16, I32 = torch.uint8, torch.float32, torch.bfloat16, torch.int32


def calls():
    t = lambda *s, dt=F32: hollow(*s, dt=dt, device="cuda:0")  # noqa: E731
    x, xs, w, ws = t(5, 256, dt=U8), t(5, 2), t(256, 256, dt=U8), t(2, 2)
    off, gu = t(3, dt=I32), t(5, 256, dt=BF16)
    return [lambda: fq.rms_norm(t(3, 8), t(8)), lambda: fq.rms_norm(t(3, 0), t(0)),
            lambda: fq.rms_norm_quant(t(3, 0), t(0), t(3, 0)), lambda: fq.rms_norm_bwd(t(3, 8), t(3, 8), t(8), t(3)),
            lambda: fq.gemm_swiglu(x, xs, w, ws), lambda: fq.gemm_swiglu_quant(x, xs, w, ws, with_gu=True),
            lambda: fq.grouped_gemm_swiglu(x, xs, t(2, 256, 256, dt=U8), t(2, 2, 2), off),
            lambda: fq.gemm_dgrad_swiglu(x, xs, t(128, 256, dt=U8), t(2, 1), gu, with_h=True),
            lambda: fq.grouped_gemm_dgrad_swiglu(x, xs, t(128, 512, dt=U8), t(4, 1), off, gu)]


@pytest.mark.parametrize("i", range(9))
def test_not_the_current_device(i):
    with current_device(1), pytest.raises(ValueError, match="current device is cuda:1"):
        calls()[i]()
