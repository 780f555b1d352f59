"""RMS norm of rows without columns."""

import pytest
import torch

import fp8_fine_grained_quant_amd as fq
from gpu_util import DEV

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def test_no_columns():
    """rstd of rows without columns is made of nothing: zeros, not what lay there."""
    for dtype in (BF16, F32):
        e, w = torch.empty(300, 0, dtype=dtype, device=DEV), torch.empty(0, device=DEV)
        for residual in (None, e):
            before = torch.full((300,), 7.0, device=DEV)
            del before  # its memory is what the call is given next
            y, total, rstd = fq.rms_norm(e, w, residual)
            assert y.shape == (300, 0) and bool((rstd == 0).all())
            before = torch.full((300,), 7.0, device=DEV)
            del before
            assert bool((fq.rms_norm_quant(e, w, residual)[4] == 0).all())
            # given outputs are left alone
            held = torch.full((300,), 7.0, device=DEV)
            fq.fp8q_rms_norm(e, w, 1e-6, torch.empty_like(e), None, None, held, residual=residual,
                             sum=None if residual is None else torch.empty_like(e))
            assert bool((held == 7).all())
