"""Gradient clipping where max_norm / norm is too small for FP32, and norms
beyond it: an output is max_norm / norm in 64 bits times the gradient, rounded
to FP32 (2^-24) and to its type (half a step); the factor's and the product's
own roundings are 2^-52."""

import numpy as np
import pytest
import torch

import fp8_fine_grained_quant_amd as fq
from gpu_util import DEV

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24


def expect(host, max_norm, out_bf16, in_place=False):
    grads = [torch.from_numpy(h).to(DEV) for h in host]
    ot = torch.bfloat16 if out_bf16 else torch.float32
    out = grads if in_place else [torch.empty_like(g, dtype=ot) for g in grads]
    norm = fq.grad_clip(grads, max_norm, out=None if in_place else out)
    n64 = float(np.sqrt(sum((h.astype(np.float64) ** 2).sum() for h in host)))
    assert n64 > max_norm
    if n64 < 3.4e38:
        assert abs(float(norm) - n64) <= 1.01 * U32 * n64
    else:
        assert float(norm) == float("inf")
    for o, h in zip(out, host):
        want = h.astype(np.float64) * (max_norm / n64)
        bound = (1.01 * U32 + (2.0 ** -8 if out_bf16 else 0.0)) * np.abs(want) + (2.0 ** -133 if out_bf16 else 2.0 ** -149)
        err = np.abs(o.double().cpu().numpy() - want)
        assert (err <= bound).all(), (max_norm, float((err / np.maximum(np.abs(want), 1e-300)).max()))


@pytest.mark.parametrize("out", ["f32", "bf16", "in place"])
@pytest.mark.parametrize("max_norm", [1e-2, 1e-4, 1e-6, 1e-10, 1e-30])
@pytest.mark.parametrize("scale", [1e34, 1e37], ids=str)
def test_small_factor(scale, max_norm, out):
    """1e37 makes a norm beyond FP32 (the norm is then infinite, the outputs are
    not); the factors go from 1e-36 to 1e-69."""
    r = np.random.Generator(np.random.PCG64(7))
    host = [np.float32(r.standard_normal(n) * scale) for n in (9001, 17, 3, 0, 20_000)]
    expect(host, max_norm, out == "bf16", out == "in place")


def test_factor_next_to_one():
    """A norm barely above the bound: in place the gradients change by less than
    FP32 holds or by one rounding, never by more."""
    h = np.float32(np.random.Generator(np.random.PCG64(8)).standard_normal(5000))
    n64 = float(np.sqrt((h.astype(np.float64) ** 2).sum()))
    for step in (1e-3, 1e-7, 1e-9, 1e-12):
        for in_place in (False, True):
            expect([h], n64 * (1 - step), False, in_place)
