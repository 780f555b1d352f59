"""Gradient clipping against 64 bits: the norm is summed in 64 bits and rounded
once (2^-24), an output is off by the factor's and the product's rounding
(2^-23 together) and its type's half step."""

import numpy as np
import pytest
import torch

import fp8_fine_grained_quant_amd as fq
import moe_ref as ref
from gpu_util import DEV, log

pytestmark = pytest.mark.gpu


def make(sizes, seed, scale=0.02):
    r = np.random.Generator(np.random.PCG64([seed, len(sizes)]))
    return [np.float32(r.standard_normal(n) * scale) for n in sizes]


def check(host, max_norm, out_bf16, in_place=False, shift=0):
    """shift: every tensor starts that many elements into its allocation."""
    place = lambda n, dt: torch.full((n + shift + 16,), 7.0, dtype=dt, device=DEV)[shift:shift + n]
    grads = []
    for h in host:
        g = place(h.size, torch.float32)
        g.copy_(torch.from_numpy(h))
        grads.append(g)
    ot = torch.bfloat16 if out_bf16 else torch.float32
    bufs = [torch.full((h.size + shift + 16,), 7.0, dtype=ot, device=DEV) for h in host]
    out = grads if in_place else [b[shift:shift + h.size] for b, h in zip(bufs, host)]
    norm = fq.grad_clip(grads, max_norm, out=None if in_place else out)
    torch.cuda.synchronize()
    n64 = np.sqrt(sum((h.astype(np.float64) ** 2).sum() for h in host)) if host else 0.0
    assert norm.shape == () and norm.dtype == torch.float32
    assert abs(float(norm) - n64) <= 1.01 * ref.U32 * n64 + 2.0 ** -149, (float(norm), n64)
    c = 1.0 if n64 <= max_norm else max_norm / n64
    for i, (o, h) in enumerate(zip(out, host)):
        want = h.astype(np.float64) * c
        bound = (2.02 * ref.U32 * (c != 1.0) + (2.0 ** -8 if out_bf16 else 0.0)) * np.abs(want) + \
            (2.0 ** -133 if out_bf16 else 2.0 ** -149)
        err = np.abs(o.cpu().double().numpy() - want)
        assert (err <= bound).all(), (i, h.size, float((err - bound).max()))
        if not in_place:
            b = bufs[i]
            assert bool((b[:shift] == 7).all() and (b[shift + h.size:] == 7).all()), i
            assert np.array_equal(grads[i].cpu().numpy(), h), i


SIZES = [[1], [37], [8191, 8192, 8193], [4, 3, 2, 1, 0, 5], [100_003, 1, 70_000], [0], [0, 0, 7], list(range(1, 98)),
         [129] * 96, [5, 0] * 200 + [33], [1_000_001, 65537]]


@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{max(s)}")
@pytest.mark.parametrize("out_bf16", [False, True], ids=["f32", "bf16"])
def test_clip(sizes, out_bf16):
    host = make(sizes, 3)
    for max_norm in (0.5, 1e6, 0.0, float("inf")):
        check(host, max_norm, out_bf16)
    for shift in (1, 2, 3):
        check(host, 0.01, out_bf16, shift=shift)
    if not out_bf16:
        check(host, 0.01, False, in_place=True)
        check(host, 1e6, False, in_place=True, shift=1)
    log(f"clip {len(sizes)} tensors")


def test_many_rows_and_shapes():
    g = [torch.randn(33, 65, device=DEV), torch.randn(2, 3, 5, device=DEV), torch.randn((), device=DEV)]
    want = torch.sqrt(sum(x.double().square().sum() for x in g))
    out = [torch.empty_like(x, dtype=torch.bfloat16) for x in g]
    norm = fq.grad_clip(g, 1.0, out=out)
    assert abs(float(norm) - float(want)) <= 1.01 * ref.U32 * float(want)
    assert all(o.shape == x.shape for o, x in zip(out, g))


@pytest.mark.parametrize("scale", [1e-30, 1e25, 1e-41])
def test_no_overflow_or_underflow(scale):
    """Squares that FP32 cannot hold."""
    check(make([5000, 17], 4, scale), float(np.float32(scale)) * 3, False)


def test_no_tensors():
    norm = fq.grad_clip([], 1.0)
    assert float(norm) == 0.0


def test_not_finite():
    for bad, kept in ((float("nan"), "nan"), (float("inf"), "zero")):
        g = [torch.ones(1000, device=DEV), torch.ones(77, device=DEV)]
        g[1][5] = bad
        norm = fq.grad_clip(g, 1.0)
        assert not bool(torch.isfinite(norm))
        assert bool(torch.isnan(g[1][5]))
        assert bool(torch.isnan(g[0]).all()) if kept == "nan" else bool((g[0] == 0).all())


def test_repeatable():
    host = make([300_007, 12_345], 6)
    norms = set()
    for _ in range(3):
        g = [torch.from_numpy(h).to(DEV) for h in host]
        norms.add(float(fq.grad_clip(g, 0.1)))
    assert len(norms) == 1
