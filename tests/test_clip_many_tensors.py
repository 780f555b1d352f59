"""Clipping many tensors: the partial sums that every block of the second pass
adds up do not grow with their number."""

import numpy as np
import pytest
import torch

import fp8_fine_grained_quant_amd as fq


def test_workspace_of_many():
    """A batch of tensors takes its table (96 tensors of 22 bytes and a few
    more), no partial sums of its own."""
    need = fq.grad_clip_workspace
    assert need(0) == 0 and need(96) == need(1)
    assert need(97) - need(96) < 96 * 24
    assert need(96 * 1000) - need(96) == 999 * (need(97) - need(96))


@pytest.mark.gpu
@pytest.mark.parametrize("count", [97, 1000, 5000])
@pytest.mark.parametrize("out_bf16", [False, True], ids=["f32", "bf16"])
def test_many(count, out_bf16):
    """Batches of fewer and of more chunks than the batches before, empty ones
    among them; in 64 bits as the other clipping tests."""
    r = np.random.Generator(np.random.PCG64(count))
    sizes = [int(r.integers(0, 40_000)) if (i // 96) % 3 == 1 else int(r.integers(0, 300)) for i in range(count)]
    sizes[200:500] = [0] * len(sizes[200:500])
    host = [np.float32(r.standard_normal(n) * 0.02) for n in sizes]
    flat = torch.from_numpy(np.concatenate(host)).cuda()
    grads = [g.clone() for g in flat.split(sizes)]
    out = [torch.empty_like(g, dtype=torch.bfloat16) for g in grads] if out_bf16 else None
    norm = fq.grad_clip(grads, 0.75, out=out)
    n64 = float(np.sqrt(sum((h.astype(np.float64) ** 2).sum() for h in host)))
    assert abs(float(norm) - n64) <= 1.01 * 2.0 ** -24 * n64
    got = torch.cat(out or grads).double().cpu().numpy()
    want = np.concatenate(host).astype(np.float64) * min(1.0, 0.75 / n64)
    bound = (1.01 * 2.0 ** -24 + (2.0 ** -8 if out_bf16 else 0.0)) * np.abs(want) + \
        (2.0 ** -133 if out_bf16 else 2.0 ** -149)
    assert (np.abs(got - want) <= bound).all()


@pytest.mark.gpu
def test_repeatable():
    gen = torch.Generator(device="cuda").manual_seed(3)
    grads = [torch.randn(9000 + i, generator=gen, device="cuda") for i in range(400)]
    norms = set()
    for _ in range(3):
        out = [torch.empty_like(g) for g in grads]
        norms.add(float(fq.grad_clip(grads, 1.0, out=out)))
    assert len(norms) == 1
