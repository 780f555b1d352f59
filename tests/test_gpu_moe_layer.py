"""The routing operators together with the grouped FP8 products, as the example
layer runs them: its gradients against the 64-bit formulas on the values that
the products took and gave, and a short training."""

import os
import sys

import numpy as np
import pytest
import torch

import fp8_fine_grained_quant_amd as fq
import moe_ref as ref

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import moe_layer  # noqa: E402

pytestmark = pytest.mark.gpu


def f64(t):
    return t.detach().cpu().double().numpy()


def test_layer_against_the_formulas():
    """With the experts' rows as the layer has them, the rest of the pass is
    linear algebra and the router: bounds as in the operators' own tests."""
    t, h, n, e, k = 300, 256, 128, 8, 3
    layer = moe_layer.MoELayer(h, n, e, k)
    layer.bias.copy_(torch.linspace(-0.2, 0.2, e))
    x = torch.randn(t, h, device="cuda").to(torch.bfloat16)
    y, kept = layer.forward(x)
    _, logits, ids, w, offsets, dst, rows, yp, _, _ = kept
    ids_ref, w_ref = ref.route(f64(logits), k, True, f64(layer.bias), True)
    assert np.array_equal(ids.cpu().numpy(), ids_ref)
    # a sigmoid, a division and a sum of k: under 40 roundings of 2^-24
    assert (np.abs(f64(w) - w_ref) <= 40 * ref.U32 * w_ref).all()
    off_ref, dst_ref, _ = ref.sort(ids_ref, e, True)
    assert np.array_equal(offsets.cpu().numpy(), off_ref) and np.array_equal(dst.cpu().numpy(), dst_ref)
    terms = ref.fetch(f64(yp), dst_ref) * f64(w)[:, :, None]
    want = terms.sum(1)
    assert (np.abs(f64(y) - want) <= (k + 1) * ref.U32 * 1.01 * np.abs(terms).sum(1) + 2.0 ** -8 * np.abs(want)).all()
    dy = torch.randn(t, n, device="cuda").to(torch.bfloat16)
    _, drouter, dweight = layer.backward(dy, kept)
    dots = f64(dy)[:, None] * ref.fetch(f64(yp), dst_ref)
    dw = dots.sum(2)
    # dw is off by (n / 64 + 32) 2^-24 of its terms' magnitudes; the router's
    # gradient weighs those errors like the dw themselves (their magnitudes)
    err = (n / 64 + 32 + 120) * ref.U32
    _, mag = ref.route_bwd(np.abs(dots).sum(2), f64(logits), ids_ref, True, True, 1.0)
    dl, _ = ref.route_bwd(dw, f64(logits), ids_ref, True, True, 1.0)
    x64 = f64(x)
    bound = err * mag.T @ np.abs(x64) + 2 * t * ref.U32 * np.abs(dl).T @ np.abs(x64)
    assert (np.abs(f64(drouter) - dl.T @ x64) <= bound).all()
    # the experts' gradient: both operands quantized, each value by at most
    # 2^-4 of itself or half the least step of its 128 tokens' largest
    g64 = ref.spread(f64(dy)[:, None] * f64(w)[:, :, None], dst_ref)
    r64 = ref.spread(x64[:, None], dst_ref)
    for ex in range(e):
        a, b = g64[off_ref[ex]:off_ref[ex + 1]], r64[off_ref[ex]:off_ref[ex + 1]]
        got = f64(dweight).reshape(e, n, h)[ex]
        ea = 2.0 ** -4 * np.abs(a) + 2.0 ** -8 * np.abs(a) + 2.0 ** -18 * np.abs(a).max(initial=0)
        eb = 2.0 ** -4 * np.abs(b) + 2.0 ** -18 * np.abs(b).max(initial=0)
        bound = ea.T @ np.abs(b) + np.abs(a).T @ eb + ea.T @ eb + 2.0 ** -9 * np.abs(a).T @ np.abs(b)
        assert (np.abs(got - a.T @ b) <= bound).all(), ex


def test_training_lowers_the_loss_and_clips():
    losses = moe_layer.train(40, say=None)
    assert all(np.isfinite(losses)) and np.mean(losses[-5:]) < 0.8 * np.mean(losses[:5]), (losses[:5], losses[-5:])
    layer = moe_layer.MoELayer(256, 128, 4, 2)
    grads = [torch.randn_like(layer.router), torch.randn_like(layer.weight)]
    want = float(torch.sqrt(sum(g.double().square().sum() for g in grads)))
    norm = layer.update(grads, torch.tensor([0, 5, 9, 9, 20], dtype=torch.int32, device="cuda"))
    assert abs(float(norm) - want) <= 2 * ref.U32 * want
    after = float(torch.sqrt(sum(g.double().square().sum() for g in grads)))
    assert abs(after - 1.0) <= 1e-6
    assert torch.equal(layer.bias.cpu(), torch.tensor([0.0, 1e-3, 1e-3, -1e-3]))
