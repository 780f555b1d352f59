"""What the native calls of the routing operators refuse before any work: wrong
kinds of objects, missing outputs, sizes out of range (CPU tensors: nothing
reaches a device)."""

import subprocess
import sys

import pytest
import torch

import fp8_fine_grained_quant_amd as fq

u8, f32, bf16, i32, i64 = torch.uint8, torch.float32, torch.bfloat16, torch.int32, torch.int64


def z(*shape, dt=f32):
    return torch.zeros(shape, dtype=dt)


def refused(error, text, fn):
    with pytest.raises(error) as e:
        fn()
    assert text in str(e.value), str(e.value)


X, IDS, W = z(6, 32), z(6, 4, dt=i32), z(6, 4)


def test_not_tensors():
    refused(TypeError, "logits: expected a tensor", lambda: fq.moe_route([[1.0, 2.0]], 1))
    refused(ValueError, "logits is required", lambda: fq.moe_route(None, 1))
    refused(TypeError, "bias: expected a tensor", lambda: fq.moe_route(X, 2, bias=3.0))
    refused(TypeError, "integer", lambda: fq.moe_route(X, "2"))
    refused(ValueError, "relu", lambda: fq.moe_route(X, 2, score="relu"))
    refused(TypeError, "dst: expected a tensor", lambda: fq.moe_dispatch(X, [0, 1]))
    refused(ValueError, "weights is required", lambda: fq.moe_combine(z(24, 8), IDS, None))
    refused(TypeError, "out: expected a tensor", lambda: fq.grad_clip([z(3)], 1.0, out=[1]))
    refused(TypeError, "sequence", lambda: fq.grad_clip(5, 1.0))
    refused(TypeError, "arguments", lambda: fq._native().moe_combine(X))


def test_missing_outputs():
    refused(ValueError, "ids is required", lambda: fq.fp8q_moe_route(X, None, W))
    refused(ValueError, "weights is required", lambda: fq.fp8q_moe_route(X, IDS, None))
    refused(ValueError, "dlogits is required", lambda: fq.fp8q_moe_route_bwd(W, X, IDS, None))
    refused(ValueError, "offsets is required", lambda: fq.fp8q_moe_sort(IDS, 8, None, IDS))
    refused(ValueError, "dst is required", lambda: fq.fp8q_moe_sort(IDS, 8, z(9, dt=i32), None))
    refused(ValueError, "dx is required", lambda: fq.fp8q_moe_dispatch_bwd(z(24, 8), IDS, None))
    refused(ValueError, "y is required", lambda: fq.fp8q_moe_combine(z(24, 8), IDS, W, None))
    refused(ValueError, "dweights is required", lambda: fq.fp8q_moe_combine_bwd(z(6, 8), z(24, 8), IDS, W, None))
    refused(ValueError, "norm is required", lambda: fq.fp8q_grad_clip([], [], 1.0, None, z(8, dt=u8)))
    refused(ValueError, "q is required", lambda: fq.fp8q_moe_dispatch(X, IDS, scale=z(24, 1)))


def test_shapes_and_types():
    refused(ValueError, "2-D", lambda: fq.moe_route(z(6), 2))
    refused(ValueError, "2-D", lambda: fq.moe_combine(z(24), IDS, W))
    refused(TypeError, "torch.int64", lambda: fq.moe_sort(z(6, 4, dt=i64), 8))
    refused(TypeError, "torch.float32", lambda: fq.moe_sort(W, 8))
    refused(ValueError, "GPU tensors only", lambda: fq.moe_sort(IDS, 8))
    refused(ValueError, "GPU tensors only", lambda: fq.moe_route(X, 2))
    refused(ValueError, "GPU tensors only", lambda: fq.grad_clip([z(3)], 1.0))
    refused(ValueError, "weights", lambda: fq.moe_combine(z(24, 8), IDS, z(6, 3)))
    refused(TypeError, "weights", lambda: fq.moe_combine(z(24, 8), IDS, z(6, 4, dt=bf16)))
    refused(ValueError, "yp: shape (24, 7), expected (24, 8)", lambda: fq.moe_combine_bwd(z(6, 8), z(24, 7), IDS, W))
    refused(TypeError, "yp: dtype torch.bfloat16", lambda: fq.moe_combine_bwd(z(6, 8), z(24, 8, dt=bf16), IDS, W))


def test_tensors_without_memory():
    """A tensor that only has a shape is refused by an exception, with the
    interpreter's lock held again."""
    from torch._subclasses.fake_tensor import FakeTensorMode
    with FakeTensorMode(allow_non_fake_inputs=True):
        x, ids, w = torch.empty(6, 32, device="cuda"), torch.empty(6, 4, dtype=i32, device="cuda"), \
            torch.empty(6, 4, device="cuda")
    for fn in (lambda: fq.fp8q_moe_route(x, ids, w), lambda: fq.fp8q_moe_route_bwd(w, x, ids, x),
               lambda: fq.fp8q_moe_sort(ids, 4, torch.empty_like(ids).view(-1)[:5], ids),
               lambda: fq.moe_combine(torch.empty_like(x), ids, w)):
        with pytest.raises((RuntimeError, ValueError, TypeError)):
            fn()
    meta = torch.empty(6, 32, device="meta")
    refused(ValueError, "GPU tensors only", lambda: fq.moe_route(meta, 2))


@pytest.mark.gpu
def test_refusals_on_the_gpu():
    d = lambda t: t.cuda()
    shape = "FP8Q_ERR_SHAPE"
    for k in (0, -1, 33, 1 << 40):
        refused(fq.Fp8qError, shape, lambda: fq.moe_route(d(z(6, 64)), k))
    refused(fq.Fp8qError, shape, lambda: fq.moe_route(d(X), 2, scale=float("nan")))
    refused(fq.Fp8qError, "FP8Q_ERR_STRIDE", lambda: fq.moe_route(d(z(1, 32)).expand(6, 32), 2))
    refused(ValueError, "contiguous rows", lambda: fq.moe_route(d(z(32, 6)).t(), 2))
    refused(TypeError, "unsupported dtype torch.float16", lambda: fq.moe_route(d(X).half(), 2))
    refused(ValueError, "must be contiguous", lambda: fq.moe_dispatch(d(X), d(z(4, 6, dt=i32)).t()))
    refused(ValueError, "24 pairs, 2000 experts", lambda: fq.moe_sort(d(IDS), 2000))
    refused(fq.Fp8qError, "FP8Q_ERR_NULL", lambda: fq.fp8q_moe_dispatch(d(X), d(IDS)))
    refused(fq.Fp8qError, shape, lambda: fq.grad_clip([d(z(3))], -1.0))
    refused(TypeError, "torch.float16", lambda: fq.grad_clip([d(z(3))], 1.0, out=[d(z(3)).half()]))
    refused(ValueError, "GPU tensors only", lambda: fq.grad_clip([d(z(3)), z(3)], 1.0))


def test_missing_build_is_named(tmp_path):
    """Without the built module the calls fail by name; there is no slower path."""
    code = ("import fp8_fine_grained_quant_amd as fq, torch\n"
            f"fq.CALLS_PATH = {str(tmp_path / '_calls.so')!r}\n"
            "try:\n    fq.moe_sort(torch.zeros(2, 2, dtype=torch.int32), 4)\n"
            "except RuntimeError as e:\n    assert 'not built' in str(e), e\nelse:\n    raise SystemExit(1)\n")
    assert subprocess.run([sys.executable, "-c", code]).returncode == 0


@pytest.mark.gpu
def test_made_rows_start_on_segments():
    """Rows and codes of any width feed the quantizers and the grouped products
    as they are (dense rows of 200 BF16 columns start off 16 bytes)."""
    x = torch.randn(300, 200, device="cuda").to(bf16)
    offsets, dst, _ = fq.moe_sort(torch.randint(0, 4, (300, 2), device="cuda").to(i32), 4)
    rows, q, s = fq.moe_dispatch_quant(x, dst)
    assert rows.shape == (600, 200) and rows.stride() == (224, 1) and q.stride() == (256, 1)
    q_t, _ = fq.quant_transpose_grouped(rows, offsets)
    assert q_t.shape[0] == 200
    assert fq.moe_dispatch(torch.randn(300, 256, device="cuda").to(bf16), dst).is_contiguous()
    again, scale = torch.empty(600, 208, dtype=u8, device="cuda")[:, :200], torch.empty(600, 2, device="cuda")
    fq.fp8q_quant_act_1x128(rows, again, scale)
    assert torch.equal(again, q) and torch.equal(scale, s)
