"""RMS norm with the residual's addition and codes, and its gradient, against 64
bits.

Bounds (U = 2^-24, relative): a row's squares are added in at most 50 steps
(16 of a thread's two pieces, 6 within a wave, 4 across the waves and a few of
scaling), all terms positive, and the root halves that: rstd is off by 28 U, y
by two products more, 30 U, beside its type's half step.  The gradient's mean is
off by 54 U of its terms' magnitudes; with the products around it dx is off by
60 U of its terms' magnitudes.  dweight adds its rows in at most rows + 40 steps
of terms that are off by 3 U."""

import numpy as np
import pytest
import torch

import block_ref as ref
import fp8_fine_grained_quant_amd as fq
from gpu_util import DEV, log

pytestmark = pytest.mark.gpu
BF16, F32, U = torch.bfloat16, torch.float32, ref.U


def rows_of(rows, cols, dtype, seed, std=1.0, pad=0, shift=0):
    """A matrix whose rows lie `pad` elements apart, the first one `shift` into
    its memory; values with large channels and rows."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g) * std
    x *= torch.where(torch.rand(cols, generator=g) < 0.05, 20.0, 1.0)
    x *= torch.where(torch.rand(rows, 1, generator=g) < 0.1, 50.0, 1.0)
    room = torch.full((rows * (cols + pad) + shift + 64,), 7.0, dtype=dtype, device=DEV)
    view = room[shift:shift + rows * (cols + pad)].view(rows, cols + pad)[:, :cols] if rows else \
        room[:0].view(0, cols)
    view.copy_(x)
    return view


def weight_of(cols, seed):
    return (1 + 0.3 * torch.randn(cols, generator=torch.Generator().manual_seed(seed))).to(DEV)


def check_forward(x, w, res, eps, y, q, s, total, rstd, what):
    t = x
    if res is not None:
        t = (x.float() + res.float()).to(x.dtype)
        assert torch.equal(total, t), what
    want, r = ref.norm(ref.f64(t), ref.f64(w), eps)
    ref.close(rstd, r, 28 * U * r, (what, "rstd"))
    bound = 30 * U * np.abs(want) + ref.tiny(F32)
    if y is not None:
        assert y.dtype == x.dtype
        ref.close(y, want, bound + ref.half_step(x.dtype) * np.abs(want) + ref.tiny(x.dtype), (what, "y"))
    if q is not None:
        ref.check_codes(q, s, want, bound, what)


SHAPES = [(1, 1), (1, 7), (3, 8), (2, 9), (5, 64), (4, 127), (4, 128), (7, 129), (2, 1000), (9, 1027), (3, 2047),
          (6, 4096), (5, 4099), (4, 7168), (100, 256), (33, 130), (70, 320), (1000, 20), (2, 8192), (3, 8193), (2, 12345), (2, 16384), (2500, 72), (1031, 640)]


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("rows, cols", SHAPES)
def test_forward(rows, cols, dtype):
    x, w = rows_of(rows, cols, dtype, 1), weight_of(cols, 2)
    res = rows_of(rows, cols, dtype, 3, pad=5, shift=3)
    y, total, rstd = fq.rms_norm(x, w)
    assert total is None
    check_forward(x, w, None, 1e-6, y, None, None, None, rstd, "rows")
    y2, q, s, total, rstd2 = fq.rms_norm_quant(x, w, res, eps=1e-3, with_output=True)
    check_forward(x, w, res, 1e-3, y2, q, s, total, rstd2, "both")
    none, q3, s3, total3, _ = fq.rms_norm_quant(x, w, res, eps=1e-3)
    assert none is None and torch.equal(q3, q) and torch.equal(s3, s) and torch.equal(total3, total)
    log(f"norm {rows}x{cols}")


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("rows, cols", SHAPES)
def test_backward(rows, cols, dtype):
    x, w = rows_of(rows, cols, dtype, 4, pad=1, shift=1), weight_of(cols, 5)
    dy, dsum = rows_of(rows, cols, dtype, 6, std=0.01), rows_of(rows, cols, dtype, 7, std=0.01, pad=3)
    rstd = torch.rsqrt(x.double().square().mean(1) + 1e-6).float()
    for given in (None, dsum):
        dx, dw = fq.rms_norm_bwd(dy, x, w, rstd, given)
        want, mag, wdw, mdw = ref.norm_bwd(*(ref.f64(t) for t in (dy, x, w, rstd)),
                                           None if given is None else ref.f64(given))
        bound = 60 * U * mag + 2 * U * np.abs(want) + ref.tiny(F32)
        rounded = bound + ref.half_step(dtype) * (np.abs(want) + bound) + ref.tiny(dtype)
        ref.close(dx, want, rounded, "dx")
        ref.close(dw, wdw, (rows + 43) * U * mdw + ref.tiny(F32), "dw")
        dx2, q, s, dw2 = fq.rms_norm_bwd_quant(dy, x, w, rstd, given)
        assert torch.equal(dx2, dx) and torch.equal(dw2, dw)
        ref.check_codes(q, s, want, bound, "codes")
        none, q3, s3, _ = fq.rms_norm_bwd_quant(dy, x, w, rstd, given, with_output=False)
        assert none is None and torch.equal(q3, q) and torch.equal(s3, s)


def test_gradient_against_differences():
    """The formula's dx and dw against central differences of the 64-bit norm."""
    r = np.random.default_rng(8)
    x, w, dy = r.standard_normal((3, 40)), 1 + 0.3 * r.standard_normal(40), r.standard_normal((3, 40))
    f = lambda x, w: (ref.norm(x, w, 1e-6)[0] * dy).sum()  # noqa: E731
    h = 1e-5
    num_x, num_w = np.zeros_like(x), np.zeros_like(w)
    for i in np.ndindex(x.shape):
        d = np.zeros_like(x)
        d[i] = h
        num_x[i] = (f(x + d, w) - f(x - d, w)) / (2 * h)
    for i in range(40):
        d = np.zeros(40)
        d[i] = h
        num_w[i] = (f(x, w + d) - f(x, w - d)) / (2 * h)
    x32, w32, dy32 = (torch.from_numpy(v).float().to(DEV) for v in (x, w, dy))
    rstd = torch.rsqrt(x32.double().square().mean(1) + 1e-6).float()
    dx, dw = fq.rms_norm_bwd(dy32, x32, w32, rstd)
    # differences: h^2 of the third derivative and 2^-52 / h; inputs rounded to FP32
    assert np.abs(ref.f64(dx) - num_x).max() <= 1e-5 and np.abs(ref.f64(dw) - num_w).max() <= 1e-5


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("cols", [200, 7168])
def test_outputs_in_place_and_strided(dtype, cols):
    """sum over x or residual, dx over dy, x or dsum; nothing beside the outputs is written."""
    x, res, w = rows_of(9, cols, dtype, 1), rows_of(9, cols, dtype, 2), weight_of(cols, 3)
    y, total, rstd = fq.rms_norm(x, w, res)
    for which in (0, 1):
        a, b = x.clone(), res.clone()
        y2, rstd2 = rows_of(9, cols, dtype, 0, pad=3, shift=1), torch.empty_like(rstd)
        q = torch.full((9, cols + 7), 99, dtype=torch.uint8, device=DEV)
        s = torch.full((9, -(-cols // 128) + 2), 7.0, device=DEV)
        fq.fp8q_rms_norm(a, w, 1e-6, y2, q[:, :cols], s[:, :-2], rstd2, residual=b, sum=(a, b)[which])
        assert torch.equal((a, b)[which], total) and torch.equal(y2, y) and torch.equal(rstd2, rstd)
        assert bool((q[:, cols:] == 99).all() and (s[:, -2:] == 7).all())
    dy, dsum = rows_of(9, cols, dtype, 4), rows_of(9, cols, dtype, 5)
    dx, dw = fq.rms_norm_bwd(dy, total, w, rstd, dsum)
    for which in range(3):
        given = [dy.clone(), total.clone(), dsum.clone()]
        dw2 = torch.empty_like(dw)
        room = torch.empty(fq.rms_norm_bwd_workspace(9, cols), dtype=torch.uint8, device=DEV)
        fq.fp8q_rms_norm_bwd(given[0], given[1], w, rstd, dw2, room, given[which], dsum=given[2])
        assert torch.equal(given[which], dx) and torch.equal(dw2, dw)
        assert all(torch.equal(v, o) for i, (v, o) in enumerate(zip(given, (dy, total, dsum))) if i != which)


def test_special_rows():
    """Zeros, the largest and smallest magnitudes whose squares FP32 holds, a NaN row beside others."""
    x = torch.randn(8, 256, device=DEV)
    x[0] = 0
    x[1] = 1e17
    x[2] = 1e-18
    x[3, 5] = float("nan")
    x[4] = 0
    x[4, 255] = -3.0
    w = weight_of(256, 1)
    y, q, s, _, rstd = fq.rms_norm_quant(x, w, with_output=True)
    keep = [0, 1, 2, 4, 5, 6, 7]
    want, r = ref.norm(ref.f64(x[keep]), ref.f64(w), float(np.float32(1e-6)))
    ref.close(rstd[keep], r, 28 * U * r, "rstd")
    ref.close(y[keep], want, 30 * U * np.abs(want) + 2.0 ** -149, "y")
    ref.check_codes(q[keep], s[keep], want, 30 * U * np.abs(want) + 2.0 ** -149, "codes")
    assert bool(torch.isnan(y[3]).all()) and bool(torch.isnan(rstd[3]))
    assert bool((y[0] == 0).all()) and bool((q[0] == 0).all())


def test_no_rows_and_no_columns():
    w = weight_of(300, 1)
    x = torch.empty(0, 300, device=DEV)
    y, q, s, total, rstd = fq.rms_norm_quant(x, w, x, with_output=True)
    assert y.shape == (0, 300) and q.shape == (0, 300) and s.shape == (0, 3) and rstd.shape == (0,)
    dx, dw = fq.rms_norm_bwd(x, x, w, rstd)
    assert dx.shape == (0, 300) and bool((dw == 0).all()) and dw.shape == (300,)
    e = torch.empty(4, 0, device=DEV)
    fq.rms_norm(e, w[:0])
    assert fq.rms_norm_bwd(e, e, w[:0], torch.empty(4, device=DEV))[1].shape == (0,)


def test_repeatable_and_captured():
    """The same bits again, and from a graph replayed with other inputs written between."""
    x, res, w = rows_of(700, 1000, BF16, 1), rows_of(700, 1000, BF16, 2), weight_of(1000, 3)
    dy = rows_of(700, 1000, BF16, 4)

    def step():
        y, q, s, total, rstd = fq.rms_norm_quant(x, w, res, with_output=True)
        return [y, q, s, total, rstd, *fq.rms_norm_bwd_quant(dy, total, w, rstd, res)]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for seed in (11, 12, 13):
        x.copy_(rows_of(700, 1000, BF16, seed))
        dy.copy_(rows_of(700, 1000, BF16, seed + 5))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in held]
        for i, (a, b) in enumerate(zip(got, step())):
            assert torch.equal(a, b), (seed, i)
