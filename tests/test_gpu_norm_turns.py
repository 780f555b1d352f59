"""RMS norm and its gradient where a block takes several rows in turn, and where
rows pass the caches (above 512 MB of matrices).

What one turn gives is compared with 64 bits in test_gpu_rms_norm.py.  A row's
results do not depend on its turn, its place or the way past the caches, so rows
of a large call have the bits of the same rows in small ones; samples of them are
compared with 64 bits as well.  dweight, which is added up over the turns, is
compared with 64 bits: a thread adds one row of every turn, a block its threads'
sums of a column (64 at most), the second
launch 1 / 32 of the blocks' parts (20 at most a compute unit) and then 32 sums
in 5 steps, of terms that are off by 3 U."""

import numpy as np
import pytest
import torch

import block_ref as ref
import fp8_fine_grained_quant_amd as fq
from gpu_util import DEV, log

pytestmark = pytest.mark.gpu
BF16, F32, U = torch.bfloat16, torch.float32, ref.U


def rows_of(rows, cols, dtype, seed, std=1.0, pad=0):
    """Rows `pad` elements apart, some channels and rows far larger than the rest."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.empty(rows, cols + pad, dtype=dtype, device=DEV)[:, :cols]
    for a in range(0, rows, 8192):
        part = torch.randn(min(8192, rows - a), cols, generator=g, device=DEV) * std
        part *= torch.where(torch.rand(len(part), 1, generator=g, device=DEV) < 0.02, 50.0, 1.0)
        part[:, ::37] *= 20.0
        x[a:a + len(part)] = part
    return x


def weight_of(cols):
    return 1 + 0.3 * torch.randn(cols, generator=torch.Generator(device=DEV).manual_seed(9), device=DEV)


def sample(rows):
    return sorted({0, 1, rows // 3, rows // 2, rows - 2, rows - 1} | set(range(5, rows, max(1, rows // 12))))


def check_dweight(dw, dy, x, rstd, what):
    rows, cols = x.shape
    want = torch.zeros(cols, dtype=torch.float64, device=DEV)
    mag = torch.zeros_like(want)
    for a in range(0, rows, 8192):
        p = dy[a:a + 8192].double() * (x[a:a + 8192].double() * rstd[a:a + 8192, None].double())
        want += p.sum(0)
        mag += p.abs().sum(0)
    units = torch.cuda.get_device_properties(0).multi_processor_count
    steps = rows // units + 1 + 64 + -(-20 * units // 32) + 5 + 3
    ref.close(dw, ref.f64(want), steps * U * ref.f64(mag) + ref.tiny(F32), what)


def check_rows(rows, cols, dtype, at_once):
    """Norm and gradient of one call against calls of at_once rows."""
    log(f"norm {rows}x{cols} {dtype}, {at_once} at once")
    x, w = rows_of(rows, cols, dtype, 1), weight_of(cols)
    res = rows_of(rows, cols, dtype, 2, pad=3)
    whole = fq.rms_norm_quant(x, w, res, eps=1e-5, with_output=True)
    plain = fq.rms_norm(x, w, eps=1e-5)
    for a in range(0, rows, at_once):
        part = slice(a, min(rows, a + at_once))
        few = fq.rms_norm_quant(x[part], w, res[part], eps=1e-5, with_output=True)
        assert all(torch.equal(v[part], f) for v, f in zip(whole, few)), part
        assert all(torch.equal(v[part], f) for v, f in zip(plain, fq.rms_norm(x[part], w, eps=1e-5)) if v is not None), part
    at = sample(rows)
    y, q, s, total, rstd = whole
    want, r = ref.norm(ref.f64(total[at]), ref.f64(w), float(np.float32(1e-5)))
    bound = 30 * U * np.abs(want) + ref.tiny(F32)
    ref.close(rstd[at], r, 28 * U * r, "rstd")
    ref.close(y[at], want, bound + ref.half_step(dtype) * np.abs(want) + ref.tiny(dtype), "y")
    ref.check_codes(q[at], s[at], want, bound, "codes")
    del whole, plain, y, q, s, res

    dy = rows_of(rows, cols, dtype, 3, std=0.01)
    dsum = rows_of(rows, cols, dtype, 4, std=0.01, pad=1)
    dx, q, s, dw = fq.rms_norm_bwd_quant(dy, total, w, rstd, dsum)
    plain = fq.rms_norm_bwd(dy, total, w, rstd)
    for a in range(0, rows, at_once):
        part = slice(a, min(rows, a + at_once))
        few = fq.rms_norm_bwd_quant(dy[part], total[part], w, rstd[part], dsum[part])
        assert all(torch.equal(v[part], f) for v, f in zip((dx, q, s), few)), part
        assert torch.equal(plain[0][part], fq.rms_norm_bwd(dy[part], total[part], w, rstd[part])[0]), part
    check_dweight(dw, dy, total, rstd, "dweight")
    assert torch.equal(plain[1], dw)
    want, mag, _, _ = ref.norm_bwd(*(ref.f64(t) for t in (dy[at], total[at], w, rstd[at])), ref.f64(dsum[at]))
    bound = 60 * U * mag + 2 * U * np.abs(want) + ref.tiny(F32)
    ref.close(dx[at], want, bound + ref.half_step(dtype) * (np.abs(want) + bound) + ref.tiny(dtype), "dx")
    ref.check_codes(q[at], s[at], want, bound, "gradient's codes")
    again = fq.rms_norm_bwd_quant(dy, total, w, rstd, dsum)
    assert all(torch.equal(a, b) for a, b in zip(again, (dx, q, s, dw)))


# On 256 compute units a turn of the norm is 512 rows (7168, 12345 and 16384
# columns), 768 (8193), 2560 (1027), 8192 (300), 16384 (200) or 32768 (20 and 3),
# one of the gradient half of that (512 of 8193, 1280 of 1027).  The small calls are
# one turn of both.
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("rows, cols, at_once", [(1801, 7168, 256), (1030, 8193, 256), (1153, 12345, 128),
                                                 (777, 16384, 256), (2999, 1027, 1000), (20_011, 300, 4096),
                                                 (40_001, 200, 8000), (70_001, 20, 16_000), (70_001, 3, 16_000)])
def test_turns(rows, cols, at_once, dtype):
    check_rows(rows, cols, dtype, at_once)


@pytest.mark.parametrize("rows, cols, at_once, dtype", [
    (16_384, 7168, 2048, BF16), (5001, 7168, 1000, F32), (70_001, 1027, 10_000, BF16), (35_003, 1027, 5000, F32),
    (350_003, 200, 50_000, BF16), (170_001, 200, 25_000, F32)])
def test_past_the_caches(rows, cols, at_once, dtype):
    """Four matrices above 512 MB pass the caches, those of the small calls do not."""
    size = 2 if dtype == BF16 else 4
    assert rows * cols * size * 4 > 512 << 20 > at_once * cols * size * 4
    check_rows(rows, cols, dtype, at_once)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("cols", [8197, 12345, 16384])
def test_in_place_of_long_rows(cols, dtype):
    """Rows of two pieces a thread: sum over x or residual, dx over dy, x or dsum
    (which FP32 rows read after the first piece has left)."""
    rows, w = 700, weight_of(cols)
    log(f"norm in place {rows}x{cols} {dtype}")
    x, res = rows_of(rows, cols, dtype, 1), rows_of(rows, cols, dtype, 2)
    y, total, rstd = fq.rms_norm(x, w, res)
    for which in (0, 1):
        given = [x.clone(), res.clone()]
        y2, rstd2 = torch.empty_like(x), torch.empty_like(rstd)
        fq.fp8q_rms_norm(given[0], w, 1e-6, y2, None, None, rstd2, residual=given[1], sum=given[which])
        assert torch.equal(given[which], total) and torch.equal(y2, y) and torch.equal(rstd2, rstd)
    dy, dsum = rows_of(rows, cols, dtype, 3, std=0.01), rows_of(rows, cols, dtype, 4, std=0.01)
    dx, dw = fq.rms_norm_bwd(dy, total, w, rstd, dsum)
    for which in range(3):
        given = [dy.clone(), total.clone(), dsum.clone()]
        dw2 = torch.empty_like(dw)
        room = torch.empty(fq.rms_norm_bwd_workspace(rows, cols), dtype=torch.uint8, device=DEV)
        fq.fp8q_rms_norm_bwd(given[0], given[1], w, rstd, dw2, room, given[which], dsum=given[2])
        assert torch.equal(given[which], dx) and torch.equal(dw2, dw)
