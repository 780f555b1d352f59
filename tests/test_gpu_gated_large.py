"""The gated block and its gradient in the large tiles, dense and by expert, and in
the small tiles of every height by expert, against 64 bits (bounds: block_ref).

The large tiles have an instance for scale rows of whole 16-byte blocks (chunks of
the contraction a multiple of 4) and one for others, and the gradient a tile 256
columns wide; by expert, a tile begins at its expert's first row, and a strip of 64
rows behind its last one only helps to load."""

import numpy as np
import pytest
import torch

import block_ref as ref
import fp8_fine_grained_quant_amd as fq
from gpu_util import log
from test_gpu_swiglu import (check_block, check_gradient, gradient_operands, offsets_of, operands, weight_values)

pytestmark = pytest.mark.gpu


def with_tile(tile, run):
    fq.set_gemm_tile(tile)
    try:
        return run()
    finally:
        fq.set_gemm_tile("auto")


def parts(counts):
    ends = np.cumsum(counts)
    return [(e, slice(int(ends[e]) - n, int(ends[e]))) for e, n in enumerate(counts) if n]


def check_experts(counts, f, k, ops, outs):
    xq, xs, wq, ws = ops
    h, gu, q, s = outs
    for e, p in parts(counts):
        check_block(xq[p], xs[p], wq[e], ws[e], h[p], gu[p], q[p], s[p])


def check_expert_gradients(counts, n, ops, outs):
    dyq, dys, wt, ws, gu = ops
    dgu, h = outs
    for e, p in parts(counts):
        check_gradient(dyq[p], dys[p], weight_values(wt, ws, n, e), gu[p], dgu[p], h[p])


# ragged, empty, one row, whole tiles, a whole strip and one row more
COUNTS = [[600, 0, 257, 1, 300, 64], [0, 0, 512, 65, 0], [129, 128, 127, 0, 193, 192, 256], [1000]]


@pytest.mark.parametrize("f, k", [(128, 128), (256, 512), (384, 640), (512, 1024), (128, 1536), (256, 2048)])
@pytest.mark.parametrize("counts", COUNTS, ids=str)
def test_block_by_expert(counts, f, k):
    log(f"gated block by expert {counts} {f}x{k}, large tiles")
    ops, off = operands(sum(counts), f, k, len(counts)), offsets_of(counts)
    run = lambda: fq.grouped_gemm_swiglu_quant(*ops, off, with_output=True, with_gu=True)  # noqa: E731
    outs = with_tile("256x128", run)
    check_experts(counts, f, k, ops, outs)
    assert all(torch.equal(a, b) for a, b in zip(outs, run()))  # the tiles that the sizes ask for: the same bits


@pytest.mark.parametrize("tile", ["256x128", "256x256"])
@pytest.mark.parametrize("n, f", [(128, 256), (512, 256), (512, 384), (640, 512), (1024, 512), (1536, 256)])
@pytest.mark.parametrize("counts", COUNTS, ids=str)
def test_gradient_by_expert(counts, n, f, tile):
    log(f"gradient by expert {counts} {n}x{f}, {tile}")
    ops, off = gradient_operands(sum(counts), n, f, len(counts)), offsets_of(counts)
    run = lambda: fq.grouped_gemm_dgrad_swiglu(*ops[:4], off, ops[4], with_h=True)  # noqa: E731
    outs = with_tile(tile, run)
    check_expert_gradients(counts, n, ops, outs)
    assert all(torch.equal(a, b) for a, b in zip(outs, run()))
    # over its input, and without h
    gu = ops[4].clone()
    with_tile(tile, lambda: fq.fp8q_grouped_gemm_dgrad_swiglu(*ops[:4], off, gu, gu))
    assert torch.equal(gu, outs[0])


@pytest.mark.parametrize("m, n, f", [(257, 512, 256), (300, 1024, 768), (1000, 1536, 512), (64, 2048, 256),
                                     (513, 128 * 21, 256), (1, 512, 512)])
def test_wide_gradient(m, n, f):
    """The 256 x 256 tile (scale rows of whole blocks), and the narrow one where they are not."""
    log(f"gradient {m}x{n}x{f}, 256x256")
    dyq, dys, wt, ws, gu = gradient_operands(m, n, f)
    run = lambda: fq.gemm_dgrad_swiglu(dyq, dys, wt, ws, gu, with_h=True)  # noqa: E731
    dgu, h = with_tile("256x256", run)
    check_gradient(dyq, dys, weight_values(wt, ws, n), gu, dgu, h)
    for other in ("256x128", "auto"):
        assert all(torch.equal(a, b) for a, b in zip((dgu, h), with_tile(other, run)))
    given = gu.clone()
    with_tile("256x256", lambda: fq.fp8q_gemm_dgrad_swiglu(dyq, dys, wt, ws, given, given))
    assert torch.equal(given, dgu)


# By the rule, on 256 compute units: large tiles of both (the gradient's 256 x 256),
# with skewed and with equal counts.
@pytest.mark.parametrize("counts", [[4000, 1, 0, 2047, 900, 300, 700, 244], [1024] * 8], ids=str)
def test_training_sizes_by_expert(counts):
    f, k, m = 2048, 512, sum(counts)
    log(f"training sizes by expert {counts}")
    ops, off = operands(m, f, k, len(counts)), offsets_of(counts)
    check_experts(counts, f, k, ops, fq.grouped_gemm_swiglu_quant(*ops, off, with_output=True, with_gu=True))
    ops = gradient_operands(m, k, f, len(counts))
    check_expert_gradients(counts, k, ops, fq.grouped_gemm_dgrad_swiglu(*ops[:4], off, ops[4], with_h=True))


def test_training_size_dense():
    """8192 rows, by the rule: the block with its codes, the gradient's 256 x 256 tile."""
    m, f, k = 8192 + 33, 2048, 512
    log("training size, dense")
    ops = operands(m, f, k)
    check_block(*ops, *fq.gemm_swiglu_quant(*ops, with_output=True, with_gu=True))
    dyq, dys, wt, ws, gu = gradient_operands(m, k, f)
    check_gradient(dyq, dys, weight_values(wt, ws, k), gu, *fq.gemm_dgrad_swiglu(dyq, dys, wt, ws, gu, with_h=True))


# By the rule, on 256 compute units, tiles of 64 and of 128 rows.
@pytest.mark.parametrize("counts, f, k", [([300, 0, 1, 500, 64, 65, 40, 30], 1024, 2048), ([700, 201, 600, 400], 1024, 640),
                                          ([97, 0, 129, 74], 4096, 256), ([40, 0, 128, 1, 2, 99, 17, 13], 4096, 128),
                                          ([80, 0, 90, 1, 2, 97, 17, 13], 4096, 384)], ids=str)
def test_small_tiles_by_expert(counts, f, k):
    m, off = sum(counts), offsets_of(counts)
    log(f"small tiles by expert {counts} {f}x{k}")
    ops = operands(m, f, k, len(counts))
    grads = gradient_operands(m, k, f, len(counts))

    def run():
        return (*fq.grouped_gemm_swiglu_quant(*ops, off, with_output=True, with_gu=True),
                *fq.grouped_gemm_dgrad_swiglu(*grads[:4], off, grads[4], with_h=True))

    outs = run()
    check_experts(counts, f, k, ops, outs[:4])
    check_expert_gradients(counts, k, grads, outs[4:])
    assert all(torch.equal(a, b) for a, b in zip(outs, with_tile("256x128", run)))
