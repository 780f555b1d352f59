"""The gated feed-forward block and its gradient, dense and by expert, against 64
bits on the dequantized operands.  Bounds: block_ref (the products' own, carried
through the block's derivative), beside half a step of BF16."""

import numpy as np
import pytest
import torch

import block_ref as ref
import fp8_fine_grained_quant_amd as fq
from gpu_util import DEV, log

pytestmark = pytest.mark.gpu
BF16, U8, U = torch.bfloat16, torch.uint8, ref.U


def few(m, f, k):
    """Whether the kernel for few rows, whose products are exact, takes these
    sizes: it is the one that needs room for codes."""
    return fq.gemm_swiglu_workspace(m, f, k, True) > 0


def operands(m, f, k, experts=0, seed=1, std=1.0):
    """Codes and scales of x [m, k] and of the stacked weights [experts, 2f, k]."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(m, k, generator=g) * std
    x *= torch.where(torch.rand(k, generator=g) < 0.02, 20.0, 1.0)
    e = max(1, experts)
    w = torch.randn(e * 2 * f, k, generator=g) * k ** -0.5
    xq, xs = fq.quant_act_1x128(x.to(DEV))
    wq, ws, _ = fq.quant_weight_128x128(w.to(DEV), transpose=False)
    if experts:
        wq, ws = wq.view(e, 2 * f, k), ws.view(e, 2 * f // 128, k // 128)
    return xq, xs, wq, ws


def reference(xq, xs, wq, ws, exact):
    """(g, its bound, u, its bound) of dense operands."""
    g, mag = ref.product(ref.values(xq, xs), ref.values(wq, ws, 128))
    f, err = g.shape[1] // 2, ref.product_error(mag, xq.shape[1] // 128, exact)
    return g[:, :f], err[:, :f], g[:, f:], err[:, f:]


def rounded(v, bound):
    return bound + 2.0 ** -8 * (np.abs(v) + bound) + ref.tiny(BF16)


def check_block(xq, xs, wq, ws, h=None, gu=None, q=None, s=None, exact=False):
    g, eg, u, eu = reference(xq, xs, wq, ws, exact)
    if gu is not None:
        ref.close(gu, np.concatenate([g, u], 1), rounded(np.concatenate([g, u], 1), np.concatenate([eg, eu], 1)), "gu")
    want, err = ref.block(g, u, eg, eu)
    if h is not None:
        ref.close(h, want, rounded(want, err), "h")
    if q is not None:
        ref.check_codes(q, s, want, err + ref.tiny(torch.float32), "codes")


DENSE = [(1, 128, 128), (2, 128, 384), (8, 2048, 1024), (15, 256, 640), (16, 384, 7168), (17, 128, 256), (31, 256, 512),
         (33, 640, 896), (48, 128, 1152), (64, 512, 2048), (65, 128, 128), (65, 256, 640), (100, 384, 512),
         (256, 128, 1024), (257, 256, 384), (300, 640, 1792), (1000, 128, 256), (513, 1024, 2048), (3, 128, 131072 // 8),
         (40, 128, 9 * 1024), (130, 128, 11 * 1024), (16, 8192, 128), (1300, 2048, 256), (2000, 1024, 896)]


@pytest.mark.parametrize("m, f, k", DENSE)
def test_block(m, f, k):
    ops = operands(m, f, k)
    h, gu, q, s = fq.gemm_swiglu_quant(*ops, with_output=True, with_gu=True)
    check_block(*ops, h, gu, q, s, exact=few(m, f, k))
    # each output alone is what it is beside the others
    h2, none = fq.gemm_swiglu(*ops)
    assert none is None and torch.equal(h2, h)
    h3, gu3 = fq.gemm_swiglu(*ops, with_gu=True)
    assert torch.equal(h3, h) and torch.equal(gu3, gu)
    none, none2, q4, s4 = fq.gemm_swiglu_quant(*ops)
    assert none is None and none2 is None and torch.equal(q4, q) and torch.equal(s4, s)
    log(f"swiglu {m}x{f}x{k}")


def test_both_kernels_are_taken():
    """Few rows of every width go to one, many rows to the other, and the cases
    above have both on either side."""
    assert few(1, 128, 128) and few(8, 2048, 7168) and few(64, 2048, 7168) and not few(4096, 2048, 7168)
    assert {few(*c) for c in DENSE if c[0] > 64} == {few(*c) for c in DENSE if c[0] <= 64} == {True, False}


def with_large_tiles(run):
    fq.set_gemm_tile("256x128")
    try:
        return run()
    finally:
        fq.set_gemm_tile("auto")


@pytest.mark.parametrize("chunks", list(range(1, 15)) + [56])
@pytest.mark.parametrize("m, f", [(700, 1024), (1000, 2048), (1025, 2048)])
def test_small_and_large_tiles_agree(m, f, chunks):
    """Tiles of every height (32, 64 and 128 rows, by the sizes) give the large
    ones' bits, for every number of chunks that the pipeline ends with."""
    k = 128 * chunks
    ops = operands(m, f, k)
    both = [run() for run in (lambda: fq.gemm_swiglu_quant(*ops, with_output=True, with_gu=True),
                              lambda: with_large_tiles(lambda: fq.gemm_swiglu_quant(*ops, with_output=True, with_gu=True)))]
    assert all(torch.equal(a, b) for a, b in zip(*both))
    dyq, dys, wt, ws, gu = gradient_operands(m, k, f)
    small = fq.gemm_dgrad_swiglu(dyq, dys, wt, ws, gu, with_h=True)
    large = with_large_tiles(lambda: fq.gemm_dgrad_swiglu(dyq, dys, wt, ws, gu, with_h=True))
    assert all(torch.equal(a, b) for a, b in zip(small, large))


def offsets_of(counts):
    return torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32, device=DEV)


GROUPED = [([5], 128, 128), ([0, 3, 0], 256, 384), ([70, 0, 1, 300, 128], 128, 512), ([256, 257, 0, 0, 40], 384, 640),
           ([0, 0, 0, 33], 128, 1024), ([1] * 9, 256, 256)]


@pytest.mark.parametrize("counts, f, k", GROUPED, ids=str)
def test_block_by_expert(counts, f, k):
    xq, xs, wq, ws = operands(sum(counts), f, k, len(counts))
    off = offsets_of(counts)
    h, gu, q, s = fq.grouped_gemm_swiglu_quant(xq, xs, wq, ws, off, with_output=True, with_gu=True)
    at = 0
    for e, n in enumerate(counts):
        if n:
            part = slice(at, at + n)
            check_block(xq[part], xs[part], wq[e], ws[e], h[part], gu[part], q[part], s[part])
        at += n
    h2, gu2 = fq.grouped_gemm_swiglu(xq, xs, wq, ws, off, with_gu=True)
    assert torch.equal(h2, h) and torch.equal(gu2, gu)
    assert torch.equal(fq.grouped_gemm_swiglu(xq, xs, wq, ws, off)[0], h)


@pytest.mark.parametrize("f, k", [(128, 128), (512, 640), (1024, 1792)])
@pytest.mark.parametrize("counts", [[1] * 20, [33, 0, 64, 65, 1], [130, 0, 0, 200, 100, 70], [0, 500, 3, 0]], ids=str)
def test_small_and_large_tiles_agree_by_expert(counts, f, k):
    m, e, off = sum(counts), len(counts), offsets_of(counts)
    ops = operands(m, f, k, e)
    grads = gradient_operands(m, k, f, e)

    def run():
        return (*fq.grouped_gemm_swiglu_quant(*ops, off, with_output=True, with_gu=True),
                *fq.grouped_gemm_dgrad_swiglu(*grads[:4], off, grads[4], with_h=True))

    assert all(torch.equal(a, b) for a, b in zip(run(), with_large_tiles(run)))


def gradient_operands(m, n, f, experts=0, seed=3):
    """dY's codes [m, n], the output projections' transposed codes [f, e n] and gu [m, 2f]."""
    g = torch.Generator().manual_seed(seed)
    e = max(1, experts)
    dyq, dys = fq.quant_act_1x128((torch.randn(m, n, generator=g) * 0.01).to(DEV))
    _, ws, wt = fq.quant_weight_128x128((torch.randn(e * n, f, generator=g) * f ** -0.5).to(DEV))
    gu = torch.randn(m, 2 * f, generator=g) * 2
    gu *= torch.where(torch.rand(m, 1, generator=g) < 0.05, 30.0, 1.0)
    return dyq, dys, wt, ws, gu.to(BF16).to(DEV)


def check_gradient(dyq, dys, w, gu, dgu, h):
    dh, mag = ref.product(ref.values(dyq, dys), w)
    f = dh.shape[1]
    g64 = ref.f64(gu)
    (dg, edg), (du, edu), (hh, eh) = ref.block_bwd(dh, ref.product_error(mag, dyq.shape[1] // 128, False), g64[:, :f],
                                                   g64[:, f:])
    ref.close(dgu[:, :f], dg, rounded(dg, edg), "dg")
    ref.close(dgu[:, f:], du, rounded(du, edu), "du")
    if h is not None:
        ref.close(h, hh, rounded(hh, eh), "h")


def weight_values(wt, ws, n, expert=0):
    """W_e^T [f, n] of the stacked transposed codes: scales [n / 128, f / 128] of the expert."""
    part = slice(expert * n, (expert + 1) * n)
    return ref.values(wt[:, part], ws[expert * n // 128:(expert + 1) * n // 128].t().contiguous(), 128)


@pytest.mark.parametrize("tile", ["auto", "256x128", "256x256"])
@pytest.mark.parametrize("m, n, f", [(1, 128, 128), (7, 384, 256), (64, 512, 128), (300, 640, 384), (257, 1024, 512),
                                     (1000, 256, 256)])
def test_gradient(m, n, f, tile):
    dyq, dys, wt, ws, gu = gradient_operands(m, n, f)
    fq.set_gemm_tile(tile)
    try:
        dgu, h = fq.gemm_dgrad_swiglu(dyq, dys, wt, ws, gu, with_h=True)
        check_gradient(dyq, dys, weight_values(wt, ws, n), gu, dgu, h)
        alone, none = fq.gemm_dgrad_swiglu(dyq, dys, wt, ws, gu)
        assert none is None and torch.equal(alone, dgu)
        fq.fp8q_gemm_dgrad_swiglu(dyq, dys, wt, ws, gu, gu)  # over its input
        assert torch.equal(gu, dgu)
    finally:
        fq.set_gemm_tile("auto")


@pytest.mark.parametrize("counts, n, f", [([5], 128, 128), ([70, 0, 1, 300, 128], 512, 256), ([0, 33, 0], 384, 384)],
                         ids=str)
def test_gradient_by_expert(counts, n, f):
    dyq, dys, wt, ws, gu = gradient_operands(sum(counts), n, f, len(counts))
    dgu, h = fq.grouped_gemm_dgrad_swiglu(dyq, dys, wt, ws, offsets_of(counts), gu, with_h=True)
    at = 0
    for e, c in enumerate(counts):
        if c:
            p = slice(at, at + c)
            check_gradient(dyq[p], dys[p], weight_values(wt, ws, n, e), gu[p], dgu[p], h[p])
        at += c


def test_gradient_against_differences():
    """block_bwd's formulas against central differences of the block in 64 bits."""
    r = np.random.default_rng(5)
    g, u, dh = r.standard_normal(400) * 4, r.standard_normal(400) * 2, r.standard_normal(400)
    f = lambda g, u: ref.block(g, u, 0.0, 0.0)[0] * dh  # noqa: E731
    (dg, _), (du, _), _ = ref.block_bwd(dh, 0.0, g, u)
    s = 1e-5
    # second-order differences: s^2 of a third derivative below 4, and 2^-52 / s
    assert np.abs((f(g + s, u) - f(g - s, u)) / (2 * s) - dg).max() <= 1e-8
    assert np.abs((f(g, u + s) - f(g, u - s)) / (2 * s) - du).max() <= 1e-8


def test_extreme_gates():
    """Gates where exp(-g) overflows or vanishes, and infinities' neighbours: finite and right."""
    m, n, f = 40, 128, 128
    dyq, dys, wt, ws, gu = gradient_operands(m, n, f)
    edge = torch.tensor([0.0, -0.0, 1e-30, -1e-30, 17.0, -17.0, 88.0, -88.0, 89.0, -89.0, 104.0, -104.0, 3e4, -3e4,
                         1e30, -1e30]).repeat(8).to(BF16).to(DEV)
    gu[:, :f] = edge
    gu[:, f:] = gu[:, f:].clamp(-4, 4)
    dgu, h = fq.gemm_dgrad_swiglu(dyq, dys, wt, ws, gu, with_h=True)
    check_gradient(dyq, dys, weight_values(wt, ws, n), gu, dgu, h)
    assert bool(torch.isfinite(dgu).all())
    # and forward, through a weight whose gates are that large
    for rows in (5, 3000):
        xq, xs, wq, ws2 = operands(rows, 128, 128, seed=9)
        ws2 = ws2.clone()
        ws2[0] *= 300.0
        h, gu2, q, s = fq.gemm_swiglu_quant(xq, xs, wq, ws2, with_output=True, with_gu=True)
        check_block(xq, xs, wq, ws2, h, gu2, q, s, exact=few(rows, 128, 128))


@pytest.mark.parametrize("m", [9, 64, 90, 2000])
def test_strided_outputs_and_rows_behind(m):
    """Outputs within wider rows, more rows behind them: nothing else is written."""
    f, k = 256, 384
    ops = operands(m, f, k)
    want = fq.gemm_swiglu_quant(*ops, with_output=True, with_gu=True)
    h = torch.full((m + 3, f + 8), 7.0, dtype=BF16, device=DEV)
    gu = torch.full((m + 3, 2 * f + 16), 7.0, dtype=BF16, device=DEV)
    q = torch.full((m + 3, f + 16), 99, dtype=U8, device=DEV)
    s = torch.full((m + 3, f // 128 + 1), 7.0, device=DEV)
    room = torch.empty(fq.gemm_swiglu_workspace(m, f, k, True), dtype=U8, device=DEV)
    fq.fp8q_gemm_swiglu(*ops, h[:m, :f], gu[:m, :2 * f], q[:m, :f], s[:m, :f // 128], room)
    for got, w, fill in ((h, want[0], 7), (gu, want[1], 7), (q, want[2], 99), (s, want[3], 7)):
        assert torch.equal(got[:m, :w.shape[1]], w)
        assert bool((got[m:] == fill).all()) and bool((got[:, w.shape[1]:] == fill).all())
    dyq, dys, wt, ws, gu = gradient_operands(m, 128, f)
    dgu, hh = fq.gemm_dgrad_swiglu(dyq, dys, wt, ws, gu, with_h=True)
    wide = torch.full((m + 3, 2 * f + 24), 7.0, dtype=BF16, device=DEV)
    wide[:m, :2 * f] = gu
    h2 = torch.full((m + 3, f + 8), 7.0, dtype=BF16, device=DEV)
    fq.fp8q_gemm_dgrad_swiglu(dyq, dys, wt, ws, wide[:m, :2 * f], wide[:m, :2 * f], h2[:m, :f])
    assert torch.equal(wide[:m, :2 * f], dgu) and torch.equal(h2[:m, :f], hh)
    assert bool((wide[m:] == 7).all()) and bool((wide[:, 2 * f:] == 7).all())
    assert bool((h2[m:] == 7).all()) and bool((h2[:, f:] == 7).all())


def test_no_rows():
    ops = operands(1, 128, 128)
    h, gu, q, s = fq.gemm_swiglu_quant(ops[0][:0], ops[1][:0], *ops[2:], with_output=True, with_gu=True)
    assert h.shape == (0, 128) and gu.shape == (0, 256) and q.shape == (0, 128) and s.shape == (0, 1)


@pytest.mark.parametrize("m", [8, 200, 3000])
def test_captured(m):
    """Replays with new inputs written between them, two graphs in turn."""
    f, k = 256, 640
    xq, xs, wq, ws = operands(m, f, k)
    dyq, dys, wt, wts, _ = gradient_operands(m, 384, f)

    def step():
        h, gu, q, s = fq.gemm_swiglu_quant(xq, xs, wq, ws, with_output=True, with_gu=True)
        return [h, gu, q, s, *fq.gemm_dgrad_swiglu(dyq, dys, wt, wts, gu, with_h=True)]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graphs, held = [], []
    for _ in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            held.append(step())
    for seed in (21, 22, 23):
        a = operands(m, f, k, seed=seed)
        xq.copy_(a[0])
        xs.copy_(a[1])
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        want = step()
        for i, w in enumerate(want):
            assert all(torch.equal(h[i], w) for h in held), (seed, i)
