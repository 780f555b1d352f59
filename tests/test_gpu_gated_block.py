"""Norm, gated block, gradients and AdamW together, as the example block runs
them: against the 64-bit formulas on the values that each step took, on a stream
of their own, and as a captured training step."""

import os
import sys

import numpy as np
import pytest
import torch

import block_ref as ref
import fp8_fine_grained_quant_amd as fq

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import gated_block  # noqa: E402

pytestmark = pytest.mark.gpu
BF16, F32, U = torch.bfloat16, torch.float32, ref.U
T, H, F = 256, 384, 256


def tensors(seed=4):
    g = torch.Generator().manual_seed(seed)
    x, residual, dy, dstream = (torch.randn(T, H, generator=g).to(BF16).to("cuda") for _ in range(4))
    return x, residual, dy * 0.01, dstream * 0.01


def rounded(v, bound):
    return bound + 2.0 ** -8 * (np.abs(v) + bound) + ref.tiny(BF16)


def quantized(v):
    """How far E4M3 codes of groups of 128 may be from v: half a step of the value
    or, below the least normal one, half the least step under the largest."""
    return 2.0 ** -4 * np.abs(v) + 2.0 ** -18 * np.abs(v).max(initial=0)


def times(a, ea, b, eb):
    """A bound of (a + ea)(b + eb) - a b, of matrices that an FP8 product takes."""
    return ea @ np.abs(b) + np.abs(a) @ eb + ea @ eb + 2.0 ** -9 * (np.abs(a) + ea) @ (np.abs(b) + eb)


def test_block_against_the_formulas():
    block = gated_block.GatedBlock(H, F)
    block.norm.add_(torch.linspace(-0.3, 0.3, H, device="cuda"))
    x, residual, dy, dstream = tensors()
    y, stream, kept = block.forward(x, residual)
    xn, _, rstd, gu, wq_t, ws, oq_t, os_ = kept
    f64 = ref.f64
    # the norm of the held stream
    assert torch.equal(stream, (x.float() + residual.float()).to(BF16))
    want, r = ref.norm(f64(stream), f64(block.norm), 1e-6)
    ref.close(rstd, r, 28 * U * r, "rstd")
    ref.close(xn, want, rounded(want, 30 * U * np.abs(want)), "xn")
    # gate and up: the products of the codes, of which the norm's are within a step
    w64 = ref.values(wq_t.t().contiguous(), ws, 128)
    g64 = want @ w64.T
    bound = times(want, quantized(want) + 31 * U * np.abs(want), w64.T, 0 * w64.T)
    ref.close(gu, g64, rounded(g64, bound), "gu")
    # the output projection of h's codes, h from gate and up as they were kept
    g, u = f64(gu)[:, :F], f64(gu)[:, F:]
    near = 2.0 ** -8 * np.abs(f64(gu))
    h, eh = ref.block(g, u, near[:, :F], near[:, F:])
    o64 = ref.values(oq_t.t().contiguous(), os_, 128)
    ref.close(y, h @ o64.T, rounded(h @ o64.T, times(h, eh + quantized(np.abs(h) + eh), o64.T, 0 * o64.T)), "y")
    # backward, from the codes of dy
    dx, (dnorm, dgate_up, dout) = block.backward(dy, dstream, kept)
    dyq, dys = fq.quant_act_1x128(dy)
    dh, mag = ref.product(ref.values(dyq, dys), o64.T)
    (dg, edg), (du, edu), (hh, ehh) = ref.block_bwd(dh, ref.product_error(mag, H // 128, False), g, u)
    d, ed = np.concatenate([dg, du], 1), rounded(np.concatenate([dg, du], 1), np.concatenate([edg, edu], 1))
    e_h = rounded(hh, ehh)
    dy64 = f64(dy)
    err = times(dy64.T, quantized(dy64.T), hh, e_h + quantized(np.abs(hh) + e_h))
    ref.close(dout, dy64.T @ hh, err, "output projection")
    eq = ed + quantized(np.abs(d) + ed)
    xn64 = f64(xn)
    ref.close(dgate_up, d.T @ xn64, times(d.T, eq.T, xn64, quantized(xn64)), "gate and up")
    dxn = d @ w64
    edxn = rounded(dxn, times(d, eq, w64, 0 * w64))
    # the norm's gradient is linear in its input: the formula of the bound's magnitudes
    want, mag, wdw, mdw = ref.norm_bwd(dxn, f64(stream), f64(block.norm), f64(rstd), f64(dstream))
    _, carried, _, mcarried = ref.norm_bwd(edxn, f64(stream), f64(block.norm), f64(rstd))
    ref.close(dx, want, rounded(want, 60 * U * (mag + carried) + carried), "dx")
    ref.close(dnorm, wdw, (T + 43) * U * (mdw + mcarried) + mcarried, "norm weight")


@pytest.mark.parametrize("bits", [8, 32])
def test_example_runs(bits):
    losses = gated_block.train(3, tokens=256, hidden=256, width=128, bits=bits, say=None)
    assert len(losses) == 3 and all(np.isfinite(losses))


def step_of(block, x, residual, dy, dstream, step=3):
    y, stream, kept = block.forward(x, residual)
    dx, grads = block.backward(dy, dstream, kept)
    norm = block.update(grads, step)
    return [y, stream, dx, norm, *grads, *block.params(), *block.states[0], *block.states[1], *sum(block.states[2], [])]


def test_on_another_stream():
    """Inputs that the stream's earlier work is still to write, outputs read by its next work."""
    want = step_of(gated_block.GatedBlock(H, F, seed=5), *tensors())
    block = gated_block.GatedBlock(H, F, seed=5)
    src, side = tensors(), torch.cuda.Stream()
    given = [torch.zeros_like(t) for t in src]
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        for a, b in zip(given, src):
            a.copy_(b)
        got = [t.clone() for t in step_of(block, *given)]
    side.synchronize()
    for i, (a, b) in enumerate(zip(got, want)):
        assert torch.equal(a, b), i


@pytest.mark.parametrize("given", ["object", "address"])
def test_streams_as_arguments(given):
    """Each call on a stream that is not the current one."""
    side = torch.cuda.Stream()
    s = side if given == "object" else side.cuda_stream
    x, residual, dy, dstream = tensors()
    block = gated_block.GatedBlock(H, F, seed=6)
    wq, ws, _ = fq.quant_weight_128x128(block.gate_up)
    _, os_, oq_t = fq.quant_weight_128x128(block.out)
    dyq, dys = fq.quant_act_1x128(dy)

    def path(stream):
        y, q, sc, total, rstd = fq.rms_norm_quant(x, block.norm, residual, with_output=True, stream=stream)
        h, gu, hq, hs = fq.gemm_swiglu_quant(q, sc, wq, ws, with_output=True, with_gu=True, stream=stream)
        dgu, h2 = fq.gemm_dgrad_swiglu(dyq, dys, oq_t, os_, gu, with_h=True, stream=stream)
        dx, dq, dsc, dw = fq.rms_norm_bwd_quant(y, total, block.norm, rstd, dstream, stream=stream)
        p, m, v = (torch.full((1000,), 0.5, device="cuda") for _ in range(3))
        torch.cuda.synchronize()
        fq.adamw([p], [dw.repeat(3)[:1000].contiguous()], [m], [v], 2, 1e-2, stream=stream)
        return [y, q, sc, total, rstd, h, gu, hq, hs, dgu, h2, dx, dq, dsc, dw, p, m, v]

    torch.cuda.synchronize()
    got = path(s)
    torch.cuda.synchronize()
    for i, (a, b) in enumerate(zip(got, path(None))):
        assert torch.equal(a, b), i


def test_captured_step():
    """Forward, backward and update in one graph, replayed with new inputs between:
    the same bits as the same steps launched one by one."""
    a, b = gated_block.GatedBlock(H, F, seed=7), gated_block.GatedBlock(H, F, seed=7)
    given = [t.clone() for t in tensors()]
    warm = gated_block.GatedBlock(H, F, seed=8)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step_of(warm, *given)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step_of(a, *given)
    for seed in (31, 32, 33):
        new = tensors(seed)
        for t, n in zip(given, new):
            t.copy_(n)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in held]
        want = step_of(b, *new)
        for i, (g, w) in enumerate(zip(got, want)):
            assert torch.equal(g, w), (seed, i)


def test_malformed_offsets_are_rejected_by_the_debug_library():
    lib = fq.load_debug_library()
    off = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    xq, xs = torch.zeros(300, 128, dtype=torch.uint8, device="cuda"), torch.ones(300, 1, device="cuda")
    wq, ws = torch.zeros(2, 256, 128, dtype=torch.uint8, device="cuda"), torch.ones(2, 2, 1, device="cuda")
    h = torch.full((300, 128), 7.0, dtype=BF16, device="cuda")
    gu = torch.zeros(300, 256, dtype=BF16, device="cuda")
    wt, wts = torch.zeros(128, 256, dtype=torch.uint8, device="cuda"), torch.ones(2, 1, device="cuda")
    p = lambda t: t.data_ptr()  # noqa: E731
    for o, status in ((off(0, 100, 300), 0), (off(0, 301, 300), 2), (off(1, 100, 300), 2), (off(0, 100, 299), 2)):
        h.fill_(7.0)
        assert lib.fp8q_grouped_gemm_swiglu(p(xq), p(xs), p(wq), p(ws), p(o), 2, 300, 128, 128, p(h), 128, None, 0, None,
                                            0, None, 0, 0) == status
        assert lib.fp8q_grouped_gemm_dgrad_swiglu(p(xq), p(xs), p(wt), p(wts), p(o), 2, 300, 128, 128, p(gu), 256, p(gu),
                                                  256, None, 0, 0) == status
        torch.cuda.synchronize()
        assert bool((h == (7.0 if status else 0.0)).all())
