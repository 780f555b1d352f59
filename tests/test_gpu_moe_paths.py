"""The routing operators where their kernels take another path: more than 8
choices, rows in several slices, rows above the cache's size, sorts of several
tiles a block, NaN logits, many equal keys.  Bounds as in test_gpu_moe."""

import numpy as np
import pytest
import torch

import fp8_fine_grained_quant_amd as fq
import moe_ref as ref
import oracle
import test_gpu_moe as base
from gpu_util import DEV, assert_bytes_equal, assert_scales_equal, log

pytestmark = pytest.mark.gpu
BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32


@pytest.mark.parametrize("t,e,k", [(3, 40, 20), (4, 100, 17), (5, 128, 16), (6, 64, 9), (70, 256, 9), (9, 48, 16),
                                   (5, 128, 8), (131, 65, 8), (33, 512, 7), (2, 1024, 8), (1, 9, 9), (77, 1023, 12)])
@pytest.mark.parametrize("bf16", [True, False], ids=["bf16", "f32"])
def test_route_paths(t, e, k, bf16):
    base.test_route(t, e, k, bf16)
    base.test_route_gradient(t, e, k, bf16)


@pytest.mark.parametrize("e,k", [(64, 8), (256, 8), (256, 12), (700, 8), (1000, 20)])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_choice_with_many_close_keys(e, k, sigmoid):
    """Clusters of keys that FP32 cannot order, below and above the number that
    one wave decides at once, around the last choice too."""
    t = 37
    for n, width in enumerate((3, 12, 60, 70, e)):
        r = base.rng_of(e, k, n, sigmoid)
        x = np.float32(r.standard_normal((t, e)))
        p = ref.scores(x.astype(np.float64), sigmoid)
        bias = np.zeros(e, np.float32)
        take = r.permutation(e)[:min(width, e)]
        # token 0's keys of these experts within a few FP32 steps of 1.25, other
        # tokens' wherever that puts them
        bias[take] = np.float32(1.25 - p[0, take] + r.integers(-2, 3, take.size) * 2.0 ** -24)
        base.check_route(torch.from_numpy(x).to(DEV), k, sigmoid, bias, True, 1.0, f"cluster of {width}")
        x[:] = x[0]  # every token is such a token
        base.check_route(torch.from_numpy(x).to(DEV), k, sigmoid, bias, False, 1.0, f"clusters of {width}")


@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("k", [4, 12])
def test_nan_logits(k, sigmoid, biased):
    """A NaN is never chosen; a softmax that is not renormalized passes it on."""
    t, e = 40, 96
    r = base.rng_of(k, sigmoid, biased)
    x = np.float32(r.standard_normal((t, e)))
    x[::2, ::5] = np.nan
    x[3, :] = np.nan
    x[4, 2:] = np.nan
    bias = np.float32(r.standard_normal(e) * 0.05) if biased else None
    clean = np.where(np.isnan(x), -np.inf, x).astype(np.float64)
    for renorm in (True, False):
        ids, w = fq.moe_route(torch.from_numpy(x).to(DEV), k, score="sigmoid" if sigmoid else "softmax",
                              bias=None if bias is None else torch.from_numpy(bias).to(DEV), renormalize=renorm)
        ids_ref, w_ref = ref.route(clean, k, sigmoid, None if bias is None else bias.astype(np.float64), renorm)
        assert_bytes_equal(ids.cpu().numpy(), ids_ref, "ids")
        w = base.f64(w)
        if not sigmoid and not renorm:
            spoiled = np.isnan(x).any(1)[:, None] & (ids_ref >= 0)
            assert np.isnan(w[spoiled]).all()
            w, w_ref = np.where(spoiled, 0.0, w), np.where(spoiled, 0.0, w_ref)
        base.close(w, w_ref, 60 * ref.U32 * np.abs(w_ref), "weights")


@pytest.mark.parametrize("t,e,k", [(131072, 128, 8), (300_001, 1024, 5), (1_100_000, 3, 1)])
def test_sort_several_tiles_a_block(t, e, k):
    base.test_sort(t, e, k)


WIDE = [(3, 4, 2, 4100), (2, 8, 8, 7168), (5, 16, 3, 8191), (4, 12, 9, 4096), (3, 6, 4, 519), (6, 8, 5, 640)]


@pytest.mark.parametrize("bf16", [True, False], ids=["bf16", "f32"])
@pytest.mark.parametrize("drop", [0.0, 0.4])
@pytest.mark.parametrize("t,e,k,h", WIDE)
def test_wide_rows(t, e, k, h, drop, bf16):
    base.test_dispatch(t, e, k, h, drop, bf16)
    base.test_dispatch_gradient_and_combine(t, e, k, h, drop, bf16)
    base.test_combine_gradient(t, e, k, h, drop, bf16)


@pytest.mark.parametrize("bf16", [True, False], ids=["bf16", "f32"])
def test_rows_above_the_cache(bf16):
    """More rows than the cache in front of the memory holds are read past it;
    the results are those of two calls on halves, which are not."""
    t, k, h = (4300, 8, 4096) if bf16 else (4300, 4, 4096)
    half = t // 2
    g = torch.Generator(device=DEV).manual_seed(5)
    dt = BF16 if bf16 else F32
    yp = torch.randn(t * k, h, generator=g, device=DEV).to(dt)
    dy = torch.randn(t, h, generator=g, device=DEV).to(dt)
    w = torch.rand(t, k, generator=g, device=DEV)
    assert yp.numel() * yp.element_size() > 256 << 20
    perm = [torch.randperm(half * k, generator=g, device=DEV).to(I32) for _ in range(2)]
    dst = torch.cat([perm[0], perm[1] + half * k]).view(t, k)
    dst[7, 1] = -1 - dst[7, 1]
    parts = [(slice(0, half), slice(0, half * k), 0), (slice(half, t), slice(half * k, t * k), half * k)]

    def moved(d, by):
        return torch.where(d >= 0, d - by, d + by).to(I32).contiguous()

    y, dx = fq.moe_combine(yp, dst, w), fq.moe_dispatch_bwd(yp, dst)
    rows, q, s, dw = fq.moe_combine_bwd_quant(dy, yp, dst, w)
    for tok, row, by in parts:
        d, args = moved(dst[tok], by), (yp[row], w[tok].contiguous())
        assert torch.equal(fq.moe_combine(args[0], d, args[1]), y[tok])
        assert torch.equal(fq.moe_dispatch_bwd(args[0], d), dx[tok])
        rows_h, q_h, s_h, dw_h = fq.moe_combine_bwd_quant(dy[tok], args[0], d, args[1])
        assert torch.equal(rows_h, rows[row]) and torch.equal(q_h, q[row]) and torch.equal(s_h, s[row])
        assert torch.equal(dw_h, dw[tok])
    # a few tokens against 64 bits
    for i in (0, 7, half, t - 1):
        on = (dst[i] >= 0).cpu().numpy()
        r = base.f64(yp[dst[i].clamp(min=0).long()]) * on[:, None]
        terms = r * base.f64(w[i])[:, None]
        base.close(base.f64(y[i]), terms.sum(0), (k + 1) * ref.U32 * 1.01 * np.abs(terms).sum(0) +
                   ref.half_step(bf16) * np.abs(terms.sum(0)), f"token {i}")
        dots = r * base.f64(dy[i])[None]
        base.close(base.f64(dw[i]), dots.sum(1), (h / 64 + 32) * ref.U32 * np.abs(dots).sum(1), f"dw {i}")
    log(f"rows above the cache, bf16={bf16}")


def test_far_wide_rows():
    """Wide rows whose element offsets pass 2^32."""
    t, k, h = 33, 4, 640
    ld = (1 << 32) // (t * k) // 64 * 64 + 64
    r = base.rng_of(9)
    d = torch.from_numpy(base.make_map(t, 6, k, 0.2, r)).to(DEV)
    big = torch.empty(t * k * ld, dtype=BF16, device=DEV)
    rows = big.view(t * k, ld)[:, :h]
    x = base.make_rows(t, h, True, r)
    fq.fp8q_moe_dispatch(x.to(DEV), d, rows)
    want = ref.spread(x.float().numpy()[:, None], d.cpu().numpy())
    assert_scales_equal(rows.float().cpu().numpy(), want, "far rows")
    near = rows.contiguous()
    w = torch.from_numpy(np.float32(r.random((t, k)))).to(DEV)
    assert torch.equal(fq.moe_combine(rows, d, w), fq.moe_combine(near, d, w))
    out = torch.empty(t * k * ld, dtype=BF16, device=DEV).view(t * k, ld)[:, :h]
    dw, dw_near = torch.empty(t, k, device=DEV), torch.empty(t, k, device=DEV)
    q, s = torch.empty(t * k, h, dtype=torch.uint8, device=DEV), torch.empty(t * k, h // 128, device=DEV)
    fq.fp8q_moe_combine_bwd(x.to(DEV), rows, d, w, dw, out, q, s)
    rows_near, q_near, s_near, dw_near = fq.moe_combine_bwd_quant(x.to(DEV), near, d, w)
    assert torch.equal(out.contiguous(), rows_near) and torch.equal(q, q_near) and torch.equal(s, s_near)
    assert torch.equal(dw, dw_near)
    q_ref, s_ref = oracle.quant_act_1x128(rows_near.float().cpu().numpy())
    assert_bytes_equal(q.cpu().numpy(), q_ref, "codes")
    assert_scales_equal(s.cpu().numpy(), s_ref, "scales")
