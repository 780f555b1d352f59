"""The MoE routing operators against 64-bit references.

Bounds: an FP32 sum of n terms is off by at most n 2^-24 of the sum of their
magnitudes; exp of a rounded difference d by (|d| + 2) 2^-24 relative; a result
stored in a type by half its step.  Ids, maps, codes and scales are exact."""

import itertools

import numpy as np
import pytest
import torch

import fp8_fine_grained_quant_amd as fq
import moe_ref as ref
import oracle
from gpu_util import DEV, assert_bytes_equal, assert_scales_equal, log

pytestmark = pytest.mark.gpu
BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32


def rng_of(*seed):
    return np.random.Generator(np.random.PCG64(list(seed)))


def to_type(a, bf16):
    t = torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32))
    return t.to(BF16) if bf16 else t


def f64(t):
    return t.detach().cpu().double().numpy()


def strided(t, pad, shift=0):
    """The same values in rows `pad` elements further apart, starting `shift`
    elements into the allocation; returns the view and the whole buffer."""
    rows, cols = t.shape
    buf = torch.full((shift + rows * (cols + pad) + 64,), 7.0, dtype=t.dtype).to(DEV)
    view = buf[shift:shift + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    view.copy_(t.to(DEV))
    return view, buf


def close(got, want, bound, what):
    got = np.asarray(got, np.float64)
    err = np.abs(got - want)
    bad = ~(err <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.size} outside, first at {np.argwhere(bad)[0].tolist()}: " \
                          f"got {got[bad][0]} want {want[bad][0]} bound {np.broadcast_to(bound, bad.shape)[bad][0]}"


# ------------------------------------------------------------------- router
def make_logits(t, e, kind, r):
    x = r.standard_normal((t, e)) * 1.5
    if kind == "masked":
        x[r.random((t, e)) < 0.3] = -np.inf
        x[::3] = -np.inf                                  # no expert at all
        x[1::5, : max(1, e - 1)] = -np.inf                # one expert left
    elif kind == "lowest":                                # masked with the type's lowest value, not -inf
        x[r.random((t, e)) < 0.5] = -3.3895e38
        x[0] = -3.3895e38
    elif kind == "ties":
        x = np.round(x)
    elif kind == "equal":
        x[:] = 0.25
    elif kind == "wide":
        x *= 60.0                                         # sigmoids that saturate, softmaxes that vanish
    return x


SHAPES = [(1, 1, 1), (1, 32, 2), (3, 8, 8), (5, 33, 4), (37, 64, 8), (9, 65, 6), (130, 160, 6), (64, 256, 8),
          (11, 257, 5), (33, 384, 8), (3, 511, 9), (7, 1000, 16), (2, 1024, 32)]


def check_route(xt, k, sigmoid, bias, renorm, scale, what):
    b = None if bias is None else torch.from_numpy(bias.astype(np.float32)).to(DEV)
    score = "sigmoid" if sigmoid else "softmax"
    ids, w = fq.moe_route(xt, k, score=score, bias=b, renormalize=renorm, scale=scale)
    torch.cuda.synchronize()
    x = f64(xt)
    ids_ref, w_ref = ref.route(x, k, sigmoid, None if b is None else f64(b), renorm, scale)
    assert_bytes_equal(ids.cpu().numpy(), ids_ref, what + " ids")
    # span of the logits the exponentials see: top - x for softmax, exact for sigmoid
    xj = np.take_along_axis(x, np.maximum(ids_ref, 0), 1)
    top = np.where(np.isfinite(x), x, -np.inf).max(1, keepdims=True)
    with np.errstate(invalid="ignore"):
        span = 0.0 if sigmoid else np.nan_to_num(np.minimum(top - xj, 110.0), nan=0.0)
    close(w.cpu().numpy(), w_ref, (span + x.shape[1] / 64 + 40) * ref.U32 * np.abs(w_ref) + 2.0 ** -140, what)
    return ids


@pytest.mark.parametrize("t,e,k", SHAPES)
@pytest.mark.parametrize("bf16", [True, False], ids=["bf16", "f32"])
def test_route(t, e, k, bf16):
    for n, (kind, sigmoid, biased, renorm) in enumerate(itertools.product(
            ["plain", "masked", "lowest", "ties", "equal", "wide"], [False, True], [False, True], [False, True])):
        r = rng_of(t, e, k, n)
        x = to_type(make_logits(t, e, kind, r), bf16)
        bias = r.standard_normal(e) * (0.05 if kind != "equal" else 0.0) if biased else None
        what = f"{kind} sigmoid={sigmoid} bias={biased} renorm={renorm}"
        check_route(x.to(DEV), k, sigmoid, bias, renorm, 2.5 if n % 3 == 0 else 1.0, what)
    log(f"route {t}x{e} k={k}")


def test_route_border_below_fp32():
    """Experts whose score + bias differ by less than FP32 resolves."""
    t, e, k = 70, 96, 6
    r = rng_of(77)
    for sigmoid in (True, False):
        x = np.float32(r.standard_normal((t, e)))
        p = ref.scores(x.astype(np.float64), sigmoid)
        bias = np.float32(r.standard_normal(e) * 0.05)
        # FP32 biases that bring the experts of row 0 within a few 2^-26 of each other
        bias[:40] = np.float32(1.5 - p[0, :40])
        key = p[0] + bias.astype(np.float64)
        assert np.unique(np.float32(key[:40])).size < 40 <= np.unique(key[:40]).size
        check_route(torch.from_numpy(x).to(DEV), k, sigmoid, bias, True, 1.0, f"border sigmoid={sigmoid}")
    for k in (1, 3, 8, 32):
        x = np.zeros((5, 200), np.float32)
        x[:, 100:] = 1.0
        check_route(torch.from_numpy(x).to(DEV), k, True, np.zeros(200), True, 1.0, f"ties k={k}")


@pytest.mark.parametrize("bf16", [True, False], ids=["bf16", "f32"])
def test_route_strided_and_bounds(bf16):
    """Odd row strides and starts; outputs next to the results stay."""
    t, e, k = 21, 129, 5
    x = to_type(make_logits(t, e, "masked", rng_of(5)), bf16)
    for pad, shift in ((0, 1), (1, 0), (3, 5), (7, 3)):
        view, _ = strided(x, pad, shift)
        check_route(view, k, False, None, True, 1.0, f"stride {pad} {shift}")
        buf = torch.full((t * k + 32,), 99, dtype=I32, device=DEV)
        w = torch.full((t * k + 32,), 99.0, device=DEV)
        fq.fp8q_moe_route(view, buf[16:16 + t * k].view(t, k), w[16:16 + t * k].view(t, k))
        assert bool((buf[:16] == 99).all() and (buf[-16:] == 99).all())
        assert bool((w[:16] == 99).all() and (w[-16:] == 99).all())
        ids, wt = fq.moe_route(view, k)
        dl_view, dl_buf = strided(torch.zeros(t, e).to(x.dtype), pad, shift)
        dl_buf.fill_(7.0)
        fq.fp8q_moe_route_bwd(wt, view, ids, dl_view)
        want = fq.moe_route_bwd(wt, x.to(DEV), ids)
        assert torch.equal(dl_view, want)
        assert int((dl_buf != 7.0).sum()) <= int((want != 7.0).sum())
        assert bool((dl_buf[:shift] == 7.0).all() and (dl_buf[-64:] == 7.0).all())


@pytest.mark.parametrize("t,e,k", SHAPES)
@pytest.mark.parametrize("bf16", [True, False], ids=["bf16", "f32"])
def test_route_gradient(t, e, k, bf16):
    for n, (kind, sigmoid, renorm) in enumerate(itertools.product(["plain", "masked", "ties", "wide"], [False, True],
                                                                  [False, True])):
        r = rng_of(t, e, k, n, 9)
        x = to_type(make_logits(t, e, kind, r), bf16)
        ids = ref.route(f64(x), k, sigmoid, r.standard_normal(e) * 0.05, renorm)[0]
        dw = np.float32(r.standard_normal((t, k)))
        dl = fq.moe_route_bwd(torch.from_numpy(dw).to(DEV), x.to(DEV), torch.from_numpy(ids).to(DEV),
                              score="sigmoid" if sigmoid else "softmax", renormalize=renorm, scale=2.5)
        torch.cuda.synchronize()
        d, mag = ref.route_bwd(dw.astype(np.float64), f64(x), ids, sigmoid, renorm, 2.5)
        xf = np.where(np.isfinite(f64(x)), f64(x), 0.0)
        span = 0.0 if sigmoid else np.minimum(xf.max() - xf.min(), 110.0)
        bound = (2 * span + e / 32 + 80) * ref.U32 * mag + ref.half_step(bf16) * np.abs(d) + 2.0 ** -130
        close(f64(dl), d, bound, f"{kind} sigmoid={sigmoid} renorm={renorm}")
    log(f"route gradient {t}x{e} k={k}")


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_gradient_against_differences(sigmoid, renorm):
    t, e, k = 6, 40, 5
    r = rng_of(31)
    x = np.float32(r.standard_normal((t, e)))
    ids = ref.route(x.astype(np.float64), k, sigmoid)[0]
    ids[2, 3] = -1
    dw = np.float32(r.standard_normal((t, k)))
    dl = f64(fq.moe_route_bwd(torch.from_numpy(dw).to(DEV), torch.from_numpy(x).to(DEV),
                              torch.from_numpy(ids).to(DEV), score="sigmoid" if sigmoid else "softmax",
                              renormalize=renorm))
    h = 1e-5
    for ex in range(e):
        xp, xm = x.astype(np.float64), x.astype(np.float64)
        xp[:, ex] += h
        xm[:, ex] -= h
        num = ((ref.weights_of(xp, ids, sigmoid, renorm, 1.0) - ref.weights_of(xm, ids, sigmoid, renorm, 1.0)) * dw
               ).sum(1) / (2 * h)
        # third derivative below 10, h^2 / 6 of it; 64-bit cancellation 1e-16 / h
        close(dl[:, ex], num, 1e-9 + 100 * ref.U32 * np.abs(dw).sum(1), f"expert {ex}")


# --------------------------------------------------------------------- sort
@pytest.mark.parametrize("t,e,k", [(1, 1, 1), (1, 32, 8), (16, 256, 8), (63, 5, 3), (65, 4, 1), (511, 96, 2),
                                   (512, 300, 8), (513, 1024, 8), (1365, 7, 3), (2731, 1000, 3), (8192, 1, 2),
                                   (32768, 256, 8), (16384, 384, 7)])
def test_sort(t, e, k):
    r = rng_of(t, e, k)
    for kind in ("even", "dropped", "one", "none", "outside"):
        ids = r.integers(0, e, (t, k))
        if kind == "dropped":
            ids[r.random((t, k)) < 0.3] = -1
        elif kind == "one":
            ids[:] = e // 2
        elif kind == "none":
            ids[:] = -1
        elif kind == "outside":
            ids[r.random((t, k)) < 0.2] = e
            ids[r.random((t, k)) < 0.2] = 2 ** 31 - 1
            ids[r.random((t, k)) < 0.2] = -2 ** 31
        ids = ids.astype(np.int32)
        for cover in (False, True):
            got = fq.moe_sort(torch.from_numpy(ids).to(DEV), e, cover=cover)
            for g, w, what in zip(got, ref.sort(ids, e, cover), ("offsets", "dst", "src")):
                assert_bytes_equal(g.cpu().numpy(), w, f"{kind} {what}")
    log(f"sort {t} x {k} over {e}")


def test_sort_empty_and_without_src():
    off, dst, src = fq.moe_sort(torch.empty((0, 4), dtype=I32, device=DEV), 6)
    assert off.cpu().tolist() == [0] * 7 and dst.shape == (0, 4) and src.shape == (0,)
    ids = rng_of(3).integers(-1, 9, (700, 8)).astype(np.int32)
    off = torch.empty(10, dtype=I32, device=DEV)
    buf = torch.full((700 * 8 + 64,), 99, dtype=I32, device=DEV)
    ws = torch.empty(fq.moe_sort_workspace(5600, 9), dtype=torch.uint8, device=DEV)
    fq.fp8q_moe_sort(torch.from_numpy(ids).to(DEV), 9, off, buf[32:-32].view(700, 8), workspace=ws)
    want = ref.sort(ids, 9)
    assert_bytes_equal(off.cpu().numpy(), want[0], "offsets")
    assert_bytes_equal(buf[32:-32].cpu().numpy(), want[1].reshape(-1), "dst")
    assert bool((buf[:32] == 99).all() and (buf[-32:] == 99).all())


# ------------------------------------------------------- rows to and from order
ROWS = [(1, 4, 1, 128), (1, 32, 8, 1), (3, 8, 2, 7), (8, 32, 8, 512), (5, 6, 3, 129), (17, 16, 4, 1000),
        (33, 64, 8, 2047), (70, 9, 6, 384), (4, 40, 32, 260), (9, 12, 9, 2176)]


def make_map(t, e, k, drop, r):
    ids = np.stack([r.permutation(e)[:k] for _ in range(t)]).astype(np.int32)
    if drop:
        ids[r.random((t, k)) < drop] = -1
    return ref.sort(ids, e)[1]


def make_rows(m, h, bf16, r, poison=None):
    x = r.standard_normal((m, h))
    x *= np.where(r.random(h) < 0.05, 20.0, 1.0) * np.where(r.random((m, 1)) < 0.1, 100.0, 1.0)
    if m > 2:
        x[1] = 0.0
    if poison is not None:
        x[poison] = np.array([np.nan, np.inf])[np.arange(h) % 2]
    return to_type(x, bf16)


@pytest.mark.parametrize("bf16", [True, False], ids=["bf16", "f32"])
@pytest.mark.parametrize("drop", [0.0, 0.3, 1.0])
@pytest.mark.parametrize("t,e,k,h", ROWS)
def test_dispatch(t, e, k, h, drop, bf16):
    r = rng_of(t, e, k, h)
    x = make_rows(t, h, bf16, r)
    dst = make_map(t, e, k, drop, r)
    d = torch.from_numpy(dst).to(DEV)
    want = ref.spread(x.float().numpy()[:, None], dst)
    q_ref, s_ref = oracle.quant_act_1x128(want)
    for pad, shift in ((0, 0), (3, 1)):
        xv, _ = strided(x, pad, shift)
        rows = fq.moe_dispatch(xv, d)
        assert rows.dtype == x.dtype
        assert_scales_equal(rows.float().cpu().numpy(), want, "rows")
        for both in (True, False):
            rows, q, s = fq.moe_dispatch_quant(xv, d, with_output=both)
            assert (rows is not None) == both
            if both:
                assert_scales_equal(rows.float().cpu().numpy(), want, "rows")
            assert_bytes_equal(q.cpu().numpy(), q_ref, "codes")
            assert_scales_equal(s.cpu().numpy(), s_ref, "scales")
    # dense odd code rows and strided outputs: nothing beside them is written
    rows_v, rows_b = strided(torch.zeros_like(to_type(want, bf16)), 5, 3)
    rows_b.fill_(7.0)
    q = torch.full((t * k, h + 9), 77, dtype=torch.uint8, device=DEV)
    s = torch.full((t * k, (h + 127) // 128 + 2), 7.0, device=DEV)
    fq.fp8q_moe_dispatch(x.to(DEV), d, rows_v, q[:, 1:1 + h], s[:, :-2])
    assert_scales_equal(rows_v.float().cpu().numpy(), want, "strided rows")
    assert_bytes_equal(q[:, 1:1 + h].cpu().numpy(), q_ref, "strided codes")
    assert_scales_equal(s[:, :-2].cpu().numpy(), s_ref, "strided scales")
    assert bool((q[:, 0] == 77).all() and (q[:, 1 + h:] == 77).all() and (s[:, -2:] == 7).all())
    pads = rows_b[3:3 + t * k * (h + 5)].view(t * k, h + 5)[:, h:]
    assert bool((pads == 7).all() and (rows_b[:3] == 7).all() and (rows_b[-64:] == 7).all())


@pytest.mark.parametrize("bf16", [True, False], ids=["bf16", "f32"])
@pytest.mark.parametrize("drop", [0.0, 0.3, 1.0])
@pytest.mark.parametrize("t,e,k,h", ROWS)
def test_dispatch_gradient_and_combine(t, e, k, h, drop, bf16):
    """Dropped pairs' rows hold NaN and infinity: they must not be used."""
    r = rng_of(t, e, k, h, 1)
    dst = make_map(t, e, k, drop, r)
    d = torch.from_numpy(dst).to(DEV)
    yp = make_rows(t * k, h, bf16, r, poison=-1 - dst[dst < 0])
    w = np.float32(r.random((t, k)) + 0.1)
    rows = ref.fetch(np.where(np.isfinite(yp.float().numpy()), yp.float().numpy(), 0.0), dst)
    for pad, shift in ((0, 0), (3, 1)):
        v, _ = strided(yp, pad, shift)
        y = f64(fq.moe_combine(v, d, torch.from_numpy(w).to(DEV)))
        terms = rows * w.astype(np.float64)[:, :, None]
        tot, mag = terms.sum(1), np.abs(terms).sum(1)
        close(y, tot, (k + 1) * ref.U32 * mag * 1.01 + ref.half_step(bf16) * np.abs(tot), "combine")
        dx = f64(fq.moe_dispatch_bwd(v, d))
        tot, mag = rows.sum(1), np.abs(rows).sum(1)
        close(dx, tot, (k + 1) * ref.U32 * mag * 1.01 + ref.half_step(bf16) * np.abs(tot), "dispatch gradient")
    out, buf = strided(torch.zeros(t, h).to(yp.dtype), 5, 3)
    buf.fill_(7.0)
    fq.fp8q_moe_combine(yp.to(DEV), d, torch.from_numpy(w).to(DEV), out)
    assert torch.equal(out, fq.moe_combine(yp.to(DEV), d, torch.from_numpy(w).to(DEV)))
    pads = buf[3:3 + t * (h + 5)].view(t, h + 5)[:, h:]
    assert bool((pads == 7).all() and (buf[:3] == 7).all() and (buf[-64:] == 7).all())


@pytest.mark.parametrize("bf16", [True, False], ids=["bf16", "f32"])
@pytest.mark.parametrize("drop", [0.0, 0.3, 1.0])
@pytest.mark.parametrize("t,e,k,h", ROWS)
def test_combine_gradient(t, e, k, h, drop, bf16):
    r = rng_of(t, e, k, h, 2)
    dst = make_map(t, e, k, drop, r)
    d = torch.from_numpy(dst).to(DEV)
    dy = make_rows(t, h, bf16, r)
    yp = make_rows(t * k, h, bf16, r, poison=-1 - dst[dst < 0])
    w = np.float32(r.random((t, k)) + 0.1)
    wg = torch.from_numpy(w).to(DEV)
    g64 = f64(dy)
    prod = ref.spread(g64[:, None] * w.astype(np.float64)[:, :, None], dst)
    terms = g64[:, None] * ref.fetch(np.where(np.isfinite(yp.float().numpy()), yp.float().numpy(), 0.0), dst)
    dw_ref, dw_mag = terms.sum(2), np.abs(terms).sum(2)
    for pad, shift in ((0, 0), (3, 1)):
        dyv, ypv = strided(dy, pad, shift)[0], strided(yp, pad + 1, shift)[0]
        rows, dw = fq.moe_combine_bwd(dyv, ypv, d, wg)
        close(f64(rows), prod, (ref.half_step(bf16) + ref.U32) * 1.01 * np.abs(prod) + 2.0 ** -130, "rows")
        close(f64(dw), dw_ref, (h / 64 + 32) * ref.U32 * dw_mag, "dw")
        for both in (True, False):
            rows_q, q, s, dw_q = fq.moe_combine_bwd_quant(dyv, ypv, d, wg, with_output=both)
            if both:
                assert torch.equal(rows_q.cpu(), rows.cpu())
            q_ref, s_ref = oracle.quant_act_1x128(rows.float().cpu().numpy())
            assert_bytes_equal(q.cpu().numpy(), q_ref, "codes")
            assert_scales_equal(s.cpu().numpy(), s_ref, "scales")
            assert torch.equal(dw_q, dw)
    # the weights' gradient against differences of the 64-bit combination (linear in w)
    step = 2.0 ** -10
    for j in range(min(k, 2)):
        up, dn = w.astype(np.float64).copy(), w.astype(np.float64).copy()
        up[:, j] += step
        dn[:, j] -= step
        fin = ref.fetch(np.where(np.isfinite(yp.float().numpy()), yp.float().numpy(), 0.0), dst)
        loss = lambda u: (g64 * (fin * u[:, :, None]).sum(1)).sum(1)
        num = (loss(up) - loss(dn)) / (2 * step)
        mag = dw_mag[:, j] * (h / 64 + 32) * ref.U32 + 1e-12 * (np.abs(terms) * w[:, :, None]).sum((1, 2)) / step
        close(f64(dw)[:, j], num, mag + 1e-300, f"differences {j}")


def test_zero_sizes():
    e = lambda *s, dt=BF16: torch.empty(*s, dtype=dt, device=DEV)
    assert fq.moe_route(e(0, 16), 4)[0].shape == (0, 4)
    assert fq.moe_route_bwd(e(0, 4, dt=F32), e(0, 16), e(0, 4, dt=I32)).shape == (0, 16)
    assert fq.moe_dispatch(e(0, 64), e(0, 4, dt=I32)).shape == (0, 64)
    assert fq.moe_combine(e(0, 64), e(0, 4, dt=I32), e(0, 4, dt=F32)).shape == (0, 64)
    rows, dw = fq.moe_combine_bwd(e(3, 0), e(6, 0), torch.arange(6, dtype=I32, device=DEV).view(3, 2),
                                  torch.ones(3, 2, device=DEV))
    assert rows.shape == (6, 0) and bool((dw == 0).all())  # a product over no columns


def test_far_rows():
    """Rows whose element offsets pass 2^31 (an 8 GiB tensor of rows, few of
    which are touched)."""
    t, k, h = 130, 2, 64
    ld = (1 << 32) // (t * k) // 64 * 64 + 64
    r = rng_of(8)
    dst = make_map(t, 4, k, 0.0, r)
    d = torch.from_numpy(dst).to(DEV)
    big = torch.empty(t * k * ld, dtype=BF16, device=DEV)
    rows = big.view(t * k, ld)[:, :h]
    assert (t * k - 1) * ld * 2 > 1 << 32
    x = make_rows(t, h, True, r)
    fq.fp8q_moe_dispatch(x.to(DEV), d, rows)
    assert_scales_equal(rows.float().cpu().numpy(), ref.spread(x.float().numpy()[:, None], dst), "far rows")
    w = torch.from_numpy(np.float32(r.random((t, k)))).to(DEV)
    assert torch.equal(fq.moe_combine(rows, d, w), fq.moe_combine(rows.contiguous(), d, w))


# --------------------------------------------------- streams, graphs, debug build
def _layer(x, logits, o):
    """The whole path on preallocated outputs, as a captured step has it."""
    fq.fp8q_moe_route(logits, o["ids"], o["w"], "sigmoid", o["bias"])
    fq.fp8q_moe_sort(o["ids"], 24, o["off"], o["dst"], o["src"], o["ws"], cover=True)
    fq.fp8q_moe_dispatch(x, o["dst"], o["rows"], o["q"], o["s"])
    fq.fp8q_moe_combine(o["rows"], o["dst"], o["w"], o["y"])
    fq.fp8q_moe_combine_bwd(x, o["rows"], o["dst"], o["w"], o["dw"], o["drows"], o["dq"], o["ds"])
    fq.fp8q_moe_dispatch_bwd(o["drows"], o["dst"], o["dx"])
    fq.fp8q_moe_route_bwd(o["dw"], logits, o["ids"], o["dl"], "sigmoid")
    fq.fp8q_grad_clip([o["dw"]], [o["dwc"]], 1.0, o["norm"], o["cws"])


def _layer_out(t, k, h, seed):
    e = lambda *s, dt=BF16: torch.zeros(s, dtype=dt, device=DEV)
    m, g, u8 = t * k, (h + 127) // 128, torch.uint8
    bias = torch.from_numpy(np.float32(rng_of(seed).standard_normal(24) * 0.05)).to(DEV)
    return dict(ids=e(t, k, dt=I32), w=e(t, k, dt=F32), off=e(25, dt=I32), dst=e(t, k, dt=I32), src=e(m, dt=I32),
                ws=e(fq.moe_sort_workspace(m, 24), dt=u8), rows=e(m, h), q=e(m, h, dt=u8), s=e(m, g, dt=F32), y=e(t, h),
                dw=e(t, k, dt=F32), drows=e(m, h), dq=e(m, h, dt=u8), ds=e(m, g, dt=F32), dx=e(t, h),
                dl=e(t, 24, dt=F32), dwc=e(t, k, dt=F32), norm=e(dt=F32), cws=e(fq.grad_clip_workspace(1), dt=u8),
                bias=bias)


def _layer_in(t, h, seed):
    r = rng_of(seed)
    return make_rows(t, h, True, r).to(DEV), torch.from_numpy(
        np.float32(make_logits(t, 24, "masked" if seed % 2 else "plain", r))).to(DEV)


def test_graph_replays_match_eager():
    t, k, h = 1200, 4, 320
    x, logits = _layer_in(t, h, 1)
    g_out, e_out = _layer_out(t, k, h, 5), _layer_out(t, k, h, 5)
    _layer(x, logits, g_out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _layer(x, logits, g_out)
    for seed in (11, 12, 13):
        xn, ln = _layer_in(t, h, seed)
        x.copy_(xn)
        logits.copy_(ln)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        _layer(xn, ln, e_out)
        torch.cuda.synchronize()
        for name in g_out:
            if name not in ("ws", "cws"):
                a, b = g_out[name], e_out[name]
                assert torch.equal(a, b), (seed, name)


def test_other_streams():
    """Every call on a side stream, with its temporaries allocated there."""
    t, k, h = 2000, 6, 256
    r = rng_of(4)
    side = torch.cuda.Stream()
    logits = torch.from_numpy(np.float32(r.standard_normal((t, 40)))).to(DEV)
    x = make_rows(t, h, True, r).to(DEV)
    torch.cuda.synchronize()

    def path(stream):
        ids, w = fq.moe_route(logits, k, stream=stream)
        off, dst, src = fq.moe_sort(ids, 40, stream=stream)
        rows, q, s = fq.moe_dispatch_quant(x, dst, stream=stream)
        y = fq.moe_combine(rows, dst, w, stream=stream)
        dr, dw = fq.moe_combine_bwd(y, rows, dst, w, stream=stream)
        dl = fq.moe_route_bwd(dw, logits, ids, stream=stream)
        dx = fq.moe_dispatch_bwd(dr, dst, stream=stream)
        norm = fq.grad_clip([dl], 1.0, stream=stream)
        return [ids, w, off, dst, src, rows, q, s, y, dr, dw, dl, dx, norm]

    want = path(None)
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream):
        got = path(stream)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_debug_build_rejects_bad_maps():
    """No launch is made for a map that is no permutation of the rows."""
    lib = fq.load_debug_library()
    x = torch.ones(4, 128, dtype=BF16, device=DEV)
    rows = torch.full((8, 128), 5.0, dtype=BF16, device=DEV)
    good = torch.tensor([[0, 1], [2, -4], [4, 5], [6, 7]], dtype=I32, device=DEV)
    for bad in ([[0, 1], [2, 3], [4, 5], [6, 8]], [[0, 0], [2, 3], [4, 5], [6, 7]], [[0, -2], [2, 3], [4, 5], [1, 7]],
                [[0, 1], [2, 3], [4, 5], [6, -2 ** 31]]):
        d = torch.tensor(bad, dtype=I32, device=DEV)
        f = lambda m: lib.fp8q_moe_dispatch(x.data_ptr(), 0, 4, 128, 128, m.data_ptr(), 2, rows.data_ptr(), 128, None,
                                            0, None, 0, None)
        assert f(d) == 2 and bool((rows == 5).all())
    assert f(good) == 0
    torch.cuda.synchronize()
    assert bool((rows[3] == 0).all()) and bool((rows[:3] == 1).all())
