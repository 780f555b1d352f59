"""Refusals of the MoE routing entry points and of gradient clipping: in the
library (fake addresses, never dereferenced: validation precedes any launch)
and in the binding (CPU tensors: shapes are checked before placement)."""

import ctypes

import pytest
import torch

import fp8_fine_grained_quant_amd as fq

OK, NULL, SHAPE, STRIDE, ALIGN, DTYPE = 0, 1, 2, 3, 4, 5
A = 1 << 20
BIG = (1 << 31) - 1
u8, f32, bf16, i32 = torch.uint8, torch.float32, torch.bfloat16, torch.int32


@pytest.fixture(scope="module", params=["product", "debug"])
def lib(request):
    return fq.load_library() if request.param == "product" else fq.load_debug_library()


def test_route(lib):
    def f(logits=A, lt=1, t=4, e=64, ld=64, k=8, score=0, bias=None, renorm=1, scale=1.0, ids=A, w=A):
        return lib.fp8q_moe_route(logits, lt, t, e, ld, k, score, bias, renorm, scale, ids, w, None)

    assert f(t=0, logits=None, ids=None, w=None) == OK
    assert f(lt=2) == DTYPE
    for bad in (dict(t=-1), dict(e=0), dict(e=1025, ld=1025), dict(k=0), dict(k=33), dict(e=4, k=5), dict(t=BIG),
                dict(score=2), dict(renorm=2), dict(scale=float("nan")), dict(scale=float("inf"))):
        assert f(**bad) == SHAPE, bad
    assert f(ld=63) == STRIDE
    assert f(logits=None) == NULL and f(ids=None) == NULL and f(w=None) == NULL
    assert f(logits=A + 2) == ALIGN and f(lt=0, logits=A + 1) == ALIGN and f(bias=A + 1) == ALIGN
    assert f(ids=A + 2) == ALIGN and f(w=A + 2) == ALIGN


def test_route_bwd(lib):
    def f(dw=A, logits=A, lt=1, t=4, e=64, ld=64, ids=A, k=8, score=0, renorm=1, scale=1.0, dl=A, ldd=64):
        return lib.fp8q_moe_route_bwd(dw, logits, lt, t, e, ld, ids, k, score, renorm, scale, dl, ldd, None)

    assert f(t=0, dw=None, logits=None, ids=None, dl=None) == OK
    assert f(lt=9) == DTYPE and f(e=2000, ld=2000, ldd=2000) == SHAPE and f(k=65) == SHAPE
    assert f(ld=60) == STRIDE and f(ldd=60) == STRIDE
    for name in ("dw", "logits", "ids", "dl"):
        assert f(**{name: None}) == NULL, name
        assert f(**{name: A + 1}) == ALIGN, name


def test_sort(lib):
    def f(ids=A, m=100, e=8, cover=0, off=A, dst=A, src=None, ws=None, n=0):
        return lib.fp8q_moe_sort(ids, m, e, cover, off, dst, src, ws, n, None)

    assert lib.fp8q_moe_sort_workspace(100, 8) == 0
    need = lib.fp8q_moe_sort_workspace(1 << 20, 256)
    assert need > 0
    assert lib.fp8q_moe_sort_workspace(-1, 8) == -1 and lib.fp8q_moe_sort_workspace(8, 0) == -1
    assert lib.fp8q_moe_sort_workspace(8, 1025) == -1 and lib.fp8q_moe_sort_workspace(BIG + 1, 8) == -1
    for bad in (dict(m=-1), dict(e=0), dict(e=1025), dict(cover=2), dict(m=BIG + 1)):
        assert f(**bad) == SHAPE, bad
    assert f(ids=None) == NULL and f(off=None) == NULL and f(dst=None) == NULL
    for name in ("ids", "off", "dst", "src"):
        assert f(**{name: A + 2}) == ALIGN, name
    assert f(m=1 << 20, e=256) == NULL
    assert f(m=1 << 20, e=256, ws=A, n=need - 1) == SHAPE
    assert f(m=1 << 20, e=256, ws=A + 1, n=need) == ALIGN


def test_rows(lib):
    def dis(x=A, xt=0, t=4, h=256, ld=256, dst=A, k=8, rows=A, ldr=256, q=A, ldq=256, s=A, lds=2):
        return lib.fp8q_moe_dispatch(x, xt, t, h, ld, dst, k, rows, ldr, q, ldq, s, lds, None)

    def dbw(drows=A, xt=0, t=4, h=256, ldr=256, dst=A, k=8, dx=A, ldx=256):
        return lib.fp8q_moe_dispatch_bwd(drows, xt, t, h, ldr, dst, k, dx, ldx, None)

    def com(yp=A, xt=0, t=4, h=256, ldr=256, dst=A, k=8, w=A, y=A, ldy=256):
        return lib.fp8q_moe_combine(yp, xt, t, h, ldr, dst, k, w, y, ldy, None)

    def cbw(dy=A, yp=A, xt=0, t=4, h=256, ldy=256, ldp=256, dst=A, k=8, w=A, rows=A, ldr=256, q=A, ldq=256, s=A, lds=2,
            dw=A):
        return lib.fp8q_moe_combine_bwd(dy, yp, xt, t, h, ldy, ldp, dst, k, w, rows, ldr, q, ldq, s, lds, dw, None)

    for f in (dis, dbw, com, cbw):
        assert f(t=0, dst=None) == OK
        assert f(xt=5) == DTYPE
        for bad in (dict(t=-1), dict(h=-1), dict(k=0), dict(k=33), dict(t=1 << 28), dict(t=1 << 20, h=1 << 20)):
            assert f(**bad) == SHAPE, bad
        assert f(dst=None) == NULL and f(dst=A + 2) == ALIGN
    for f, names in ((dis, ("x",)), (dbw, ("drows", "dx")), (com, ("yp", "y")), (cbw, ("dy", "yp"))):
        for name in names:
            assert f(**{name: None}) == NULL, name
            assert f(**{name: A + 1}) == ALIGN, name
    for f, names in ((dis, ("ld", "ldr", "ldq")), (dbw, ("ldr", "ldx")), (com, ("ldr", "ldy")),
                     (cbw, ("ldy", "ldp", "ldr", "ldq"))):
        for name in names:
            assert f(**{name: 255}) == STRIDE, name
    for f in (dis, cbw):
        assert f(rows=None, q=None, s=None) == NULL and f(s=None) == NULL
        assert f(lds=1) == STRIDE and f(s=A + 2) == ALIGN and f(rows=A + 1) == ALIGN
        assert f(rows=A + 2, xt=1) == ALIGN
    for f in (com, cbw):
        assert f(w=None) == NULL and f(w=A + 2) == ALIGN
    assert cbw(dw=None) == NULL and cbw(dw=A + 2) == ALIGN
    assert dis(h=0, x=None, dst=None) == OK


def test_clip(lib):
    class Grad(ctypes.Structure):
        _fields_ = [("g", ctypes.c_void_p), ("out", ctypes.c_void_p), ("len", ctypes.c_int64)]

    need = lib.fp8q_grad_clip_workspace(2)
    assert need > 0 and lib.fp8q_grad_clip_workspace(0) == 0 and lib.fp8q_grad_clip_workspace(-1) == -1
    assert lib.fp8q_grad_clip_workspace(1000) > need

    def f(g=A, out=A, n=100, ot=1, max_norm=1.0, ws=A, size=need, norm=A, count=2):
        arr = (Grad * 2)(Grad(A, A, 4), Grad(g, out, n))
        return lib.fp8q_grad_clip(ctypes.cast(arr, ctypes.c_void_p), count, ot, max_norm, ws, size, norm, None)

    assert f(ot=2) == DTYPE
    for bad in (dict(count=-1), dict(max_norm=-1.0), dict(max_norm=float("nan")), dict(n=-1), dict(n=1 << 62),
                dict(size=need - 1)):
        assert f(**bad) == SHAPE, bad
    assert f(g=None) == NULL and f(out=None) == NULL and f(ws=None) == NULL and f(norm=None) == NULL
    assert f(g=A + 2) == ALIGN and f(out=A + 2) == ALIGN and f(ot=0, out=A + 1) == ALIGN
    assert f(ws=A + 4) == ALIGN and f(norm=A + 1) == ALIGN
    assert lib.fp8q_grad_clip(None, 2, 1, 1.0, A, need, A, None) == NULL


# ------------------------------------------------------------------- binding
def z(*shape, dt=f32):
    return torch.zeros(shape, dtype=dt)


def refused(fn, what):
    with pytest.raises((ValueError, TypeError)) as ei:
        fn()
    assert what in str(ei.value), str(ei.value)


def placed(fn):
    with pytest.raises(ValueError, match="GPU tensors only"):
        fn()


def test_binding_route_and_sort():
    x, ids, w = z(6, 32), z(6, 4, dt=i32), z(6, 4)
    placed(lambda: fq.fp8q_moe_route(x, ids, w))
    placed(lambda: fq.fp8q_moe_route(x, ids, w, "sigmoid", z(32)))
    refused(lambda: fq.fp8q_moe_route(x, z(5, 4, dt=i32), w), "ids")
    refused(lambda: fq.fp8q_moe_route(x, z(6, 4, dt=torch.int64), w), "ids")
    refused(lambda: fq.fp8q_moe_route(x, ids, z(6, 3)), "weights")
    refused(lambda: fq.fp8q_moe_route(x, ids, w, bias=z(31)), "bias")
    refused(lambda: fq.fp8q_moe_route(x, ids, w, bias=z(32, dt=bf16)), "bias")
    placed(lambda: fq.fp8q_moe_route_bwd(w, x, ids, z(6, 32)))
    refused(lambda: fq.fp8q_moe_route_bwd(z(6, 5), x, ids, z(6, 32)), "dweights")
    refused(lambda: fq.fp8q_moe_route_bwd(w, x, ids, z(6, 31)), "dlogits")
    refused(lambda: fq.fp8q_moe_route_bwd(w, x, ids, z(6, 32, dt=bf16)), "dlogits")
    refused(lambda: fq._score("relu"), "relu")
    off, dst, src = z(33, dt=i32), z(6, 4, dt=i32), z(24, dt=i32)
    placed(lambda: fq.fp8q_moe_sort(ids, 32, off, dst, src))
    refused(lambda: fq.fp8q_moe_sort(ids, 31, off, dst, src), "offsets")
    refused(lambda: fq.fp8q_moe_sort(ids, 32, off, z(6, 3, dt=i32), src), "dst")
    refused(lambda: fq.fp8q_moe_sort(ids, 32, off, dst, z(23, dt=i32)), "src")
    refused(lambda: fq.fp8q_moe_sort(z(24, dt=i32), 32, off, dst, src), "ids")
    refused(lambda: fq.moe_sort_workspace(100, 2000), "2000")


def test_binding_rows():
    x, dst, rows, q, s, w = z(6, 200, dt=bf16), z(6, 4, dt=i32), z(24, 200, dt=bf16), z(24, 200, dt=u8), z(24, 2), z(6, 4)
    placed(lambda: fq.fp8q_moe_dispatch(x, dst, rows, q, s))
    refused(lambda: fq.fp8q_moe_dispatch(x, z(5, 4, dt=i32), rows), "dst")
    refused(lambda: fq.fp8q_moe_dispatch(x, dst, z(23, 200, dt=bf16)), "rows")
    refused(lambda: fq.fp8q_moe_dispatch(x, dst, z(24, 200)), "rows")
    refused(lambda: fq.fp8q_moe_dispatch(x, dst, rows, q[:, :199], s), "q")
    refused(lambda: fq.fp8q_moe_dispatch(x, dst, rows, q, z(24, 1)), "scale")
    refused(lambda: fq.fp8q_moe_dispatch(x, dst, rows, q), "scale")
    placed(lambda: fq.fp8q_moe_dispatch_bwd(rows, dst, x))
    refused(lambda: fq.fp8q_moe_dispatch_bwd(rows[:23], dst, x), "drows")
    refused(lambda: fq.fp8q_moe_dispatch_bwd(rows, dst, z(6, 200)), "dx")
    placed(lambda: fq.fp8q_moe_combine(rows, dst, w, x))
    refused(lambda: fq.fp8q_moe_combine(rows, dst, z(6, 5), x), "weights")
    refused(lambda: fq.fp8q_moe_combine(rows, dst, w, x[:5]), "y")
    dw = z(6, 4)
    placed(lambda: fq.fp8q_moe_combine_bwd(x, rows, dst, w, dw, rows, q, s))
    refused(lambda: fq.fp8q_moe_combine_bwd(x, rows[:, :199], dst, w, dw, rows, q, s), "yp")
    refused(lambda: fq.fp8q_moe_combine_bwd(x, rows, dst, w, z(6, 3), rows, q, s), "dweights")
    refused(lambda: fq.fp8q_moe_combine_bwd(x, rows, dst, w, dw, z(24, 200), q, s), "rows")


def test_binding_clip():
    g, ws, norm = [z(5), z(3, 4)], z(64, dt=u8), z()
    placed(lambda: fq.fp8q_grad_clip(g, g, 1.0, norm, ws))
    refused(lambda: fq.fp8q_grad_clip(g, g[:1], 1.0, norm, ws), "out")
    refused(lambda: fq.fp8q_grad_clip([z(5, dt=bf16)], [z(5)], 1.0, norm, ws), "bfloat16")
    refused(lambda: fq.fp8q_grad_clip(g, [z(5), z(12)], 1.0, norm, ws), "out")
    refused(lambda: fq.fp8q_grad_clip(g, [z(5), z(3, 4, dt=bf16)], 1.0, norm, ws), "bfloat16")
    refused(lambda: fq.fp8q_grad_clip([z(4, 3).t()], [z(3, 4)], 1.0, norm, ws), "contiguous")
