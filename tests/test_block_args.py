"""Refusals of the training block's entry points: in the library (fake addresses,
never dereferenced: validation precedes any launch) and in the binding (CPU
tensors, or tensors without memory: shapes are checked before any access)."""

import ctypes

import pytest
import torch

import fp8_fine_grained_quant_amd as fq
from fake_device import NO_MEMORY, current_device, hollow

OK, NULL, SHAPE, STRIDE, ALIGN, DTYPE = 0, 1, 2, 3, 4, 5
A = 1 << 20
BIG = (1 << 31) - 1
u8, f32, bf16, i32 = torch.uint8, torch.float32, torch.bfloat16, torch.int32


@pytest.fixture(scope="module", params=["product", "debug"])
def lib(request):
    return fq.load_library() if request.param == "product" else fq.load_debug_library()


def test_norm(lib):
    def f(x=A, t=0, rows=4, cols=256, ldx=256, res=A, ldr=256, w=A, eps=1e-6, y=A, ldy=256, q=A, ldq=256, s=A, lds=2,
          tot=A, ldt=256, rstd=A):
        return lib.fp8q_rms_norm(x, t, rows, cols, ldx, res, ldr, w, eps, y, ldy, q, ldq, s, lds, tot, ldt, rstd, None)

    assert f(rows=0, x=None, w=None, rstd=None) == OK and f(cols=0, x=None) == OK
    assert f(t=2) == DTYPE
    for bad in (dict(rows=-1), dict(cols=-1), dict(cols=16385, ldx=20000), dict(rows=BIG + 1), dict(eps=-1e-6),
                dict(eps=float("nan")), dict(eps=float("inf"))):
        assert f(**bad) == SHAPE, bad
    for name in ("ldx", "ldr", "ldy", "ldq", "lds", "ldt"):
        assert f(**{name: 1}) == STRIDE, name
    for name in ("x", "w", "tot", "rstd", "s"):
        assert f(**{name: None}) == NULL, name
    assert f(y=None, q=None, s=None) == NULL and f(q=None) == NULL
    for name in ("x", "res", "w", "y", "s", "tot", "rstd"):
        assert f(**{name: A + 1}) == ALIGN, name
    assert f(t=1, x=A + 2) == ALIGN


def test_norm_bwd(lib):
    need = lib.fp8q_rms_norm_bwd_workspace(4, 256)
    assert need >= 256 * 4
    assert lib.fp8q_rms_norm_bwd_workspace(0, 256) == 0 and lib.fp8q_rms_norm_bwd_workspace(4, 0) == 0
    for bad in ((-1, 4), (4, -1), (4, 16385), (BIG + 1, 4)):
        assert lib.fp8q_rms_norm_bwd_workspace(*bad) == -1

    def f(dy=A, x=A, t=0, rows=4, cols=256, ldy=256, ldx=256, w=A, rstd=A, dsum=A, lds=256, dx=A, lddx=256, q=A,
          ldq=256, s=A, ldsc=2, dw=A, ws=A, n=need):
        return lib.fp8q_rms_norm_bwd(dy, x, t, rows, cols, ldy, ldx, w, rstd, dsum, lds, dx, lddx, q, ldq, s, ldsc, dw,
                                     ws, n, None)

    assert f(cols=0, dy=None, dw=None) == OK
    assert f(t=2) == DTYPE and f(rows=-1) == SHAPE and f(cols=16385) == SHAPE and f(n=need - 1) == SHAPE
    for name in ("ldy", "ldx", "lds", "lddx", "ldq", "ldsc"):
        assert f(**{name: 1}) == STRIDE, name
    for name in ("dy", "x", "w", "rstd", "dw", "ws", "s"):
        assert f(**{name: None}) == NULL, name
    assert f(dx=None, q=None, s=None) == NULL and f(rows=0, dw=None) == NULL
    for name in ("dy", "x", "w", "rstd", "dsum", "dx", "s", "dw"):
        assert f(**{name: A + 1}) == ALIGN, name
    assert f(ws=A + 2) == ALIGN


@pytest.mark.parametrize("grouped", [False, True])
def test_swiglu(lib, grouped):
    def f(xq=A, xs=A, wq=A, ws=A, off=A, e=4, m=100, n=256, k=384, h=A, ldh=256, gu=A, ldg=512, q=A, ldq=256, s=A,
          lds=2, room=None, nroom=0):
        if grouped:
            return lib.fp8q_grouped_gemm_swiglu(xq, xs, wq, ws, off, e, m, n, k, h, ldh, gu, ldg, q, ldq, s, lds, None)
        return lib.fp8q_gemm_swiglu(xq, xs, wq, ws, m, n, k, h, ldh, gu, ldg, q, ldq, s, lds, room, nroom, None)

    assert f(m=0, xq=None) == OK and f(n=0, xq=None) == OK
    for bad in (dict(m=-1), dict(n=-128), dict(k=-128), dict(n=200), dict(k=100), dict(k=0), dict(k=131200),
                dict(n=1 << 30), dict(m=BIG + 1), dict(m=BIG, n=1 << 29)):
        assert f(**bad) == SHAPE, bad
    for name in ("xq", "xs", "wq", "ws", "s") + (("off",) if grouped else ()):
        assert f(**{name: None}) == NULL, name
    assert f(h=None, gu=None, q=None, s=None) == NULL and f(q=None) == NULL
    for name in ("ldh", "ldg", "ldq", "lds"):
        assert f(**{name: 1}) == STRIDE, name
    for name in ("xq", "wq", "h", "gu", "q"):
        assert f(**{name: A + 8}) == ALIGN, name
    for name in ("xs", "ws", "s") + (("off",) if grouped else ()):
        assert f(**{name: A + 2}) == ALIGN, name
    assert f(ldh=260) == ALIGN and f(ldg=516) == ALIGN and f(ldq=264) == ALIGN
    if grouped:
        assert f(e=0) == SHAPE and f(e=65537) == SHAPE
        return
    work = lib.fp8q_gemm_swiglu_workspace
    assert work(64, 256, 384, 1) == 64 * 256 * 4 and work(64, 256, 384, 0) == 0 and work(8192, 2048, 7168, 1) == 0
    assert work(-1, 256, 384, 1) == -1 and work(4, BIG, 384, 1) == -1 and work(4, 256, 100, 1) == -1
    assert f(m=64) == NULL and f(m=64, room=A + 4, nroom=1 << 20) == ALIGN and f(m=64, room=A, nroom=65535) == SHAPE


@pytest.mark.parametrize("grouped", [False, True])
def test_dgrad_swiglu(lib, grouped):
    def f(dyq=A, dys=A, wt=A, ws=A, off=A, e=4, m=100, n=384, k=256, gu=A, ldg=512, dgu=A, ldd=512, h=A, ldh=256):
        if grouped:
            return lib.fp8q_grouped_gemm_dgrad_swiglu(dyq, dys, wt, ws, off, e, m, n, k, gu, ldg, dgu, ldd, h, ldh, None)
        return lib.fp8q_gemm_dgrad_swiglu(dyq, dys, wt, ws, m, n, k, gu, ldg, dgu, ldd, h, ldh, None)

    assert f(m=0, dyq=None) == OK and f(k=0, dyq=None) == OK
    for bad in (dict(m=-1), dict(n=-128), dict(k=-128), dict(n=200), dict(k=100), dict(n=0), dict(n=131200),
                dict(k=1 << 30), dict(m=BIG + 1), dict(m=BIG, k=1 << 29)):
        assert f(**bad) == SHAPE, bad
    for name in ("dyq", "dys", "wt", "ws", "gu", "dgu") + (("off",) if grouped else ()):
        assert f(**{name: None}) == NULL, name
    for name in ("ldg", "ldd", "ldh"):
        assert f(**{name: 1}) == STRIDE, name
        assert f(**{name: 1028}) == ALIGN, name
    for name in ("dyq", "wt", "gu", "dgu", "h"):
        assert f(**{name: A + 8}) == ALIGN, name
    if grouped:
        assert f(e=0) == SHAPE and f(e=65536, n=128 * 128) == SHAPE


def adamw_call(lib, tensors, n=None, gt=1, bits=32, lr=1e-3, b1=0.9, b2=0.95, eps=1e-8, wd=0.1, step=1, seed=0,
               norm=None, most=float("inf")):
    class Tensor(ctypes.Structure):
        _fields_ = [(f, ctypes.c_void_p) for f in ("p", "g", "m", "v", "ms", "vs", "copy")] + [("len", ctypes.c_int64)]

    arr = (Tensor * max(1, len(tensors)))()
    for a, t in zip(arr, tensors):
        a.p, a.g, a.m, a.v, a.ms, a.vs, a.copy, a.len = t
    return lib.fp8q_adamw(ctypes.cast(arr, ctypes.c_void_p) if tensors else None, len(tensors) if n is None else n, gt,
                          bits, lr, b1, b2, eps, wd, step, seed, norm, most, None)


def test_adamw(lib):
    base = dict(p=A, g=A, m=A, v=A, ms=A, vs=A, copy=A, len=100)  # one tensor: its own parts are not compared
    one = lambda **k: [tuple({**base, **k}.values())]  # noqa: E731
    assert adamw_call(lib, []) == OK and adamw_call(lib, one(len=0, p=None)) == OK
    assert adamw_call(lib, [], n=3) == NULL and adamw_call(lib, [], n=-1) == SHAPE
    assert adamw_call(lib, one(), gt=2) == DTYPE
    nan, inf = float("nan"), float("inf")
    for bad in (dict(bits=16), dict(bits=0), dict(step=0), dict(step=-3), dict(b1=1.0), dict(b1=-0.1), dict(b2=1.0),
                dict(b2=nan), dict(eps=-1e-8), dict(eps=nan), dict(eps=inf), dict(lr=nan), dict(lr=inf), dict(wd=nan),
                dict(wd=inf), dict(lr=1e300), dict(eps=1e39), dict(most=-1.0), dict(most=nan)):
        assert adamw_call(lib, one(), **bad) == SHAPE, bad
    assert adamw_call(lib, one(len=-1)) == SHAPE and adamw_call(lib, one(len=1 << 45)) == SHAPE
    assert adamw_call(lib, one(len=(1 << 35) - 2047)) == SHAPE  # more than a launch's blocks hold
    for name in ("p", "g", "m", "v"):
        assert adamw_call(lib, one(**{name: None})) == NULL, name
    for name in ("ms", "vs"):
        assert adamw_call(lib, one(**{name: None}), bits=8) == NULL, name
        assert adamw_call(lib, one(**{name: A + 2}), bits=8) == ALIGN, name
    for name in ("p", "g", "m", "v"):
        assert adamw_call(lib, one(**{name: A + 2})) == ALIGN, name
    assert adamw_call(lib, one(g=A + 1), gt=0) == ALIGN and adamw_call(lib, one(copy=A + 1)) == ALIGN
    assert adamw_call(lib, one(), norm=A + 2) == ALIGN


@pytest.mark.parametrize("at", [[0, 0], [0, 396], [4000, 0, 3604], [800, 400, 0, 420], [0, 1200, 2400, 1100]])
def test_adamw_refuses_parameters_given_twice(lib, at):
    free = lambda i: A + (1 << 16) * (i + 1)  # noqa: E731
    for which, bits in ((0, 32), (2, 32), (3, 32), (0, 8), (6, 8)):
        t = [[free(i) + (k << 14) for k in range(7)] + [100] for i in range(len(at))]
        for i, a in enumerate(at):
            t[i][which] = A + (a if which != 6 else a // 2)
        assert adamw_call(lib, [tuple(x) for x in t], bits=bits) == SHAPE, (which, bits)
    for which in (2, 3):  # codes: 100 bytes a tensor
        t = [[free(i) + (k << 14) for k in range(7)] + [100] for i in range(len(at))]
        for i, a in enumerate(at):
            t[i][which] = A + a // 4
        assert adamw_call(lib, [tuple(x) for x in t], bits=8) == SHAPE, which


def z(*shape, dt=f32):
    return torch.zeros(shape, dtype=dt)


def refused(error, text, fn):
    with pytest.raises(error) as e:
        fn()
    assert text in str(e.value), str(e.value)


def test_binding_norm():
    refused(ValueError, "GPU tensors only", lambda: fq.rms_norm(z(3, 8), z(8)))
    refused(ValueError, "weight: shape (7), expected (8)", lambda: fq.rms_norm(z(3, 8), z(7)))
    refused(TypeError, "weight: dtype torch.bfloat16", lambda: fq.rms_norm(z(3, 8), z(8, dt=bf16)))
    refused(TypeError, "residual: dtype torch.float32", lambda: fq.rms_norm(z(3, 8, dt=bf16), z(8), z(3, 8)))
    refused(ValueError, "residual: shape", lambda: fq.rms_norm(z(3, 8), z(8), z(2, 8)))
    refused(ValueError, "expected 2-D", lambda: fq.rms_norm(z(8), z(8)))
    refused(ValueError, "x is required", lambda: fq.rms_norm(None, z(8)))
    refused(ValueError, "sum is required", lambda: fq.fp8q_rms_norm(z(3, 8), z(8), 1e-6, z(3, 8), None, None, z(3),
                                                                    residual=z(3, 8)))
    refused(ValueError, "rstd is required", lambda: fq.fp8q_rms_norm(z(3, 8), z(8), 1e-6, z(3, 8), None, None, None))
    refused(ValueError, "scale is required", lambda: fq.fp8q_rms_norm(z(3, 8), z(8), 1e-6, None, z(3, 8, dt=u8), None,
                                                                      z(3)))
    refused(ValueError, "x: shape", lambda: fq.rms_norm_bwd(z(3, 8), z(3, 7), z(8), z(3)))
    refused(ValueError, "rstd: shape", lambda: fq.rms_norm_bwd(z(3, 8), z(3, 8), z(8), z(2)))
    refused(ValueError, "dsum: shape", lambda: fq.rms_norm_bwd(z(3, 8), z(3, 8), z(8), z(3), z(3, 9)))
    refused(ValueError, "dweight is required",
            lambda: fq.fp8q_rms_norm_bwd(z(3, 8), z(3, 8), z(8), z(3), None, z(8, dt=u8)))
    refused(ValueError, "out of range", lambda: fq.rms_norm_bwd_workspace(3, 20000))


def test_binding_swiglu():
    x, xs, w, ws = z(5, 256, dt=u8), z(5, 2), z(256, 256, dt=u8), z(2, 2)
    refused(ValueError, "GPU tensors only", lambda: fq.gemm_swiglu(x, xs, w, ws))
    refused(ValueError, "wq: shape (256, 128)", lambda: fq.gemm_swiglu(x, xs, z(256, 128, dt=u8), ws))
    refused(ValueError, "as many of up as of gate", lambda: fq.gemm_swiglu(x, xs, z(255, 256, dt=u8), ws))
    refused(ValueError, "xs: shape", lambda: fq.gemm_swiglu(x, z(5, 1), w, ws))
    refused(ValueError, "ws: shape", lambda: fq.gemm_swiglu(x, xs, w, z(1, 2)))
    refused(TypeError, "xq: dtype", lambda: fq.gemm_swiglu(z(5, 256), xs, w, ws))
    refused(ValueError, "offsets is required", lambda: fq.grouped_gemm_swiglu(x, xs, w, ws, None))
    refused(ValueError, "expected [experts, 2 * width, K]",
            lambda: fq.grouped_gemm_swiglu(x, xs, w, ws, z(3, dt=i32)))
    refused(ValueError, "offsets: shape", lambda: fq.grouped_gemm_swiglu(x, xs, z(2, 256, 256, dt=u8), z(2, 2, 2),
                                                                         z(4, dt=i32)))
    refused(ValueError, "gu: shape", lambda: fq.fp8q_gemm_swiglu(x, xs, w, ws, None, z(5, 128, dt=bf16)))
    refused(ValueError, "scale is required", lambda: fq.fp8q_gemm_swiglu(x, xs, w, ws, None, q=z(5, 128, dt=u8)))
    wt, wts, gu = z(128, 256, dt=u8), z(2, 1), z(5, 256, dt=bf16)
    refused(ValueError, "GPU tensors only", lambda: fq.gemm_dgrad_swiglu(x, xs, wt, wts, gu))
    refused(ValueError, "gu: shape", lambda: fq.gemm_dgrad_swiglu(x, xs, wt, wts, z(5, 128, dt=bf16)))
    refused(TypeError, "gu: dtype", lambda: fq.gemm_dgrad_swiglu(x, xs, wt, wts, z(5, 256)))
    refused(ValueError, "ws: shape", lambda: fq.gemm_dgrad_swiglu(x, xs, wt, z(1, 2), gu))
    refused(ValueError, "dgu is required", lambda: fq.fp8q_gemm_dgrad_swiglu(x, xs, wt, wts, gu, None))
    refused(ValueError, "wq_t: shape", lambda: fq.grouped_gemm_dgrad_swiglu(x, xs, wt, wts, z(3, dt=i32), gu))
    refused(ValueError, "offsets: shape", lambda: fq.grouped_gemm_dgrad_swiglu(x, xs, wt, wts, z(1, dt=i32), gu))


def test_binding_adamw():
    one = lambda n=5, dt=f32: [z(n, dt=dt)]  # noqa: E731
    go = lambda *a, **k: fq.adamw(*a, step=1, lr=1e-3, **k)  # noqa: E731
    refused(ValueError, "GPU tensors only", lambda: go(one(), one(), one(), one()))
    refused(ValueError, "grads: 2 tensors for 1 parameters", lambda: go(one(), one() * 2, one(), one()))
    refused(ValueError, "exp_avg: shape (4), expected (5)", lambda: go(one(), one(), one(4), one()))
    refused(TypeError, "params: dtype torch.bfloat16", lambda: go(one(dt=bf16), one(), one(), one()))
    refused(TypeError, "exp_avg: dtype torch.uint8, expected torch.float32", lambda: go(one(), one(), one(dt=u8), one()))
    refused(TypeError, "exp_avg: dtype torch.float32, expected torch.uint8",
            lambda: go(one(), one(), one(), one(), scales=([z(1)], [z(1)])))
    refused(ValueError, "exp_avg scales: shape (2), expected (1)",
            lambda: go(one(), one(), one(dt=u8), one(dt=u8), scales=([z(2)], [z(1)])))
    refused(ValueError, "scales of one state", lambda: go(one(), one(), one(), one(), scales=([z(1)], None)))
    refused(TypeError, "unsupported dtype torch.float16",
            lambda: go(*[[hollow(5, dt=d)] for d in (f32, torch.float16, f32, f32)]))
    refused(ValueError, "must be contiguous", lambda: go([z(4, 6).t()], [z(6, 4)], [z(6, 4)], [z(6, 4)]))
    refused(TypeError, "copies: dtype", lambda: go(one(), one(), one(), one(), copies=one()))
    refused(TypeError, "sequence", lambda: go(5, one(), one(), one()))
    refused(ValueError, "norm: shape", lambda: go(one(), one(), one(), one(), norm=z(2)))
    with pytest.raises((OverflowError, TypeError)):
        go(one(), one(), one(), one(), seed=-1)
    with pytest.raises(ValueError):
        fq.adamw_states([z(3)], bits=16)
    m, v, s = fq.adamw_states([z(300), z(2, 3)], bits=8)
    assert [t.shape for t in m] == [(300,), (2, 3)] and m[0].dtype == u8 and v[1].dtype == u8
    assert [len(t) for t in s[0]] == [3, 1] and fq.adamw_states([z(3)])[2] is None


def calls(device="cuda:0", other="cuda:0"):
    """Every call of the block with tensors that have no memory."""
    t = lambda *s, dt=f32: hollow(*s, dt=dt, device=device)  # noqa: E731
    o = lambda *s, dt=f32: hollow(*s, dt=dt, device=other)  # noqa: E731
    codes = dict(xq=t(5, 256, dt=u8), xs=t(5, 2), wq=t(256, 256, dt=u8), ws=o(2, 2))
    by_expert = dict(codes, wq=t(2, 256, 256, dt=u8), ws=o(2, 2, 2), offsets=t(3, dt=i32))
    grad = dict(dyq=t(5, 256, dt=u8), dys=t(5, 2), wq_t=t(128, 256, dt=u8), ws=o(2, 1), gu=t(5, 256, dt=bf16))
    grouped = dict(grad, wq_t=t(128, 512, dt=u8), ws=o(4, 1), offsets=t(3, dt=i32))
    h, gu = t(5, 128, dt=bf16), t(5, 256, dt=bf16)
    return [lambda: fq.fp8q_rms_norm(t(3, 8), o(8), 1e-6, t(3, 8), None, None, t(3)),
            lambda: fq.fp8q_rms_norm_bwd(t(3, 8), t(3, 8), t(8), t(3), t(8), o(4096, dt=u8), t(3, 8)),
            lambda: fq.fp8q_gemm_swiglu(**codes, h=h),
            lambda: fq.fp8q_grouped_gemm_swiglu(**by_expert, h=h),
            lambda: fq.fp8q_gemm_dgrad_swiglu(**grad, dgu=gu),
            lambda: fq.fp8q_grouped_gemm_dgrad_swiglu(**grouped, dgu=gu),
            lambda: fq.adamw([t(9)], [t(9)], [o(9)], [t(9)], 1, 1e-3),
            lambda: fq.adamw([], [], [], [], 1, 1e-3, norm=o()) if other != device else
            fq.adamw([t(9)], [t(9)], [t(9)], [t(9)], 1, 1e-3, norm=t())]


def test_devices():
    """Checked before any access: tensors of one device, which is the current one."""
    with current_device(0):
        for i, call in enumerate(calls()):
            with pytest.raises(RuntimeError, match=NO_MEMORY):
                call()
            assert i >= 0
        for call in calls(other="cuda:1"):
            with pytest.raises(ValueError, match="device"):
                call()
    with current_device(1):
        for call in calls():
            with pytest.raises(ValueError, match="current device is cuda:1"):
                call()
