"""64-bit references of the training block's operators (norm, gated block, AdamW)
in NumPy, and the comparisons their tests share.  U is half a step of FP32."""

import numpy as np
import torch

U = 2.0 ** -24
FLOOR = 2.0 ** -100
GRID = np.array([(8 + (c & 7)) * 2.0 ** ((c >> 3) - 10) if c >> 3 else (c & 7) * 2.0 ** -9 for c in range(127)])


def f64(t):
    return t.detach().cpu().double().numpy()


def half_step(dtype):
    return 2.0 ** -8 if dtype == torch.bfloat16 else 0.0


def tiny(dtype):
    """Half the least step of a type."""
    return 2.0 ** -134 if dtype == torch.bfloat16 else 2.0 ** -150


def values(q, s, rows=1):
    """Codes times their scales; a scale stands for 128 columns, and `rows` rows."""
    v = q.detach().cpu().view(torch.float8_e4m3fn).double().numpy()
    s = np.repeat(np.repeat(f64(s), rows, -2), 128, -1)
    return v * s[..., :v.shape[-2], :v.shape[-1]]


def close(got, want, bound, what):
    """got (tensor) within `bound` of want; where want is NaN or infinite, the same."""
    got = f64(got)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    odd = ~np.isfinite(want)
    assert np.array_equal(got[odd], want[odd], equal_nan=True), what
    err = np.abs(got - want)[~odd] - np.broadcast_to(bound, want.shape)[~odd]
    assert not err.size or (err <= 0).all(), (what, int((err > 0).sum()), float(err.max()))


def check_codes(q, s, want, bound, what):
    """Codes and scales of rows that are `want` to within `bound`: the scale is
    that of the group's largest, and each code is the nearest to its value over
    the scale that was stored, to within the errors of the value (bound / scale)
    and of the multiplication by the inverse scale (3 U)."""
    cols = want.shape[1]
    pad = ((0, 0), (0, -cols % 128))
    group = np.pad(np.abs(want), pad).reshape(len(want), -1, 128)
    slack = np.pad(np.broadcast_to(bound, want.shape), pad).reshape(group.shape).max(2)
    amax = group.max(2)
    sg = f64(s)
    assert (np.abs(sg * 448 - np.maximum(amax, FLOOR)) <= slack + 3 * U * amax + U * FLOOR).all(), (what, "scales")
    of = np.repeat(sg, 128, 1)[:, :cols]
    v = q.detach().cpu().view(torch.float8_e4m3fn).double().numpy()
    y = want / of
    off = bound / of + 4 * U * np.abs(y)
    # half the distance of the codes around the value, as far as it may lie
    e = np.maximum(np.floor(np.log2(np.maximum(np.abs(y) + off, 2.0 ** -9))), -6)
    err = np.abs(v - np.clip(y, -448, 448)) - (2.0 ** (e - 4) + off)
    assert not err.size or (err <= 0).all(), (what, "codes", int((err > 0).sum()), float(err.max()))


# ------------------------------------------------------------------------ norm
def norm(t, w, eps):
    """(y, rstd) of rows t in float64."""
    rstd = 1.0 / np.sqrt((t * t).mean(1) + eps)
    return t * rstd[:, None] * w, rstd


def norm_bwd(dy, x, w, rstd, dsum=None):
    """(dx, magnitude of dx's terms, dw, magnitude of dw's terms)."""
    h = x * rstd[:, None]
    a = dy * w
    n = x.shape[1]
    dx = rstd[:, None] * (a - h * (a * h).sum(1, keepdims=True) / n)
    mag = rstd[:, None] * (np.abs(a) + np.abs(h) * np.abs(a * h).sum(1, keepdims=True) / n)
    if dsum is not None:
        dx, mag = dx + dsum, mag + np.abs(dsum) / 16
    return dx, mag, (dy * h).sum(0), np.abs(dy * h).sum(0)


# ----------------------------------------------------------------- gated block
def sigmoid(g):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-g))


def product(x, w):
    """x W^T and the sum of its terms' magnitudes."""
    return x @ w.T, np.abs(x) @ np.abs(w).T


def product_error(mag, chunks, exact):
    """How far g and u may be off.  exact products: 128 terms of a chunk and the
    chunks, added in FP32, and two scalings.  FP8 products: 2^-10 of the terms
    beside that (each group of 8 is cut 13 bits below its largest)."""
    return (140 + chunks) * U * mag if exact else (2.0 ** -10 + (chunks + 17) * U) * mag


def block(g, u, eg, eu):
    """h and how far it may be off where g and u are off by eg and eu: |silu'| is
    at most 1.1, and the sigmoid and the products round 8 times."""
    s = g * sigmoid(g)
    h = s * u
    return h, 1.1 * eg * (np.abs(u) + eu) + np.abs(s) * eu + 8 * U * np.abs(h)


# Below 2^-126 FP32's steps are 2^-149 whatever the value: the exponential there
# is off by two of them, its sum with 1 does not change it and the division adds
# half of one.
LEAST = 2.5 * 2.0 ** -149


def block_bwd(dh, ed, g, u):
    """(dg, du, h) and their bounds where dh is off by ed: the sigmoid's 5
    roundings count where g multiplies it too; a sigmoid below 2^-126 is off by
    LEAST, times what multiplies it."""
    s = sigmoid(g)
    f, m = s * (1 + g * (1 - s)), s * (1 + np.abs(g))
    dg, du, h = dh * u * f, dh * g * s, g * s * u
    d = np.abs(dh) + ed
    return (dg, np.abs(u) * (ed * np.abs(f) + d * (16 * U * m + LEAST * (1 + 2 * np.abs(g))))), \
        (du, np.abs(g) * (s * (ed + 8 * U * d) + LEAST * d)), (h, 8 * U * np.abs(h) + LEAST * np.abs(g * u))


# ----------------------------------------------------------------------- AdamW
def mix(x):
    x = ((x ^ (x >> 16)) * 0x6C8E9CF5) & 0xFFFFFFFF
    x = ((x ^ (x >> 15)) * 0xB2D05E13) & 0xFFFFFFFF
    return x ^ (x >> 16)


def random_bits(n, seed, tensor):
    key = mix((mix((seed + 0x9E3779B1 * tensor) & 0xFFFFFFFF) + (seed >> 32)) & 0xFFFFFFFF)
    at = np.arange(n, dtype=np.uint64)
    return mix((at * np.uint64(0x85297A4D) + np.uint64(key)) & np.uint64(0xFFFFFFFF)).astype(np.int64)


def moments(m, v, scales=None):
    """The two moments in float64 from states or codes (flat)."""
    if scales is None:
        return f64(m).reshape(-1), f64(v).reshape(-1)
    held = lambda q, s: q.cpu().reshape(-1).view(torch.float8_e4m3fn).double().numpy() * \
        np.repeat(f64(s), 128)[:q.numel()]
    return held(m, scales[0]), held(v, scales[1]) ** 2


def adamw(p, g, m, v, step, lr, beta1, beta2, eps, decay, c=1.0):
    """{p, m, v} and {their bounds} after a step, all flat float64.  Bounds: g' has
    one rounding more where it is clipped; m and v 4 and 6 of their terms (the
    beta's and 1 - beta's own among them), the root half of v's and one more, the
    step 8 beside those, and p one of each of its terms."""
    g = g * c
    m2, v2 = beta1 * m + (1 - beta1) * g, beta2 * v + (1 - beta2) * g * g
    em = 5 * U * (np.abs(beta1 * m) + np.abs((1 - beta1) * g)) + 2.0 ** -148
    ev = 8 * U * v2 + 2.0 ** -147
    root, size = np.sqrt(v2 / (1 - beta2 ** step)), lr / (1 - beta1 ** step)
    move = size * m2 / (root + eps)
    p2 = p - lr * decay * p - move
    ep = 3 * U * np.abs(p) + 2 * U * np.abs(p2) + abs(size) * em / (root + eps) + 16 * U * np.abs(move)
    return {"p": p2, "m": m2, "v": v2}, {"p": ep, "m": em, "v": ev}


def check_state(q, s, want, bound, part, positive, what):
    """A state's codes and scales: each code is the one that the rounding with
    `part` in [0, 1) gives, or its neighbour where the value's error may move it
    over the border between them."""
    n = want.size
    group = np.pad(np.abs(want), (0, -n % 128)).reshape(-1, 128).max(1)
    slack = np.pad(bound, (0, -n % 128)).reshape(-1, 128).max(1)
    sg = f64(s)
    assert (np.abs(sg * 448 - np.maximum(group, FLOOR)) <= slack + 3 * U * group + U * FLOOR).all(), (what, "scales")
    of = np.repeat(sg, 128)[:n]
    y = want / of
    off = bound / of + 4 * U * np.abs(y)
    code = q.cpu().reshape(-1).view(torch.float8_e4m3fn).double().numpy()
    assert (np.sign(code) * np.sign(y) >= 0).all(), what
    ok = np.zeros(n, bool)
    for shift in (-1, 0, 1):
        a = np.abs(y) + shift * off
        at = np.clip(np.searchsorted(GRID, a, side="right") - 1, 0, 125)
        where = (a - GRID[at]) / (GRID[at + 1] - GRID[at])
        for border in (-2.0 ** -19, 0.0, 2.0 ** -19):  # t + part itself is rounded, below 17
            got = np.where(where + part + border >= 1, GRID[at + 1], GRID[at])
            if positive:
                got = np.where((np.abs(y) > 0) & (got == 0), GRID[1], got)
            ok |= np.abs(code) == got
    assert ok.all(), (what, int((~ok).sum()), np.nonzero(~ok)[0][:5])
