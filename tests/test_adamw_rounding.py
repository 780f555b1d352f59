"""The random rounding of AdamW's 8-bit states over many steps, and its bits for
elements past 2^32.

The root of the second moment decays without a gradient by sqrt(beta2) a step,
whatever its rounding was, so its mean over many elements after STEPS steps is
beta2^(STEPS / 2) if each rounding keeps the mean.  The first element of every
group is held at the group's largest value by its gradient, so that the scales stay
and the others move through the codes: to the nearest code they would not move at
all, and rounded down they would lose a code every step."""

import numpy as np
import pytest
import torch

import block_ref as ref
import fp8_fine_grained_quant_amd as fq

DEV = "cuda:0"
BF16, F32, U8 = torch.bfloat16, torch.float32, torch.uint8
BETA2, STEPS, GROUPS, SCALE = 0.999, 200, 512, 1e-3

# A value just below its code (sqrt(beta2) of it, 5.01e-4 down) is rounded with the
# variance (to the code below) x (to the code above) <= 1/8 x 5.01e-4 of its square,
# STEPS times: 0.1125 relative for an element, by the root of their number for the
# mean, of which five are allowed.  16 random bits round 2^-16 of a code too low,
# which is 1/8 of the value, and the arithmetic is off by 6 U a step.
TOLERANCE = 5 * np.sqrt(STEPS * 5.01e-4 / 8 * 1.013) / np.sqrt(GROUPS * 127) + STEPS * (2.0 ** -16 / 8 + 6 * ref.U)


def first_codes():
    """Codes of magnitude 1 to 256, the largest, 448, first in every group."""
    c = np.random.default_rng(4).integers(0x38, 0x79, (GROUPS, 128))
    c[:, 0] = 0x7E
    return c


def mean_ratio(before, after):
    return (after[:, 1:] / before[:, 1:]).mean()


def off(ratio):
    return abs(ratio - BETA2 ** (STEPS / 2))


def emulate(rounding):
    rng = np.random.default_rng(7)
    held = ref.GRID[first_codes()] * SCALE
    before, top = held.copy(), held[:, 0].copy()
    for _ in range(STEPS):
        held = held * np.sqrt(BETA2)
        held[:, 0] = top
        y = held / SCALE
        lo = np.clip(np.searchsorted(ref.GRID, y, side="right") - 1, 0, 125)
        t = (y - ref.GRID[lo]) / (ref.GRID[lo + 1] - ref.GRID[lo])
        part = {"random": np.floor(rng.random(y.shape) * 65536) / 65536, "nearest": 0.5, "down": 0.0}[rounding]
        held = ref.GRID[lo + (t + part >= 1)] * SCALE
    return mean_ratio(before, held)


def test_bound_tells_the_roundings_apart():
    assert off(emulate("random")) <= TOLERANCE
    assert off(emulate("nearest")) > 10 * TOLERANCE and off(emulate("down")) > 10 * TOLERANCE


@pytest.mark.gpu
def test_root_keeps_its_mean():
    codes = torch.from_numpy(first_codes().astype(np.uint8)).to(DEV)
    p, g = torch.zeros(codes.shape, device=DEV), torch.zeros(codes.shape, device=DEV)
    g[:, 0] = 448 * SCALE
    m, v = torch.zeros_like(codes), codes.clone()
    scales = ([torch.zeros(GROUPS, device=DEV)], [torch.full((GROUPS,), SCALE, device=DEV)])
    root = lambda: np.sqrt(ref.moments(m, v, (scales[0][0], scales[1][0]))[1]).reshape(GROUPS, 128)  # noqa: E731
    before = root()
    for t in range(1, STEPS + 1):
        fq.adamw([p], [g], [m], [v], t, 1e-3, betas=(0.9, BETA2), scales=scales, seed=1000 + t)
    assert off(mean_ratio(before, root())) <= TOLERANCE


# ------------------------------------------------------------ past 2^32 elements
FAR = 1 << 32


def bits_at(first, n, seed, tensor):
    """The documented random bits of elements first .. first + n of a tensor."""
    key = int(ref.mix((ref.mix((seed + 0x9E3779B1 * tensor) & 0xFFFFFFFF) + (seed >> 32)) & 0xFFFFFFFF))
    return np.array([ref.mix(((i & 0xFFFFFFFF) * 0x85297A4D + (i >> 32) * 0x27D4EB2F + key) & 0xFFFFFFFF)
                     for i in range(first, first + n)], np.int64)


def test_bits():
    """Those of test_gpu_adamw.py's first elements, and others 2^32 elements later."""
    assert np.array_equal(bits_at(0, 300, 77 << 31, 3), ref.random_bits(300, 77 << 31, 3))
    assert not (bits_at(FAR, 300, 5, 0) == bits_at(0, 300, 5, 0)).any()


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [8, 32])
def test_past_32_bits(bits):
    """A tensor of more than 2^32 elements: its ends against 64 bits, zeros between."""
    n, seed, step = FAR + 4096 + 77, (3 << 33) + 5, 5
    hyper = dict(lr=3e-3, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1)
    state = U8 if bits == 8 else F32
    zeros = lambda dtype, k=n: torch.zeros(k, dtype=dtype, device=DEV)  # noqa: E731
    p, g, m, v, copy = zeros(F32), zeros(BF16), zeros(state), zeros(state), zeros(BF16)
    s = [zeros(F32, -(-n // 128)) for _ in range(2)] if bits == 8 else None
    ends = [(0, 5000), (FAR - 4096, n)]
    gen = torch.Generator().manual_seed(12)
    rand = lambda k, std: (torch.randn(k, generator=gen) * std).to(DEV)  # noqa: E731
    for a, b in ends:
        k = b - a
        p[a:b], g[a:b] = rand(k, 0.02), rand(k, 1e-3).to(BF16)
        for to, x, sc in ((m, rand(k, 3e-4), 0), (v, rand(k, 1e-3).abs(), 1)):
            if bits == 8:
                q, qs = fq.quant_act_1x128(torch.nn.functional.pad(x, (0, -k % 16)).view(1, -1))
                to[a:b] = q.view(-1)[:k]
                s[sc][a // 128:-(-b // 128)] = qs.view(-1)
            else:
                to[a:b] = x if sc == 0 else x.square()
    part = lambda t, a, b: t[a:b].clone()  # noqa: E731
    held = lambda a, b: None if s is None else tuple(x[a // 128:-(-b // 128)] for x in s)  # noqa: E731
    before = [(ref.f64(p[a:b]), ref.f64(g[a:b]), *ref.moments(part(m, a, b), part(v, a, b), held(a, b)))
              for a, b in ends]
    fq.adamw([p], [g], [m], [v], step, scales=None if s is None else ([s[0]], [s[1]]), seed=seed, copies=[copy], **hyper)
    for (a, b), old in zip(ends, before):
        want, bound = ref.adamw(*old, step, hyper["lr"], *hyper["betas"], hyper["eps"], hyper["weight_decay"])
        ref.close(p[a:b], want["p"], bound["p"], (a, "p"))
        assert torch.equal(copy[a:b], p[a:b].to(BF16))
        if bits == 32:
            ref.close(m[a:b], want["m"], bound["m"], (a, "m"))
            ref.close(v[a:b], want["v"], bound["v"], (a, "v"))
            continue
        r = bits_at(a, b - a, seed, 0)
        root = np.sqrt(want["v"])
        eroot = np.sqrt(want["v"] + bound["v"]) - root + 2 * ref.U * root
        sm, sv = held(a, b)
        ref.check_state(part(m, a, b), sm, want["m"], bound["m"], (r & 0xFFFF) / 65536, False, (a, "m"))
        ref.check_state(part(v, a, b), sv, root, eroot, (r >> 16) / 65536, True, (a, "v"))
    for t in (p, m, v, copy):
        for a in range(5000, FAR - 4096, 1 << 28):
            assert not bool(t[a:min(a + (1 << 28), FAR - 4096)].any())
