"""AdamW over many tensors against 64 bits, states in 32 and in 8 bits.  Bounds:
block_ref.adamw; a state's code is the one that the random rounding gives for
some value within the state's bound."""

import numpy as np
import pytest
import torch

import block_ref as ref
import fp8_fine_grained_quant_amd as fq
from gpu_util import DEV, log

pytestmark = pytest.mark.gpu
BF16, F32, U8 = torch.bfloat16, torch.float32, torch.uint8
HYPER = dict(lr=3e-3, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1)


def place(n, dtype, shift, fill=7):
    """n elements `shift` into their memory, and that memory."""
    room = torch.full((n + shift + 16,), fill, dtype=dtype, device=DEV)
    return room[shift:shift + n], room


class Case:
    def __init__(self, sizes, bits=32, grads=F32, copies=True, shift=0, seed=1, scale=1e-3):
        g = torch.Generator().manual_seed(seed)
        self.sizes, self.bits, self.rooms = sizes, bits, []
        rand = lambda n, std: torch.randn(n, generator=g) * std  # noqa: E731
        self.p = self.put([rand(n, 0.02) for n in sizes], F32, shift)
        self.g = self.put([rand(n, scale) for n in sizes], grads, shift)
        m, v = [rand(n, scale / 3) for n in sizes], [rand(n, scale).square() for n in sizes]
        self.scales = None
        if bits == 8:
            held = []
            self.scales = ([], [])
            for k, xs in enumerate((m, [x.sqrt() for x in v])):
                codes = []
                for x in xs:
                    q, s = fq.quant_act_1x128(torch.nn.functional.pad(x, (0, -len(x) % 16)).view(1, -1).to(DEV)) \
                        if len(x) else (torch.empty(1, 0, dtype=U8), torch.empty(1, 0))
                    codes.append(q.view(-1)[:len(x)].cpu())
                    self.scales[k].append(s.reshape(-1).to(DEV).clone())
                held.append(self.put(codes, U8, shift, 99))
            self.m, self.v = held
        else:
            self.m, self.v = self.put(m, F32, shift), self.put(v, F32, shift)
        self.copies = self.put([torch.zeros(n) for n in sizes], BF16, shift) if copies else None

    def put(self, xs, dtype, shift, fill=7):
        out = []
        for x in xs:
            t, room = place(len(x), dtype, shift, fill)
            t.copy_(x.to(dtype))
            out.append(t)
            self.rooms.append((room, shift, len(x), fill))
        return out

    def run(self, step=5, seed=77, norm=None, max_norm=float("inf"), **more):
        """One step on the GPU, checked against the step in 64 bits."""
        h = {**HYPER, **more}
        before = [(ref.f64(p), ref.f64(g), *ref.moments(m, v, s)) for p, g, m, v, s in
                  zip(self.p, self.g, self.m, self.v,
                      zip(*self.scales) if self.scales else [None] * len(self.p))]
        grads = [g.clone() for g in self.g]
        fq.adamw(self.p, self.g, self.m, self.v, step, scales=self.scales, seed=seed, norm=norm, max_norm=max_norm,
                 copies=self.copies, **h)
        torch.cuda.synchronize()
        c = 1.0 if norm is None or float(norm) <= max_norm else max_norm / float(norm)
        for i, (p, g, m, v) in enumerate(before):
            want, bound = ref.adamw(p, g, m, v, step, h["lr"], *h["betas"], h["eps"], h["weight_decay"], c)
            ref.close(self.p[i], want["p"], bound["p"], (i, "p"))
            if self.copies:
                assert torch.equal(self.copies[i], self.p[i].to(BF16)), i
            if self.scales is None:
                ref.close(self.m[i], want["m"], bound["m"], (i, "m"))
                ref.close(self.v[i], want["v"], bound["v"], (i, "v"))
            else:
                r = ref.random_bits(len(p), seed, i)
                root = np.sqrt(want["v"])
                eroot = np.sqrt(want["v"] + bound["v"]) - root + 2 * ref.U * root
                ref.check_state(self.m[i], self.scales[0][i], want["m"], bound["m"], (r & 0xFFFF) / 65536, False,
                                (i, "m"))
                ref.check_state(self.v[i], self.scales[1][i], root, eroot, (r >> 16) / 65536, True, (i, "v"))
        assert all(torch.equal(a, b) for a, b in zip(grads, self.g))
        for room, shift, n, fill in self.rooms:
            assert bool((room[:shift] == fill).all() and (room[shift + n:] == fill).all())


SIZES = [[1], [3], [37], [127, 128, 129], [8191, 8192, 8193], [4, 3, 2, 1, 0, 5], [100_003, 1, 70_000], [0], [0, 0, 7],
         list(range(1, 98)), [2049] * 50, [64, 65, 66, 67, 68, 191, 192, 193]]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{max(s)}")
def test_step(sizes, bits):
    Case(sizes, bits).run()
    Case(sizes, bits, BF16, copies=False).run(step=1, seed=0)
    for shift in (1, 2, 3):
        Case(sizes, bits, (F32, BF16)[shift % 2], shift=shift, seed=shift).run(seed=(shift << 40) + shift)
    log(f"adamw {len(sizes)} tensors, {bits} bits")


@pytest.mark.parametrize("bits", [32, 8])
def test_hyperparameters(bits):
    for step, more in ((1, dict(betas=(0.0, 0.0))), (1000, dict(betas=(0.9, 0.999))), (3, dict(weight_decay=0.0)),
                       (7, dict(lr=0.0)), (7, dict(eps=1e-3)), (2, dict(lr=-1e-3)), (1 << 40, dict())):
        Case([3000, 17], bits).run(step=step, **more)


@pytest.mark.parametrize("bits", [32, 8])
def test_clipping_as_grad_clip(bits):
    """The step's own clipping is that of clipped gradients: bit for bit where the
    factor is 1 or 0.  Between, grad_clip has its norm in 64 bits and the step the
    FP32 that it left, so the factor is off by 2^-24 and a clipped gradient by two
    roundings, of which a moment keeps 1 - beta beside its own one."""
    for max_norm in (0.01, 1e6, 0.0):
        a, b = Case([5000, 129, 1], bits, seed=4), Case([5000, 129, 1], bits, seed=4)
        norm = fq.grad_clip(a.g, float("inf"))
        fq.grad_clip(b.g, max_norm)
        a.run(norm=norm, max_norm=max_norm)
        b.run()
        if max_norm != 0.01:
            assert all(torch.equal(x, y) for x, y in zip(a.p + a.m + a.v, b.p + b.m + b.v))
        elif bits == 32:
            for x, y, g in zip(a.m, b.m, b.g):
                assert bool(((x - y).abs() <= ref.U * (2 * 0.1 * 2 * g.abs() + 2 * (y.abs() + 0.2 * g.abs()))).all())


def test_many_steps_from_new_states():
    """Twenty steps from zeros in 8 bits follow those in 32 bits: a step's rounding
    changes a moment by less than a step of E4M3, 1/8 of it, at random."""
    n = 20_000
    gen = torch.Generator(device=DEV).manual_seed(3)
    p32 = [torch.zeros(n, device=DEV)]
    p8 = [torch.zeros(n, device=DEV)]
    s32, s8 = fq.adamw_states(p32), fq.adamw_states(p8, bits=8)
    for t in range(1, 21):
        g = [torch.randn(n, generator=gen, device=DEV) + 0.5]
        fq.adamw(p32, g, *s32[:2], step=t, lr=1e-2, scales=s32[2])
        fq.adamw(p8, g, *s8[:2], step=t, lr=1e-2, scales=s8[2], seed=t)
    # every step is at most lr / (1 - 1/8) in size here as there: the mean moves alike
    assert abs(float(p8[0].mean() / p32[0].mean()) - 1) < 0.125
    assert float((p8[0] - p32[0]).abs().max()) < 20 * 1e-2


def test_rounding_keeps_the_mean():
    """Held values are right in the mean: with beta2 = 0.999 and no gradient, v
    decays, where the nearest code would never move.  65536 elements: the mean's
    deviation is below 1/8 / 2 / 256 of the value, four of those are allowed."""
    n = 65536
    p = [torch.zeros(n, device=DEV)]
    q = torch.full((n,), 0x70, dtype=U8, device=DEV)  # 128 of 448: between a group's other values
    q[::128] = 0x7E
    m, v = [torch.zeros(n, dtype=U8, device=DEV)], [q.clone()]
    scales = ([torch.zeros(n // 128, device=DEV)], [torch.full((n // 128,), 1e-3, device=DEV)])
    before = ref.moments(m[0], v[0], (scales[0][0], scales[1][0]))[1]
    fq.adamw(p, [torch.zeros(n, device=DEV)], m, v, 1, 1e-3, betas=(0.9, 0.9), scales=scales, seed=5)
    after = ref.moments(m[0], v[0], (scales[0][0], scales[1][0]))[1]
    ratio = np.sqrt(after).sum() / np.sqrt(before).sum()
    assert abs(ratio - np.sqrt(0.9)) < 4 * (1 / 8) / 2 / 256


def test_second_moment_never_vanishes():
    """An element far below its group's largest keeps a root above zero, so that
    its step stays bounded when its gradient stops."""
    n = 256
    p, g = [torch.zeros(n, device=DEV)], [torch.full((n,), 1e-7, device=DEV)]
    g[0][0] = 1e3
    m, v, scales = fq.adamw_states(p, bits=8)
    for t in range(1, 30):
        fq.adamw(p, g, m, v, t, 1e-3, scales=scales, seed=t)
        assert bool((v[0] > 0).all())
        g[0].zero_()
    assert float(p[0].abs().max()) < 1.0


def test_repeatable_and_seeded():
    runs = []
    for seed in (9, 9, 10):
        c = Case([10_000, 77], 8, seed=2)
        c.run(seed=seed)
        runs.append(c)
    same = lambda a, b: all(torch.equal(x, y) for x, y in zip(a.m + a.v, b.m + b.v))  # noqa: E731
    assert same(runs[0], runs[1]) and not same(runs[0], runs[2])
    # the second tensor's bits are not the first one's
    assert not np.array_equal(ref.random_bits(77, 9, 0), ref.random_bits(77, 9, 1))


def test_not_finite():
    for bad in (float("nan"), float("inf")):
        for bits in (32, 8):
            c = Case([1000], bits, copies=False)
            c.g[0][300] = bad
            fq.adamw(c.p, c.g, c.m, c.v, 3, scales=c.scales, **HYPER)
            p = c.p[0]
            assert not bool(torch.isfinite(p[300])) and bool(torch.isfinite(p[:300]).all())
            if bits == 8:
                held = torch.from_numpy(ref.moments(c.m[0], c.v[0], (c.scales[0][0], c.scales[1][0]))[1])
                assert bool(torch.isnan(held[256:384]).all()) and bool(torch.isfinite(held[:256]).all())


@pytest.mark.parametrize("bits", [32, 8])
def test_shapes_and_tables(bits):
    """Tensors of any shape, and more of them than one launch takes."""
    p = [torch.randn(s, device=DEV) for s in [(3, 5), (), (2, 3, 4), (128, 2)] * 30]
    g = [torch.randn_like(x) for x in p]
    flat = [x.clone().view(-1) for x in p]
    a, b = fq.adamw_states(p, bits), fq.adamw_states(flat, bits)
    fq.adamw(p, g, a[0], a[1], 1, 1e-2, scales=a[2])
    for i, f in enumerate(flat):  # one at a time: the same step
        fq.adamw([f], [g[i].view(-1)], [b[0][i]], [b[1][i]], 1, 1e-2,
                 scales=None if b[2] is None else ([b[2][0][i]], [b[2][1][i]]))
        assert torch.equal(f, p[i].view(-1))


def test_codes_of_either_type():
    """States as bytes or as the type that names their format: the same step."""
    a, b = Case([700, 31], 8, seed=3), Case([700, 31], 8, seed=3)
    a.run()
    as_values = lambda ts: [t.view(torch.float8_e4m3fn) for t in ts]  # noqa: E731
    fq.adamw(b.p, b.g, as_values(b.m), as_values(b.v), 5, scales=b.scales, seed=77, copies=b.copies, **HYPER)
    assert all(torch.equal(x, y) for x, y in zip(a.p + a.m + a.v, b.p + b.m + b.v))
    with pytest.raises(TypeError):
        fq.adamw(b.p, b.g, as_values(b.m), b.v, 5, 1e-3, scales=b.scales)


def test_no_tensors_and_parameters_given_twice():
    fq.adamw([], [], [], [], 1, 1e-3)
    x = [torch.zeros(100, device=DEV)]
    with pytest.raises(fq.Fp8qError, match="SHAPE"):
        fq.adamw(x * 2, x * 2, [x[0].clone(), x[0].clone()], [x[0].clone(), x[0].clone()], 1, 1e-3)


def test_captured():
    """A captured step repeats its numbers on what lies there."""
    a, b = Case([5000, 129], 8, seed=6), Case([5000, 129], 8, seed=6)
    go = lambda c: fq.adamw(c.p, c.g, c.m, c.v, 4, scales=c.scales, seed=3, copies=c.copies, **HYPER)  # noqa: E731
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go(a)
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        go(b)
        for x, y in zip(a.p + a.m + a.v + a.copies, b.p + b.m + b.v + b.copies):
            assert torch.equal(x, y)
