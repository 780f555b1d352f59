"""Cases and plain forms of a training block's operators around the FP8 products.

Three operators stand beside the quantizers, the products and the clipping:

    norm    root-mean-square norm of token rows with the residual's addition,
            to rows and / or 1x128 E4M3 codes, and its gradient
    swiglu  the gated feed-forward block h = silu(x Wg^T) * (x Wu^T): both
            projections, the activation and the product in one step, dense and
            by expert, and the gradient of gate and up from that of the block's output
    adamw   an AdamW step over many tensors, states in 32 or in 8 bits

With `own` false every operator is computed by elementary torch operations,
with `own` true by the library's entry points.  Codes are E4M3 values with an
FP32 scale per 128 columns (weights: per 128 x 128 block): s = max(amax, 2^-100) / 448.
"""

import math

import torch

own = False

DEV = "cuda:0"
BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
FP8, FP8_MAX, AMAX_FLOOR = torch.float8_e4m3fn, 448.0, 2.0 ** -100
EPS = 1e-6
M32 = 0xFFFFFFFF


def listed():
    return [
        # eight sequences generating one token each, straight to the codes the products read
        norm("norm_decode", 8, 7168, "bf16", "codes", residual=True),
        # the rows of a training batch: codes for the product, rows for the weight gradient
        norm("norm_train", 4096, 7168, "bf16", "both", residual=True),
        # the first norm of a model in FP32, odd sizes
        norm("norm_odd", 1531, 2047, "f32", "rows", residual=False),
        # the backward of a large batch: the stream's gradient joins, and leaves as codes as well
        norm("norm_bwd_train", 16384, 7168, "bf16", "both", residual=True, backward=True),
        # a norm's backward at odd sizes in FP32
        norm("norm_bwd_odd", 2999, 1027, "f32", "rows", residual=False, backward=True),
        # eight tokens being generated: the weights are read once for few rows
        swiglu("swiglu_decode", 8, 2048, 7168, "codes"),
        # a training batch through one gated block, gate and up kept for the backward
        swiglu("swiglu_train", 4096, 2048, 7168, "rows", keep=True),
        # the 16384-row MoE layer: 32 experts' gated blocks, some without a token
        swiglu("swiglu_experts", 16384, 2048, 7168, "rows", experts=32),
        # the backward of a gated block through its output projection, the block's output made again
        swiglu("swiglu_bwd_train", 4096, 2048, 7168, "rows", keep=True, backward=True),
        # the small tensors of a model (norms, biases, routers): states in 32 bits
        adamw("adamw_small", 60, 37, 100_000, 32, "f32", copies=False),
        # tensors of all sizes with BF16 gradients, clipped by their norm, states in 8 bits
        adamw("adamw_odd", 200, 100, 2_000_000, 8, "bf16", copies=True, clip=True),
        # the expert weights of half an MoE layer, states in 8 bits, BF16 copies for the products
        adamw("adamw_experts", 2, 8 * 2048 * 7168, 8 * 2048 * 7168, 8, "f32", copies=True),
    ]


def norm(name, rows, cols, dtype, out, residual, backward=False):
    return {"name": name, "op": "norm", "rows": rows, "cols": cols, "dtype": dtype, "out": out, "residual": residual,
            "backward": backward}


def swiglu(name, rows, width, inner, out, keep=False, experts=0, backward=False):
    """`rows` tokens, gate and up of `width` columns each, contraction over `inner`; experts 0: one dense block."""
    return {"name": name, "op": "swiglu", "rows": rows, "width": width, "inner": inner, "out": out, "keep": keep,
            "experts": experts, "backward": backward}


def adamw(name, tensors, least, most, bits, grads, copies, clip=False, align=64):
    """`tensors` FP32 parameters with between `least` and `most` elements, each from a multiple of `align` on."""
    return {"name": name, "op": "adamw", "tensors": tensors, "least": least, "most": most, "bits": bits,
            "grads": grads, "copies": copies, "clip": clip, "align": align}


def log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "swiglu", "swiglu", "adamw"])
    if op == "norm":
        cols = log_int(rng, 64, 16384)
        if rng.random() < 0.6:
            cols = -(-cols // 128) * 128
        rows = log_int(rng, 1, min(32768, 230_000_000 // cols))
        case = norm("", rows, cols, rng.choice(["bf16", "bf16", "f32"]), rng.choice(["rows", "codes", "both"]),
                    residual=rng.random() < 0.6, backward=rng.random() < 0.5)
    elif op == "swiglu":
        width, inner = 128 * log_int(rng, 1, 32), 128 * log_int(rng, 1, 56)
        if rng.random() < 0.3:
            # a few generated tokens: codes (FP32 scales are asked of the exact path, which few rows take)
            case = swiglu("", rng.randint(1, 16), width, inner, rng.choice(["codes", "rows"]))
        else:
            backward = rng.random() < 0.4
            experts = rng.choice([0, 0, rng.randint(2, 48)])
            experts = min(experts, 940_000_000 // (2 * width * inner))
            rows = log_int(rng, 17, min(16384, 480_000_000_000 // (width * inner)))
            case = swiglu("", rows, width, inner, "rows", keep=backward or rng.random() < 0.5, experts=experts,
                          backward=backward)
    else:
        count = rng.randint(1, 120)
        most = log_int(rng, 100, 200_000_000 // count)
        case = adamw("", count, log_int(rng, 1, most), most, rng.choice([8, 8, 32]), rng.choice(["f32", "bf16"]),
                     copies=rng.random() < 0.5, clip=rng.random() < 0.5, align=rng.choice([64, 64, 1]))
    del case["name"]
    return case


def work(case):
    op = case["op"]
    if op == "adamw":
        n = sum(adamw_sizes(case))
        state = 16 if case["bits"] == 32 else 4 + 16 / 128
        return {"bytes": n * (8 + (4 if case["grads"] == "f32" else 2) + state + (2 if case["copies"] else 0)),
                "flops": 12 * n}
    if op == "norm":
        n, es = case["rows"] * case["cols"], 2 if case["dtype"] == "bf16" else 4
        groups = case["rows"] * -(-case["cols"] // 128)
        out = (n * es if case["out"] != "codes" else 0) + (n + 4 * groups if case["out"] != "rows" else 0)
        # forward: x (and the residual, and their sum out); backward: dy and x (and the stream's gradient)
        rows = (2 if case["backward"] else 1) + (0 if not case["residual"] else 1 if case["backward"] else 2)
        return {"bytes": rows * n * es + out + 4 * case["rows"] + (8 if case["backward"] else 4) * case["cols"],
                "flops": (10 if case["backward"] else 5) * n}
    m, f, k = case["rows"], case["width"], case["inner"]
    experts = min(max(1, case["experts"]), m)
    if case["backward"]:  # the output projection's weights, gate and up in, their gradients and h out
        return {"bytes": m * k + 4 * m * (k // 128) + experts * f * k + 10 * m * f, "flops": 2 * m * f * k}
    out = m * f + 4 * m * (f // 128) if case["out"] == "codes" else 2 * m * f
    return {"bytes": m * k + 4 * m * (k // 128) + experts * 2 * f * k + out + (4 * m * f if case["keep"] else 0),
            "flops": 4 * m * f * k}


# ------------------------------------------------------------------- inputs
def adamw_sizes(case):
    """Element counts spread over the case's range by their logarithm, most of them odd."""
    lo, hi, n = math.log(case["least"]), math.log(case["most"]), case["tensors"]
    if case["least"] == case["most"]:
        return [case["most"]] * n
    return [max(1, min(case["most"], int(math.exp(lo + (hi - lo) * i / max(1, n - 1))) | 1)) for i in range(n)]


def dtype_of(name):
    return BF16 if name == "bf16" else F32


def make_rows(rows, cols, dtype, gen):
    """Activations with some channels, and some rows, far larger than the rest."""
    x = torch.randn(rows, cols, generator=gen, device=DEV)
    x *= torch.where(torch.rand(cols, generator=gen, device=DEV) < 0.02, 20.0, 1.0)
    x *= torch.where(torch.rand(rows, 1, generator=gen, device=DEV) < 0.01, 100.0, 1.0)
    return x.to(dtype)


def make_weight(experts, rows, cols, std, gen):
    """Codes of normally distributed weights whose blocks' largest value is near 448, and their block scales."""
    shape = (max(1, experts), rows, cols)
    q = torch.randn(shape, generator=gen, device=DEV).mul_(105.0).clamp_(-FP8_MAX, FP8_MAX).to(FP8)
    s = std / 105.0 * (0.8 + 0.4 * torch.rand(shape[0], rows // 128, cols // 128, generator=gen, device=DEV))
    return (q, s) if experts else (q[0], s[0])


def make_counts(rows, experts, gen):
    """Tokens per expert, some experts far more popular than others, one in eight without any."""
    rank = torch.randperm(experts, generator=gen, device=DEV).float() + 1
    share = torch.where(rank > 1 + experts * 7 // 8, 0.0, 1.0 / rank)
    ends = torch.round(torch.cumsum(share.double(), 0) / share.double().sum() * rows).long().tolist()
    return [b - a for a, b in zip([0] + ends[:-1], ends)]


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    s = {"case": case}
    if case["op"] == "norm":
        m, n, dt = case["rows"], case["cols"], dtype_of(case["dtype"])
        s["x"] = make_rows(m, n, dt, gen)
        s["w"] = 1.0 + 0.2 * torch.randn(n, generator=gen, device=DEV)
        s["other"] = make_rows(m, n, dt, gen) if case["residual"] else None
        if case["backward"]:
            s["dy"] = (make_rows(m, n, F32, gen) * 1e-2).to(dt)
            s["rstd"] = torch.rsqrt(s["x"].double().square().mean(1) + EPS).float()
        return s
    if case["op"] == "swiglu":
        m, f, k, e = case["rows"], case["width"], case["inner"], case["experts"]
        x = make_rows(m, k, F32, gen) * (1e-2 if case["backward"] else 1.0)
        s["xq"], s["xs"] = plain_quant(x)
        if e:
            s["counts"] = make_counts(m, e, gen)
            ends = torch.tensor([0] + s["counts"], device=DEV).cumsum(0)
            s["offsets"] = ends.to(torch.int32)
        if case["backward"]:
            # the output projection's transposed codes [width, inner] (by expert side by side: [width, experts * inner]),
            # its block scales [inner / 128, width / 128] (by expert stacked)
            q, sc = make_weight(e, f, k, 0.02, gen)
            s["wq"] = q.permute(1, 0, 2).reshape(f, e * k).contiguous() if e else q
            s["ws"] = sc.transpose(-1, -2).reshape(-1, f // 128).contiguous()
            s["gu"] = make_rows(m, 2 * f, BF16, gen)
        else:
            s["wq"], s["ws"] = make_weight(e, 2 * f, k, k ** -0.5, gen)
        return s
    return prepare_adamw(s, case, seed, gen)


def prepare_adamw(s, case, seed, gen):
    """Every kind of value (parameters, gradients, states, copies) lies in one buffer, its tensors one after the
    other, each from a multiple of `align` elements on, as a program holds them that shards or saves them whole."""
    sizes, align = adamw_sizes(case), case["align"]
    first = [0]
    for n in sizes:
        first.append(-(-(first[-1] + n) // align) * align)
    groups = [-(-n // 128) for n in sizes]
    first_group = [sum(groups[:i]) for i in range(len(groups))]
    views = lambda buf: [buf[a:a + n] for a, n in zip(first, sizes)]  # noqa: E731
    rand = lambda std: torch.randn(first[-1], generator=gen, device=DEV).mul_(std)  # noqa: E731
    flat = {"p": rand(0.02), "m": rand(3e-4), "v": rand(1e-3).square_()}
    s["g"] = views(rand(1e-3).to(dtype_of(case["grads"])))
    s["scales"] = None
    if case["bits"] == 8:
        for kind, x in (("m", flat["m"]), ("v", flat["v"].sqrt_())):
            held = [plain_quant(v.reshape(1, -1)) for v in views(x)]
            flat[kind] = torch.zeros(first[-1], device=DEV).to(FP8)
            flat[kind + "_scales"] = torch.cat([sc.reshape(-1) for _, sc in held])
            for v, (q, _) in zip(views(flat[kind]), held):
                v.copy_(q.reshape(-1))
        s["scales"] = tuple([flat[kind][a:a + n] for a, n in zip(first_group, groups)]
                            for kind in ("m_scales", "v_scales"))
    s["copies"] = None
    if case["copies"]:
        flat["copies"] = torch.zeros(first[-1], dtype=BF16, device=DEV)
        s["copies"] = views(flat["copies"])
    s["p"], s["m"], s["v"], s["flat"] = views(flat["p"]), views(flat["m"]), views(flat["v"]), flat
    s["norm"] = torch.stack([g.double().square().sum() for g in s["g"]]).sum().sqrt().float() if case["clip"] else None
    s["max_norm"] = 0.3 * 1e-3 * math.sqrt(sum(sizes)) if case["clip"] else math.inf  # the norm is about 1e-3 sqrt(n)
    s["step"] = dict(step=10 + seed % 7, lr=3e-4, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1, seed=seed)
    return s


# -------------------------------------------------------------- plain forms
def plain_quant(x):
    """1x128 E4M3 codes and scales of the rows of x."""
    cols = x.shape[1]
    v = torch.nn.functional.pad(x.float(), (0, -cols % 128)).reshape(x.shape[0], -1, 128)
    amax = v.abs().amax(2).clamp(min=AMAX_FLOOR)
    q = (v * (FP8_MAX / amax).unsqueeze(2)).to(FP8)
    return q.reshape(x.shape[0], -1)[:, :cols].contiguous(), amax / FP8_MAX


def outputs(rows, case):
    """Rows in their type, codes and scales, or both; the codes are those of the rows before their rounding."""
    q, s = plain_quant(rows) if case["out"] != "rows" else (None, None)
    return {"rows": rows.to(dtype_of(case["dtype"])) if case["out"] != "codes" else None, "codes": q, "scales": s}


def plain_norm(s):
    case, x, w = s["case"], s["x"], s["w"]
    if not case["backward"]:
        total = None
        if s["other"] is not None:  # the residual stream is held in its type, and the norm is that of what is held
            x = total = (x.float() + s["other"].float()).to(x.dtype)
        rstd = torch.rsqrt(x.float().square().mean(1) + EPS)
        return {**outputs(x.float() * rstd.unsqueeze(1) * w, case), "sum": total, "rstd": rstd}
    xhat = x.float() * s["rstd"].unsqueeze(1)
    dy = s["dy"].float()
    dxhat = dy * w
    dx = (dxhat - xhat * (dxhat * xhat).mean(1, keepdim=True)) * s["rstd"].unsqueeze(1)
    if s["other"] is not None:
        dx = dx + s["other"].float()
    return {**outputs(dx, case), "dw": (dy * xhat).sum(0, dtype=F64).float()}


def plain_spread(q, s, rows):
    """Codes times their scales in FP32; a scale stands for 128 columns, and for `rows` rows."""
    s = s.repeat_interleave(rows, -2) if rows > 1 else s
    return (q.float().unflatten(-1, (-1, 128)) * s.unsqueeze(-1)).flatten(-2)


def plain_product(s, wq, ws):
    """x W^T in FP32, by expert where there are experts."""
    x, w = plain_spread(s["xq"], s["xs"], 1), plain_spread(wq, ws, 128)
    if "counts" not in s:
        return x @ w.t()
    return torch.cat([a @ b.t() for a, b in zip(x.split(s["counts"]), w)])


def plain_swiglu(s):
    case = s["case"]
    f, k, e = case["width"], case["inner"], case["experts"]
    if not case["backward"]:
        gu = plain_product(s, s["wq"], s["ws"])
        g, u = gu[:, :f], gu[:, f:]
        h = g * torch.sigmoid(g) * u
        if case["out"] == "codes":
            q, sc = plain_quant(h)
            return {"codes": q, "scales": sc}
        return {"h": h.to(BF16), "gu": gu.to(BF16) if case["keep"] else None}
    wq, ws = s["wq"], s["ws"]
    if e:
        wq, ws = wq.unflatten(1, (e, k)).transpose(0, 1), ws.unflatten(0, (e, -1))
    dh = plain_product(s, wq, ws.transpose(-1, -2))
    g, u = s["gu"][:, :f].float(), s["gu"][:, f:].float()
    sig = torch.sigmoid(g)
    dgu = torch.cat([dh * u * sig * (1 + g * (1 - sig)), dh * g * sig], 1)
    return {"dgu": dgu.to(BF16), "h": (g * sig * u).to(BF16)}


def mix(x):
    """A 32-bit number to another, all of whose bits depend on all of x's."""
    x = ((x ^ (x >> 16)) * 0x6C8E9CF5) & M32
    x = ((x ^ (x >> 15)) * 0xB2D05E13) & M32
    return x ^ (x >> 16)


def plain_random(n, seed, tensor):
    """The 32 random bits of every element of a list's `tensor`-th tensor."""
    key = mix((mix((seed + 0x9E3779B1 * tensor) & M32) + (seed >> 32)) & M32)
    at = torch.arange(n, device=DEV)
    return mix(((at & M32) * 0x85297A4D + (at >> 32) * 0x27D4EB2F + key) & M32)


def plain_round(y, bits, positive):
    """y (at most 448 in magnitude) to one of the two E4M3 values around it: away from
    zero where the fraction of their distance and bits / 65536 add up to 1.  positive:
    what is above zero stays so."""
    e = (torch.frexp(y).exponent - 1).clamp(min=-6)
    t = torch.floor(torch.ldexp(y.abs(), 3 - e) + bits.float() / 65536)
    if positive:
        t = torch.where(y > 0, t.clamp(min=1), t)
    return torch.copysign(torch.ldexp(t, e - 3), y).clamp(-FP8_MAX, FP8_MAX).to(FP8)


def plain_hold(x, bits, positive):
    """A state as codes and one scale per 128 elements, randomly rounded."""
    n = x.numel()
    v = torch.nn.functional.pad(x, (0, -n % 128)).reshape(-1, 128)
    amax = v.abs().amax(1).clamp(min=AMAX_FLOOR)
    y = (v * (FP8_MAX / amax).unsqueeze(1)).reshape(-1)[:n]
    return plain_round(y, bits, positive), amax / FP8_MAX


def plain_held(q, s):
    """The values of codes and scales."""
    return q.float() * s.repeat_interleave(128)[:q.numel()]


def plain_moments(s, i):
    """The two moments of tensor i in FP32."""
    if s["scales"] is None:
        return s["m"][i], s["v"][i]
    return plain_held(s["m"][i], s["scales"][0][i]), plain_held(s["v"][i], s["scales"][1][i]).square()


def plain_adamw_one(s, i):
    a, p = s["step"], s["p"][i]
    g = s["g"][i].float()
    if s["norm"] is not None:
        norm = s["norm"].double()
        g = (g.double() * torch.where(norm <= s["max_norm"], 1.0, s["max_norm"] / norm)).float()
    (b1, b2), t = a["betas"], a["step"]
    m, v = plain_moments(s, i)
    m = m * b1 + g * (1 - b1)
    v = v * b2 + g * g * (1 - b2)
    root = v.sqrt()
    step = a["lr"] / (1 - b1 ** t) * m / (root / math.sqrt(1 - b2 ** t) + a["eps"])
    p.copy_(p * (1 - a["lr"] * a["weight_decay"]) - step)
    if s["copies"]:
        s["copies"][i].copy_(p)
    if s["scales"] is None:
        s["m"][i].copy_(m)
        s["v"][i].copy_(v)
        return None
    r = plain_random(p.numel(), a["seed"], i)
    for k, (x, held, bits) in enumerate(((m, s["m"][i], r & 0xFFFF), (root, s["v"][i], r >> 16))):
        q, sc = plain_hold(x, bits, k == 1)
        held.copy_(q)
        s["scales"][k][i].copy_(sc)
    return None


def plain_adamw(s):
    [plain_adamw_one(s, i) for i in range(len(s["p"]))]
    return s["flat"]  # everything that a step changes


# --------------------------------------------------------- the library's calls
def as_codes(q):
    return q.view(torch.uint8)


def as_values(q):
    return q.view(FP8)


def library_norm(fq, s):
    case = s["case"]
    out = case["out"]
    if not case["backward"]:
        if out == "rows":
            y, total, rstd = fq.rms_norm(s["x"], s["w"], s["other"], eps=EPS)
            return {"rows": y, "sum": total, "rstd": rstd}
        y, q, sc, total, rstd = fq.rms_norm_quant(s["x"], s["w"], s["other"], eps=EPS, with_output=out == "both")
        return {"rows": y, "codes": as_values(q), "scales": sc, "sum": total, "rstd": rstd}
    if out == "rows":
        dx, dw = fq.rms_norm_bwd(s["dy"], s["x"], s["w"], s["rstd"], s["other"])
        return {"rows": dx, "dw": dw}
    dx, q, sc, dw = fq.rms_norm_bwd_quant(s["dy"], s["x"], s["w"], s["rstd"], s["other"], with_output=out == "both")
    return {"rows": dx, "codes": as_values(q), "scales": sc, "dw": dw}


def library_swiglu(fq, s):
    case = s["case"]
    xq, xs, wq, ws = as_codes(s["xq"]), s["xs"], as_codes(s["wq"]), s["ws"]
    if case["backward"]:
        if case["experts"]:
            dgu, h = fq.grouped_gemm_dgrad_swiglu(xq, xs, wq, ws, s["offsets"], s["gu"], with_h=True)
        else:
            dgu, h = fq.gemm_dgrad_swiglu(xq, xs, wq, ws, s["gu"], with_h=True)
        return {"dgu": dgu, "h": h}
    if case["experts"]:
        h, gu = fq.grouped_gemm_swiglu(xq, xs, wq, ws, s["offsets"], with_gu=case["keep"])
        return {"h": h, "gu": gu}
    if case["out"] == "codes":
        _, _, q, sc = fq.gemm_swiglu_quant(xq, xs, wq, ws, with_output=False)
        return {"codes": as_values(q), "scales": sc}
    h, gu = fq.gemm_swiglu(xq, xs, wq, ws, with_gu=case["keep"])
    return {"h": h, "gu": gu}


def library_adamw(fq, s):
    fq.adamw(s["p"], s["g"], s["m"], s["v"], scales=s["scales"], copies=s["copies"], norm=s["norm"], max_norm=s["max_norm"],
             **s["step"])
    return s["flat"]


def run(state):
    op = state["case"]["op"]
    if own:
        import fp8_fine_grained_quant_amd as fq
        return {"norm": library_norm, "swiglu": library_swiglu, "adamw": library_adamw}[op](fq, state)
    return {"norm": plain_norm, "swiglu": plain_swiglu, "adamw": plain_adamw}[op](state)


# ------------------------------------------------------ definitions in 64 bits
GRID = [(8 + (c & 7)) * 2.0 ** ((c >> 3) - 10) if c >> 3 else (c & 7) * 2.0 ** -9 for c in range(127)]


def exact_neighbours(y):
    """The E4M3 values below and above |y|, and where between them it lies."""
    grid = torch.tensor(GRID + [480.0], dtype=F64, device=y.device)
    at = (torch.searchsorted(grid, y.abs(), right=True) - 1).clamp(max=126)
    return grid[at], grid[at + 1], (y.abs() - grid[at]) / (grid[at + 1] - grid[at]), at


def exact_groups(v):
    """The largest magnitude of every 128 columns of v's rows, floored."""
    group = torch.arange(v.shape[1], device=v.device) // 128
    amax = torch.zeros(v.shape[0], -(-v.shape[1] // 128), dtype=F64, device=v.device)
    return amax.scatter_reduce(1, group.expand_as(v), v.abs(), "amax").clamp(min=AMAX_FLOOR), group


def exact_quant(v):
    """Each group over its own scale, rounded to the nearest E4M3 value (ties to the even code)."""
    amax, group = exact_groups(v)
    y = v * (FP8_MAX / amax)[:, group]
    lo, hi, part, at = exact_neighbours(y)
    up = (part > 0.5) | ((part == 0.5) & (at % 2 == 1))
    return torch.copysign(torch.where(up, hi, lo).clamp(max=FP8_MAX), y), amax / FP8_MAX


def exact_rows(rows, case):
    q, s = exact_quant(rows) if case["out"] != "rows" else (None, None)
    return {"rows": rows if case["out"] != "codes" else None, "codes": q, "scales": s}


def exact_norm(s, case):
    x, w = s["x"].double(), s["w"].double()
    if not case["backward"]:
        total = x + s["other"].double() if case["residual"] else None
        if total is not None:  # the sum as it is held
            x = total.float().to(s["x"].dtype).double()
        mean = torch.einsum("ij,ij->i", x, x) / x.shape[1]
        y = x / torch.sqrt(mean + EPS)[:, None] * w[None]
        return {**exact_rows(y, case), "sum": total, "rstd": (mean + EPS) ** -0.5}
    dy, r = s["dy"].double(), s["rstd"].double()[:, None]
    inner = torch.einsum("ij,ij->i", dy * w[None], x)[:, None] / x.shape[1]
    dx = r * w[None] * dy - r ** 3 * inner * x
    if case["residual"]:
        dx += s["other"].double()
    return {**exact_rows(dx, case), "dw": torch.einsum("ij,ij->j", dy, x * r)}


def exact_values(q, s, rows):
    """Codes times scales, the code (i, j)'s scale at (i / rows, j / 128)."""
    i = torch.arange(q.shape[0], device=q.device) // rows
    j = torch.arange(q.shape[1], device=q.device) // 128
    return q.double() * s.double()[i][:, j]


def exact_swiglu(s, case):
    f, k, m = case["width"], case["inner"], case["rows"]
    counts = s.get("counts", [m])
    x = exact_values(s["xq"], s["xs"], 1)
    gu = s["gu"].double() if case["backward"] else torch.empty(m, 2 * f, dtype=F64, device=x.device)
    dh = torch.empty(m, f, dtype=F64, device=x.device)
    at = 0
    for e, n in enumerate(counts):
        if case["backward"]:
            w = exact_values(s["wq"][:, e * k:(e + 1) * k].t(), s["ws"][e * (k // 128):(e + 1) * (k // 128)], 128)
            dh[at:at + n] = x[at:at + n] @ w
        else:
            q, sc = (s["wq"][e], s["ws"][e]) if case["experts"] else (s["wq"], s["ws"])
            gu[at:at + n] = x[at:at + n] @ exact_values(q, sc, 128).t()
        at += n
    g, u = gu[:, :f], gu[:, f:]
    silu = g / (1 + torch.exp(-g))
    if not case["backward"]:
        if case["out"] == "codes":
            q, sc = exact_quant(silu * u)
            return {"codes": q, "scales": sc}
        return {"h": silu * u, "gu": gu if case["keep"] else None}
    slope = (1 + torch.exp(-g) * (1 + g)) / (1 + torch.exp(-g)) ** 2  # d silu / d g
    slope = torch.where(g < -300, 0.0, slope)
    return {"dgu": torch.cat([dh * u * slope, dh * silu], 1), "h": silu * u}


def exact_random(n, seed, tensor):
    """The random bits again, products taken by halves of 16 bits."""
    def times(x, c):
        return (x * (c & 0xFFFF) + ((x * (c >> 16)) % 65536) * 65536) % 2 ** 32

    def mixed(x):
        x = times(x ^ x // 65536, 0x6C8E9CF5)
        x = times(x ^ x // 32768, 0xB2D05E13)
        return x ^ x // 65536

    key = mixed((mixed((seed + 0x9E3779B1 * tensor) % 2 ** 32) + seed // 2 ** 32) % 2 ** 32)
    at = torch.arange(n, device=DEV)
    return mixed((times(at % 2 ** 32, 0x85297A4D) + times(at // 2 ** 32, 0x27D4EB2F) + key) % 2 ** 32)


def exact_hold(x, part, positive):
    amax, group = exact_groups(x.reshape(1, -1))
    y = x * (FP8_MAX / amax)[0, group]
    lo, hi, where, at = exact_neighbours(y)
    value = torch.where(where + part >= 1, hi, lo).clamp(max=FP8_MAX)
    if positive:
        value = torch.where((y > 0) & (value == 0), GRID[1], value)
    return torch.copysign(value, y), amax[0] / FP8_MAX


def exact_adamw(s, case):
    a, flat = s["step"], s["flat"]
    out = {k: v.double() for k, v in flat.items()}
    first = [v.storage_offset() for v in s["p"]]
    group = 0
    (b1, b2), t = a["betas"], a["step"]
    c = 1.0 if s["norm"] is None else min(1.0, s["max_norm"] / float(s["norm"]))
    for i, (p, g) in enumerate(zip(s["p"], s["g"])):
        at, n = first[i], p.numel()
        groups = -(-n // 128)
        m, v = s["m"][i].double(), s["v"][i].double()
        if s["scales"]:
            of = torch.arange(n, device=DEV) // 128
            m, v = m * s["scales"][0][i].double()[of], (v * s["scales"][1][i].double()[of]) ** 2
        g = g.double() * c
        m = b1 * m + (1 - b1) * g
        v = b2 * v + (1 - b2) * g ** 2
        new = p.double() - a["lr"] * (m / (1 - b1 ** t) / (torch.sqrt(v / (1 - b2 ** t)) + a["eps"])
                                      + a["weight_decay"] * p.double())
        out["p"][at:at + n] = new
        if s["copies"]:
            out["copies"][at:at + n] = new
        if s["scales"]:
            r = exact_random(n, a["seed"], i)
            m, out["m_scales"][group:group + groups] = exact_hold(m, (r % 65536) / 65536.0, False)
            v, out["v_scales"][group:group + groups] = exact_hold(v.sqrt(), (r // 65536) / 65536.0, True)
        out["m"][at:at + n] = m
        out["v"][at:at + n] = v
        group += groups
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": exact_norm, "swiglu": exact_swiglu, "adamw": exact_adamw}[case["op"]](s, case)
