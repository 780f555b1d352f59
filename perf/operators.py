"""Cases and plain forms of the MoE routing operators and of gradient clipping.

Five operators stand around the grouped FP8 products of an MoE layer:

    route     logits -> the chosen experts and their weights, and its gradient
    sort      the chosen experts -> rows in expert order and the map to them
    dispatch  token rows into expert order (with 1x128 E4M3 codes), and its gradient
    combine   expert rows back into token order with the weights, and its gradient
    clip      the global norm of many gradients, and their clipping

T tokens choose k of E experts each; pair t*k + j is token t's j-th choice.
With `own` false every operator is computed by elementary torch operations,
with `own` true by the library's entry points.  Codes are E4M3 values with an
FP32 scale per 128 columns: s = max(amax, 2^-100) / 448.
"""

import math

import torch

own = False

DEV = "cuda:0"
BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
FP8_MAX, AMAX_FLOOR = 448.0, 2.0 ** -100


def listed():
    return [
        # one token being generated, 32 experts: the router's smallest call
        route("route_decode", 1, 32, 2, "bf16", "softmax", bias=False, renorm=True),
        # a training batch over many small experts, balanced by a bias on the choice
        route("route_train", 16384, 256, 8, "f32", "sigmoid", bias=True, renorm=True, scale=2.5, masked=0.01),
        # the backward of a softmax router whose weights are not renormalized (a dense gradient), odd sizes
        route("route_bwd_odd", 8191, 160, 6, "bf16", "softmax", bias=False, renorm=False, masked=0.02, backward=True),
        # sixteen sequences generating one token each
        sort("sort_decode", 16, 256, 8),
        # a large training batch, some pairs not kept (padding tokens, experts of another device)
        sort("sort_train", 32768, 256, 8, dropped=0.05),
        # eight tokens being generated, straight to the codes the grouped product reads
        dispatch("dispatch_decode", 8, 32, 8, 7168, "bf16", "codes"),
        # the 16384-row MoE layer: rows for the weight gradient, codes for the product
        dispatch("dispatch_train", 2048, 32, 8, 7168, "bf16", "both"),
        # its gradient at odd sizes in FP32, some pairs dropped
        dispatch("dispatch_bwd_odd", 1531, 32, 6, 2047, "f32", "rows", dropped=0.1, backward=True),
        # eight generated tokens coming back
        combine("combine_decode", 8, 32, 8, 7168, "bf16", "rows"),
        # the backward of a 32768-row MoE layer, output gradients straight to codes as well
        combine("combine_bwd_train", 4096, 32, 8, 7168, "bf16", "both", backward=True),
        # the small tensors of a model: norms, biases, routers, odd sizes
        clip("clip_small", 60, 37, 100_000, "f32"),
        # the expert weights' gradients of a 32-expert MoE layer, clipped to BF16 for the optimizer
        clip("clip_experts", 4, 8 * 2048 * 7168, 8 * 2048 * 7168, "bf16"),
    ]


def route(name, tokens, experts, k, dtype, score, bias, renorm, scale=1.0, masked=0.0, backward=False):
    return {"name": name, "op": "route", "tokens": tokens, "experts": experts, "k": k, "dtype": dtype, "score": score,
            "bias": bias, "renorm": renorm, "scale": scale, "masked": masked, "backward": backward}


def sort(name, tokens, experts, k, dropped=0.0):
    return {"name": name, "op": "sort", "tokens": tokens, "experts": experts, "k": k, "dropped": dropped}


def dispatch(name, tokens, experts, k, cols, dtype, out, dropped=0.0, backward=False):
    return {"name": name, "op": "dispatch", "tokens": tokens, "experts": experts, "k": k, "cols": cols, "dtype": dtype,
            "out": out, "dropped": dropped, "backward": backward}


def combine(name, tokens, experts, k, cols, dtype, out, dropped=0.0, backward=False):
    return {**dispatch(name, tokens, experts, k, cols, dtype, out, dropped, backward), "op": "combine"}


def clip(name, tensors, least, most, out_dtype, max_norm=1.0):
    """`tensors` FP32 gradients with between `least` and `most` elements."""
    return {"name": name, "op": "clip", "tensors": tensors, "least": least, "most": most, "out_dtype": out_dtype,
            "max_norm": max_norm}


def log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "route", "sort", "dispatch", "dispatch", "combine", "combine", "clip"])
    if op == "clip":
        count = rng.randint(1, 60)
        most = log_int(rng, 100, 400_000_000 // count)
        case = clip("", count, log_int(rng, 1, most), most, rng.choice(["f32", "bf16"]), rng.choice([0.5, 1.0, 1e6]))
    else:
        k = rng.randint(1, 8)
        experts = log_int(rng, max(k, 4), 384)
        dropped = rng.choice([0.0, 0.0, rng.uniform(0.0, 0.3)])
        dtype = rng.choice(["bf16", "bf16", "f32"])
        if op == "route":
            case = route("", log_int(rng, 1, 16384), experts, k, dtype, rng.choice(["softmax", "sigmoid"]),
                         bias=rng.random() < 0.5, renorm=rng.random() < 0.5, scale=rng.choice([1.0, 2.5]),
                         masked=rng.choice([0.0, 0.05]), backward=rng.random() < 0.5)
        elif op == "sort":
            case = sort("", log_int(rng, 1, 32768), experts, k, dropped)
        else:
            cols = log_int(rng, 64, 8192)
            if rng.random() < 0.6:
                cols = -(-cols // 128) * 128
            tokens = log_int(rng, 1, min(16384, 230_000_000 // (cols * k)))
            out = rng.choice(["rows", "codes", "both"])
            case = (dispatch if op == "dispatch" else combine)("", tokens, experts, k, cols, dtype, out, dropped,
                                                               backward=rng.random() < 0.5)
    del case["name"]
    return case


def work(case):
    op = case["op"]
    if op == "clip":
        n = sum(clip_sizes(case))
        return {"bytes": n * (4 + (2 if case["out_dtype"] == "bf16" else 4)) + 4, "flops": 3 * n}
    t, k = case["tokens"], case["k"]
    if op == "sort":
        return {"bytes": 12 * t * k + 4 * case["experts"] + 4, "flops": 0}
    es = 2 if case["dtype"] == "bf16" else 4
    if op == "route":
        n = t * case["experts"]
        if not case["backward"]:
            return {"bytes": n * es + 8 * t * k + (4 * case["experts"] if case["bias"] else 0), "flops": 4 * n}
        # the logits: all of them for the dense gradient, else the chosen ones
        dense = case["score"] == "softmax" and not case["renorm"]
        return {"bytes": n * es + (n if dense else t * k) * es + 8 * t * k, "flops": 4 * n}
    h = case["cols"]
    m = t * k
    out = (m * h * es if case["out"] != "codes" else 0) + (m * (h + 4 * -(-h // 128)) if case["out"] != "rows" else 0)
    if op == "dispatch":
        if case["backward"]:
            return {"bytes": (m + t) * h * es + 4 * m, "flops": m * h}
        return {"bytes": t * h * es + out + 4 * m, "flops": 0}
    if not case["backward"]:
        return {"bytes": (m + t) * h * es + 8 * m, "flops": 2 * m * h}
    return {"bytes": (m + t) * h * es + out + 12 * m, "flops": 3 * m * h}


# ------------------------------------------------------------------- inputs
def clip_sizes(case):
    """Element counts spread over the case's range by their logarithm, most of them odd."""
    lo, hi, n = math.log(case["least"]), math.log(case["most"]), case["tensors"]
    if case["least"] == case["most"]:
        return [case["most"]] * n
    return [max(1, min(case["most"], int(math.exp(lo + (hi - lo) * i / max(1, n - 1))) | 1)) for i in range(n)]


def dtype_of(name):
    return BF16 if name == "bf16" else F32


def make_logits(case, gen):
    """Router logits: some experts liked by all tokens, and a fraction of experts
    masked for a token (-inf); where experts are masked, one token in 64 is padding
    and has no expert at all."""
    t, e = case["tokens"], case["experts"]
    x = torch.randn(t, e, generator=gen, device=DEV) * 1.5 + torch.randn(e, generator=gen, device=DEV) * 0.7
    if case["masked"]:
        x.masked_fill_(torch.rand(t, e, generator=gen, device=DEV) < case["masked"], -math.inf)
        x.masked_fill_(torch.rand(t, 1, generator=gen, device=DEV) < 1 / 64, -math.inf)
    return x.to(dtype_of(case["dtype"]))


def make_ids(case, gen):
    """k different experts per token, some experts far more popular than others;
    a dropped pair has the id -1."""
    t, e, k = case["tokens"], case["experts"], case["k"]
    rank = torch.randperm(e, generator=gen, device=DEV).float() + 1
    gumbel = -torch.log(-torch.log(torch.rand(t, e, generator=gen, device=DEV).clamp(1e-7, 1 - 1e-7)))
    ids = torch.topk(gumbel - torch.log(rank), k, dim=1).indices.to(torch.int32)
    if case["dropped"]:
        ids.masked_fill_(torch.rand(t, k, generator=gen, device=DEV) < case["dropped"], -1)
    return ids


def make_rows(rows, cols, dtype, gen):
    """Activations with some channels, and some rows, far larger than the rest."""
    x = torch.randn(rows, cols, generator=gen, device=DEV)
    x *= torch.where(torch.rand(cols, generator=gen, device=DEV) < 0.02, 20.0, 1.0)
    x *= torch.where(torch.rand(rows, 1, generator=gen, device=DEV) < 0.01, 100.0, 1.0)
    return x.to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    s = {"case": case}
    op = case["op"]
    if op == "clip":
        out = dtype_of(case["out_dtype"])
        s["grads"] = [torch.randn(n, generator=gen, device=DEV) * 0.02 for n in clip_sizes(case)]
        s["out"] = [torch.empty_like(g, dtype=out) for g in s["grads"]]
        return s
    if op == "route":
        s["logits"] = make_logits(case, gen)
        s["bias"] = torch.randn(case["experts"], generator=gen, device=DEV) * 0.05 if case["bias"] else None
        if case["backward"]:
            s["ids"] = plain_route(s["logits"], s["bias"], case)[0]
            s["dw"] = torch.randn(case["tokens"], case["k"], generator=gen, device=DEV)
        return s
    ids = make_ids(case, gen)
    if op == "sort":
        s["ids"] = ids
        return s
    _, s["dst"], _ = plain_sort(ids, case["experts"])
    t, m, dt = case["tokens"], case["tokens"] * case["k"], dtype_of(case["dtype"])
    if op == "dispatch":
        s["x"] = make_rows(m if case["backward"] else t, case["cols"], dt, gen)
        return s
    w = torch.rand(t, case["k"], generator=gen, device=DEV) + 0.1
    s["w"] = w / w.sum(1, keepdim=True)
    s["yp"] = make_rows(m, case["cols"], dt, gen)
    if case["backward"]:
        s["dy"] = make_rows(t, case["cols"], dt, gen)
    return s


# -------------------------------------------------------------- plain forms
def plain_route(logits, bias, case):
    """The k greatest in descending order, ties to the lowest index, -1 for a
    masked expert.  Without a bias the logits decide, with one the score plus
    the bias in 64 bits (a border between two experts may lie below 32)."""
    k = case["k"]
    if bias is None:
        key = logits.float()
    else:
        x = logits.double()
        score = torch.sigmoid(x) if case["score"] == "sigmoid" else plain_softmax(x)
        key = (score + bias.double()).masked_fill(logits == -math.inf, -math.inf)
    ids = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :k]
    chosen = torch.gather(logits, 1, ids).float()
    gone = chosen == -math.inf
    w = torch.gather(plain_scores(logits, case), 1, ids)
    w = w.masked_fill(gone, 0.0)
    if case["renorm"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, 0.0)
    return ids.masked_fill(gone, -1).to(torch.int32), w * case["scale"]


def plain_softmax(x):
    """Softmax of each row; a row of -inf alone gives zeros."""
    top = x.amax(1, keepdim=True)
    e = torch.exp(x - torch.where(top == -math.inf, 0.0, top))
    total = e.sum(1, keepdim=True)
    return torch.where(total > 0, e / total, 0.0)


def plain_scores(logits, case):
    x = logits.float()
    return torch.sigmoid(x) if case["score"] == "sigmoid" else plain_softmax(x)


def plain_route_bwd(dw, logits, ids, case):
    gone = ids < 0
    at = ids.clamp(min=0).long()
    g = (dw * case["scale"]).masked_fill(gone, 0.0)
    p = plain_scores(logits, case)
    ps = torch.gather(p, 1, at).masked_fill(gone, 0.0)
    if case["renorm"]:  # the gradient of the chosen scores over their sum
        total = ps.sum(1, keepdim=True)
        g = torch.where(total > 0, (g - (g * ps).sum(1, keepdim=True) / total) / total, 0.0).masked_fill(gone, 0.0)
    dp = torch.zeros_like(p).scatter_add(1, at, g)
    if case["score"] == "sigmoid":
        dl = dp * p * (1 - p)
    else:
        dl = p * (dp - (p * dp).sum(1, keepdim=True))
    return dl.to(logits.dtype)


def plain_sort(ids, experts):
    flat = ids.reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < experts), flat, experts)
    ordered, src = torch.sort(key, stable=True)
    offsets = torch.searchsorted(ordered, torch.arange(experts + 1, device=ids.device))
    row = torch.empty_like(src).scatter_(0, src, torch.arange(src.numel(), device=ids.device))
    dst = torch.where(key < experts, row, -1 - row)
    return offsets.to(torch.int32), dst.to(torch.int32).reshape(ids.shape), src.to(torch.int32)


def plain_quant(x):
    """1x128 E4M3 codes and scales of the rows of x."""
    cols = x.shape[1]
    v = torch.nn.functional.pad(x.float(), (0, -cols % 128)).reshape(x.shape[0], -1, 128)
    amax = v.abs().amax(2).clamp(min=AMAX_FLOOR)
    q = (v * (FP8_MAX / amax).unsqueeze(2)).to(torch.float8_e4m3fn)
    return q.reshape(x.shape[0], -1)[:, :cols].contiguous(), amax / FP8_MAX


def plain_spread(v, dst):
    """v[t, j] (or v[t]) as the rows dst[t, j] of the expert order, zeros for a dropped pair."""
    t, k = dst.shape
    flat = dst.reshape(-1).long()
    row = torch.where(flat < 0, -1 - flat, flat)
    v = v.expand(t, k, v.shape[-1]).reshape(t * k, -1).masked_fill((flat < 0).unsqueeze(1), 0.0)
    return torch.empty_like(v).index_copy_(0, row, v)


def plain_fetch(rows, dst):
    """rows[dst[t, j]] in 32 bits, zeros for a dropped pair."""
    return rows[dst.clamp(min=0).long()].float().masked_fill((dst < 0).unsqueeze(2), 0.0)


def outputs(rows, case):
    """What a forward dispatch, or a backward combine, hands on: rows, codes and scales, or both."""
    q, s = plain_quant(rows) if case["out"] != "rows" else (None, None)
    return {"rows": rows if case["out"] != "codes" else None, "codes": q, "scales": s}


def plain(s):
    case = s["case"]
    op = case["op"]
    if op == "clip":
        norm = sum(g.square().sum(dtype=F64) for g in s["grads"]).sqrt()
        c = torch.where(norm <= case["max_norm"], 1.0, case["max_norm"] / norm).float()
        return {"norm": norm.float(), "grads": [(g * c).to(o.dtype) for g, o in zip(s["grads"], s["out"])]}
    if op == "route":
        if case["backward"]:
            return plain_route_bwd(s["dw"], s["logits"], s["ids"], case)
        return plain_route(s["logits"], s["bias"], case)
    if op == "sort":
        return plain_sort(s["ids"], case["experts"])
    dst = s["dst"]
    if op == "dispatch":
        if case["backward"]:
            return plain_fetch(s["x"], dst).sum(1).to(s["x"].dtype)
        return outputs(plain_spread(s["x"].unsqueeze(1), dst), case)
    if not case["backward"]:
        return (plain_fetch(s["yp"], dst) * s["w"].unsqueeze(2)).sum(1).to(s["yp"].dtype)
    dy = s["dy"].float().unsqueeze(1)
    dw = (plain_fetch(s["yp"], dst) * dy).sum(2)
    rows = plain_spread((dy * s["w"].unsqueeze(2)).to(s["yp"].dtype), dst)
    return {**outputs(rows, case), "dw": dw}


# --------------------------------------------------------- the library's calls
def as_values(q):
    return q.view(torch.float8_e4m3fn)


def library(s):
    import fp8_fine_grained_quant_amd as fq
    case = s["case"]
    op = case["op"]
    if op == "clip":
        return {"norm": fq.grad_clip(s["grads"], case["max_norm"], out=s["out"]), "grads": s["out"]}
    if op == "route":
        if case["backward"]:
            return fq.moe_route_bwd(s["dw"], s["logits"], s["ids"], score=case["score"],
                                    renormalize=case["renorm"], scale=case["scale"])
        return fq.moe_route(s["logits"], case["k"], score=case["score"], bias=s["bias"],
                            renormalize=case["renorm"], scale=case["scale"])
    if op == "sort":
        return fq.moe_sort(s["ids"], case["experts"])
    dst, out = s["dst"], case["out"]
    if op == "dispatch":
        if case["backward"]:
            return fq.moe_dispatch_bwd(s["x"], dst)
        if out == "rows":
            return {"rows": fq.moe_dispatch(s["x"], dst)}
        rows, q, sc = fq.moe_dispatch_quant(s["x"], dst, with_output=out == "both")
        return {"rows": rows, "codes": as_values(q), "scales": sc}
    if not case["backward"]:
        return fq.moe_combine(s["yp"], dst, s["w"])
    if out == "rows":
        rows, dw = fq.moe_combine_bwd(s["dy"], s["yp"], dst, s["w"])
        return {"rows": rows, "dw": dw}
    rows, q, sc, dw = fq.moe_combine_bwd_quant(s["dy"], s["yp"], dst, s["w"], with_output=out == "both")
    return {"rows": rows, "codes": as_values(q), "scales": sc, "dw": dw}


def run(state):
    return library(state) if own else plain(state)


# ------------------------------------------------------ definitions in 64 bits
def exact_scores(x, case):
    if case["score"] == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-x))
    return torch.exp(x - torch.logsumexp(x, 1, keepdim=True)).nan_to_num(0.0)


def exact_quant(v):
    """Each group over its own scale, rounded to the nearest E4M3 value (ties to even)."""
    cols = v.shape[1]
    group = torch.arange(cols, device=v.device) // 128
    amax = torch.zeros(v.shape[0], -(-cols // 128), dtype=F64, device=v.device)
    amax = amax.scatter_reduce(1, group.expand_as(v), v.abs(), "amax").clamp(min=AMAX_FLOOR)
    y = v * (FP8_MAX / amax)[:, group]
    step = torch.exp2(torch.frexp(y).exponent.clamp(min=-5).double() - 4)  # 3 mantissa bits, least exponent -6
    return torch.round(y / step) * step, amax / FP8_MAX


def exact_rows(rows, case):
    q, s = exact_quant(rows) if case["out"] != "rows" else (None, None)
    return {"rows": rows if case["out"] != "codes" else None, "codes": q, "scales": s}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "clip":
        norm = torch.linalg.vector_norm(torch.stack([torch.linalg.vector_norm(g, dtype=F64) for g in s["grads"]]))
        c = min(1.0, case["max_norm"] / float(norm))
        return {"norm": norm, "grads": [g.double() * c for g in s["grads"]]}
    if op == "sort":
        n, e = s["ids"].numel(), case["experts"]
        key = torch.where((s["ids"] < 0) | (s["ids"] >= e), e, s["ids"]).reshape(-1).long()
        src = torch.argsort(key * n + torch.arange(n, device=key.device))
        dst = torch.argsort(src)
        offsets = torch.cumsum(torch.bincount(key + 1, minlength=e + 2), 0)[:e + 1]
        return offsets, torch.where(key == e, -1 - dst, dst).reshape(s["ids"].shape), src
    if op == "route":
        x = s["logits"].double()
        p = exact_scores(x, case)
        if not case["backward"]:
            key = x if s["bias"] is None else torch.where(x == -math.inf, -math.inf, p + s["bias"].double())
            at = torch.argsort(key, dim=1, descending=True, stable=True)[:, :case["k"]]
            gone = torch.gather(x, 1, at) == -math.inf
            w = torch.where(gone, 0.0, torch.gather(p, 1, at))
            if case["renorm"]:
                w = (w / w.sum(1, keepdim=True)).nan_to_num(0.0)
            return torch.where(gone, -1, at), w * case["scale"]
        # through the matrix of derivatives, one output weight after the other
        dl = torch.zeros_like(x)
        kept = s["ids"] >= 0
        at = s["ids"].clamp(min=0).long()
        chosen = torch.zeros_like(p).scatter_add(1, at, kept.double())
        total = (p * chosen).sum(1) if case["renorm"] else torch.ones(len(p), dtype=F64, device=p.device)
        slope = p * (1 - p) if case["score"] == "sigmoid" else None
        for j in range(case["k"]):
            one = torch.zeros_like(p).scatter_(1, at[:, j:j + 1], kept[:, j:j + 1].double())
            pj = (p * one).sum(1, keepdim=True)
            dj = one * slope if slope is not None else pj * (one - p)          # d p_j / d l
            if case["renorm"]:
                ds = chosen * slope if slope is not None else p * (chosen - total.unsqueeze(1))  # d total / d l
                dj = dj / total.unsqueeze(1) - pj * ds / total.unsqueeze(1) ** 2
            dl += torch.where(kept[:, j:j + 1], dj.nan_to_num(0.0), 0.0) * (s["dw"][:, j:j + 1].double() * case["scale"])
        return dl
    dst = s["dst"].long()
    t, k = dst.shape
    token = torch.arange(t * k, device=dst.device) // k
    kept = dst.reshape(-1) >= 0
    if op == "dispatch" and not case["backward"]:
        rows = torch.zeros(t * k, case["cols"], dtype=F64, device=dst.device)
        rows[dst.reshape(-1)[kept]] = s["x"].double()[token[kept]]
        return exact_rows(rows, case)
    if not case["backward"] or op == "dispatch":
        rows = s["x"] if op == "dispatch" else s["yp"]
        total = torch.zeros(t, case["cols"], dtype=F64, device=dst.device)
        for j in range(k):
            at = dst[:, j]
            w = s["w"][:, j].double() if op == "combine" else torch.ones(t, dtype=F64, device=dst.device)
            total += rows[at.clamp(min=0)].double() * torch.where(at < 0, 0.0, w).unsqueeze(1)
        return total
    rows = torch.zeros(t * k, case["cols"], dtype=F64, device=dst.device)
    dw = torch.zeros(t, k, dtype=F64, device=dst.device)
    for j in range(k):
        on = dst[:, j] >= 0
        at, dy = dst[on, j], s["dy"][on].double()
        rows[at] = dy * s["w"][on, j:j + 1].double()
        dw[on, j] = (dy * s["yp"][at].double()).sum(1)
    if case["out"] == "rows":
        return {"rows": rows, "codes": None, "scales": None, "dw": dw}
    # the codes are those of the rows as they are handed on, in their own type
    q, sc = exact_quant(rows.to(s["yp"].dtype).double())
    return {"rows": rows if case["out"] == "both" else None, "codes": q, "scales": sc, "dw": dw}
