"""Token counts whose work takes more threads than one launch may have (2^32):
the result is that of calls on parts of the tokens, bit for bit."""

import pytest
import torch

import fp8_fine_grained_quant_amd as fq

pytestmark = pytest.mark.gpu

DEV, I32, BF16 = "cuda", torch.int32, torch.bfloat16
PART = 1 << 24


@pytest.fixture(autouse=True)
def give_back():
    yield
    torch.cuda.empty_cache()


def parts(tokens):
    return [(a, min(tokens, a + PART)) for a in range(0, tokens, PART)]


def test_route_and_gradient():
    """64 lanes a token (over 8 and over 16 choices): 2^26 tokens are 2^32."""
    t, e = (1 << 26) + 37, 17
    assert t * 64 > 1 << 32
    gen = torch.Generator(device=DEV).manual_seed(1)
    logits = torch.empty(t, e, dtype=BF16, device=DEV)
    for a, b in parts(t):
        logits[a:b] = torch.randn(b - a, e, generator=gen, device=DEV)
    ids, w = fq.moe_route(logits, e)
    dl = fq.moe_route_bwd(w, logits, ids, renormalize=False)
    for a, b in parts(t):
        ids2, w2 = fq.moe_route(logits[a:b], e)
        assert torch.equal(ids[a:b], ids2) and torch.equal(w[a:b], w2), a
        dl2 = fq.moe_route_bwd(w2, logits[a:b], ids2, renormalize=False)
        assert torch.equal(dl[a:b], dl2), a


def test_route_short():
    """8 lanes a token: 2^29 tokens are 2^32."""
    t = (1 << 29) + 3
    logits = torch.empty(t, 2, dtype=BF16, device=DEV)
    for a, b in parts(t):
        logits[a:b] = (torch.arange(a, b, device=DEV) * 7 % 11 - 5).unsqueeze(1) * torch.tensor([1.0, -1.0], device=DEV)
    ids, w = fq.moe_route(logits, 1, score="sigmoid", renormalize=False)
    for a, b in parts(t):
        ids2, w2 = fq.moe_route(logits[a:b], 1, score="sigmoid", renormalize=False)
        assert torch.equal(ids[a:b], ids2) and torch.equal(w[a:b], w2), a
        assert torch.equal(ids[a:b, 0], (logits[a:b, 1] > logits[a:b, 0]).to(I32)), a


def test_combine_gradient():
    """16 lanes for two choices of a token: 2^25 tokens of 16 choices are 2^32."""
    t, k, h = (1 << 25) + 5, 16, 4
    m = t * k
    assert t * (k // 2) * 16 > 1 << 32
    gen = torch.Generator(device=DEV).manual_seed(2)
    dst = (m - 1 - torch.arange(m, device=DEV)).to(I32)
    dst[::97] = -1 - dst[::97]
    dst = dst.view(t, k)
    w = torch.rand(t, k, generator=gen, device=DEV)
    dy = torch.randn(t, h, generator=gen, device=DEV).to(BF16)
    yp = torch.empty(m, h, dtype=BF16, device=DEV)
    for a in range(0, m, 1 << 27):
        yp[a:a + (1 << 27)] = torch.randn(min(m - a, 1 << 27), h, generator=gen, device=DEV)
    rows, dw = fq.moe_combine_bwd(dy, yp, dst, w)
    for a, b in parts(t):
        first, last = m - b * k, m - a * k  # the rows of these tokens
        d = dst[a:b]
        d = torch.where(d >= 0, d - first, d + first)
        rows2, dw2 = fq.moe_combine_bwd(dy[a:b], yp[first:last], d, w[a:b])
        assert torch.equal(rows[first:last], rows2) and torch.equal(dw[a:b], dw2), a
