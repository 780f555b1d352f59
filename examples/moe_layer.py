"""A mixture-of-experts layer trained with the library's calls from the
router's logits to the clipped gradients.

    PYTHONPATH=. python examples/moe_layer.py [steps]

Every token goes to k of E experts, each one linear map W_e [N, H]:

    forward   logits = x R^T, route, sort, dispatch (with codes), grouped FP8
              product, combine
    backward  combine gradient (with codes), grouped Dgrad and Wgrad, dispatch
              gradient, router gradient
    step      gradients clipped by their global norm, then plain SGD; the bias
              on the choice moves towards experts with fewer tokens

Nothing is read back to the host between the logits and the update."""

import sys

import torch

import fp8_fine_grained_quant_amd as fq

BF16 = torch.bfloat16


class MoELayer:
    """Router R [E, H] and stacked experts W [E*N, H], both FP32."""

    def __init__(self, hidden, out, experts, k, device="cuda", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)
        self.out, self.experts, self.k = out, experts, k
        self.router = torch.randn(experts, hidden, generator=g, device=device) * hidden ** -0.5
        self.weight = torch.randn(experts * out, hidden, generator=g, device=device) * hidden ** -0.5
        self.bias = torch.zeros(experts, device=device)

    def forward(self, x):
        """y [T, N] of x [T, H] (BF16), and what the backward pass needs."""
        logits = x.float() @ self.router.t()
        ids, w = fq.moe_route(logits, self.k, score="sigmoid", bias=self.bias)
        offsets, dst, _ = fq.moe_sort(ids, self.experts, cover=True)
        rows, xq, xs = fq.moe_dispatch_quant(x, dst)
        wq, ws, wq_t = fq.quant_weight_128x128(self.weight)
        yp = fq.grouped_gemm(xq, xs, wq.view(self.experts, self.out, -1),
                             ws.view(self.experts, self.out // 128, -1), offsets)
        return fq.moe_combine(yp, dst, w), (x, logits, ids, w, offsets, dst, rows, yp, wq_t, ws)

    def backward(self, dy, kept):
        """dx [T, H] and the gradients of the router and of the experts."""
        x, logits, ids, w, offsets, dst, rows, yp, wq_t, ws = kept
        dyp, dyq, dys, dw = fq.moe_combine_bwd_quant(dy, yp, dst, w)
        drows = fq.grouped_gemm_dgrad(dyq, dys, wq_t, ws, offsets)
        dweight = fq.grouped_gemm_wgrad(*fq.quant_transpose_grouped(dyp, offsets),
                                        *fq.quant_transpose_grouped(rows, offsets), offsets, rows.shape[0])
        dlogits = fq.moe_route_bwd(dw, logits, ids, score="sigmoid")
        dx = fq.moe_dispatch_bwd(drows, dst).float() + dlogits @ self.router
        return dx.to(x.dtype), dlogits.t() @ x.float(), dweight.view(self.weight.shape)

    def update(self, grads, offsets, rate=2.0, max_norm=1.0, balance=1e-3):
        """Clips the gradients in place, applies them; returns their norm."""
        norm = fq.grad_clip(list(grads), max_norm)
        for p, g in zip((self.router, self.weight), grads):
            p.sub_(g, alpha=rate)
        load = offsets[1:] - offsets[:-1]
        self.bias.add_(torch.sign(load.float().mean() - load), alpha=balance)
        return norm


def train(steps, tokens=2048, hidden=512, out=256, experts=16, k=4, device="cuda", say=print):
    """Fits the layer to a layer of other weights; returns the losses."""
    layer = MoELayer(hidden, out, experts, k, device, seed=1)
    teacher = MoELayer(hidden, out, experts, k, device, seed=2)
    g = torch.Generator(device=device).manual_seed(3)
    losses = []
    for step in range(steps):
        x = torch.randn(tokens, hidden, generator=g, device=device).to(BF16)
        want, _ = teacher.forward(x)
        y, kept = layer.forward(x)
        diff = y.float() - want.float()
        losses.append(diff.square().mean())
        dy = (diff * (2.0 / tokens)).to(BF16)
        _, *grads = layer.backward(dy, kept)
        norm = layer.update(grads, kept[4])
        if say and step % 10 == 0:
            say(f"step {step}: loss {float(losses[-1]):.4f}, gradient norm {float(norm):.3f}")
    return [float(v) for v in losses]


if __name__ == "__main__":
    train(int(sys.argv[1]) if len(sys.argv) > 1 else 100)
