"""A pre-norm gated feed-forward block trained with the library's calls from the
residual stream to the optimizer's step.

    PYTHONPATH=. python examples/gated_block.py [steps]

    forward   norm of the stream (with the residual's addition and codes), gated
              block (both projections, activation and product in one kernel),
              FP8 output projection
    backward  output projection's Dgrad with the block's derivative, Dgrad and
              Wgrad of the stacked projections, norm gradient
    step      global norm of the gradients, AdamW with 8-bit states that clips
              by it

Nothing is read back to the host between the stream and the update."""

import sys

import torch

import fp8_fine_grained_quant_amd as fq

BF16 = torch.bfloat16


class GatedBlock:
    """Norm weight [H], gate and up stacked [2F, H], output projection [H, F], all FP32."""

    def __init__(self, hidden, width, device="cuda", seed=0, bits=8):
        g = torch.Generator(device=device).manual_seed(seed)
        self.norm = torch.ones(hidden, device=device)
        self.gate_up = torch.randn(2 * width, hidden, generator=g, device=device) * hidden ** -0.5
        self.out = torch.randn(hidden, width, generator=g, device=device) * width ** -0.5
        self.states = fq.adamw_states(self.params(), bits)

    def params(self):
        return [self.norm, self.gate_up, self.out]

    def forward(self, x, residual):
        """y and the stream x + residual (both [T, H] BF16), and what the backward pass needs."""
        xn, xq, xs, stream, rstd = fq.rms_norm_quant(x, self.norm, residual, with_output=True)
        wq, ws, wq_t = fq.quant_weight_128x128(self.gate_up)
        h, gu, hq, hs = fq.gemm_swiglu_quant(xq, xs, wq, ws, with_gu=True)
        oq, os_, oq_t = fq.quant_weight_128x128(self.out)
        y = fq.gemm_fprop(hq, hs, oq, os_)
        return y, stream, (xn, stream, rstd, gu, wq_t, ws, oq_t, os_)

    def backward(self, dy, dstream, kept):
        """Gradient of x and residual [T, H] and those of the parameters; T a multiple of 128."""
        xn, stream, rstd, gu, wq_t, ws, oq_t, os_ = kept
        dyq, dys, dyq_t, dys_t = fq.quant_act_transpose(dy)
        dgu, h = fq.gemm_dgrad_swiglu(dyq, dys, oq_t, os_, gu, with_h=True)
        dout = fq.gemm_wgrad(dyq_t, dys_t, *fq.quant_transpose(h))
        dq, ds, dq_t, ds_t = fq.quant_act_transpose(dgu)
        dgate_up = fq.gemm_wgrad(dq_t, ds_t, *fq.quant_transpose(xn))
        dxn = fq.gemm_dgrad(dq, ds, wq_t, ws)
        dx, dnorm = fq.rms_norm_bwd(dxn, stream, self.norm, rstd, dstream)
        return dx, [dnorm, dgate_up, dout]

    def update(self, grads, step, rate=3e-3, max_norm=1.0):
        """One AdamW step, clipped; returns the gradients' norm."""
        norm = fq.grad_clip(grads, float("inf"))
        m, v, scales = self.states
        fq.adamw(self.params(), grads, m, v, step, rate, weight_decay=0.01, scales=scales, seed=step, norm=norm,
                 max_norm=max_norm)
        return norm


def train(steps, tokens=1024, hidden=512, width=512, device="cuda", bits=8, say=print):
    """Fits the block to a block of other weights; returns the losses."""
    block, teacher = GatedBlock(hidden, width, device, seed=1, bits=bits), GatedBlock(hidden, width, device, seed=2)
    g = torch.Generator(device=device).manual_seed(3)
    losses = []
    for step in range(1, steps + 1):
        x, residual = (torch.randn(tokens, hidden, generator=g, device=device).to(BF16) for _ in range(2))
        want, _, _ = teacher.forward(x, residual)
        y, stream, kept = block.forward(x, residual)
        diff = y.float() - want.float()
        losses.append(diff.square().mean())
        _, grads = block.backward((diff * (2.0 / tokens)).to(BF16), torch.zeros_like(stream), kept)
        norm = block.update(grads, step)
        if say and step % 10 == 1:
            say(f"step {step}: loss {float(losses[-1]):.4f}, gradient norm {float(norm):.3f}")
    return [float(v) for v in losses]


if __name__ == "__main__":
    train(int(sys.argv[1]) if len(sys.argv) > 1 else 100)
