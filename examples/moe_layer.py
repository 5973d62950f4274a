"""A mixture-of-experts feed-forward layer on the block-scaled FP8 or the 8-bit integer operators.

    python examples/moe_layer.py [--tokens 64] [--hidden 2048] [--inner 1024] [--experts 32] [--top 4] [--steps 20] [--format fp8]

One decoder layer's second half, as a serving loop runs it: the residual
addition and the RMS norm leave the normalized rows as FP8 codes (and in bf16
for the router, and for rows in 8-bit integers), the router picks each token's
experts and sorts the choices by expert, each expert's gate and up projections
are one grouped product over its rows, the gated activation leaves codes again,
a second grouped product brings them back, and the choices are summed with the
router's weights.  Weights are random; nothing is read back to the host between
the steps.
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from weight_only_bit_dequant_amd import block, experts, int8  # noqa: E402


class MoELayer:
    """Experts' weights in codes; ``gate_up`` [E, 2 inner, hidden], ``down`` [E, hidden, inner], both bf16; ``ops``: block or int8."""

    def __init__(self, gain, router, gate_up, down, top, eps=1e-5, ops=block):
        self.gain, self.router, self.top, self.eps, self.ops = gain, router, top, eps, ops
        self.experts = router.shape[0]
        self.gate_up, self.down = ops.quantize_weight(gate_up), ops.quantize_weight(down)

    def route(self, y):
        """Each token's experts and weights, and the order that sorts the choices by expert."""
        return experts.route(y.float() @ self.router.float().t(), self.top)

    def __call__(self, x, residual):
        """bf16 x, residual [M, hidden] -> (layer output, new residual)."""
        y = torch.empty_like(x)
        xq, xs, residual, _ = block.add_rmsnorm_quantize(x, self.gain, self.eps, residual=residual, y_out=y)
        if self.ops is int8:  # (the norm has no form that leaves INT8 codes: its FP8 ones are not used)
            xq, xs = int8.quantize_act(y)
        r = self.route(y)
        gu = self.ops.grouped_linear(xq, xs, self.gate_up, r.offsets, rows=r.rows)
        z = self.ops.grouped_linear(*self.ops.silu_mul_quantize(gu), self.down, r.offsets)
        return experts.combine(z, r.places, r.weights), residual


def random_layer(hidden, inner, experts, top, seed=0, device="cuda", ops=block):
    g = torch.Generator(device=device).manual_seed(seed)

    def draw(*shape, scale=1.0):
        return (torch.randn(*shape, generator=g, device=device) * scale).to(torch.bfloat16)

    gain = (1 + 0.1 * torch.randn(hidden, generator=g, device=device)).to(torch.bfloat16)
    weights = (draw(experts, hidden, scale=hidden**-0.5), draw(experts, 2 * inner, hidden, scale=hidden**-0.5),
               draw(experts, hidden, inner, scale=inner**-0.5))
    return MoELayer(gain, *weights, top, ops=ops), weights, draw


def float_layer(layer, weights, x, residual):
    """The same layer in float32 from the unquantized weights (the layer's own routing)."""
    router, gate_up, down = (w.float() for w in weights)
    h = x.float() + residual.float()
    y = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + layer.eps) * layer.gain.float()
    r = layer.route(y.to(torch.bfloat16))
    z = torch.empty(r.rows.numel(), h.shape[1], device=h.device)
    off = r.offsets.tolist()
    for e in range(layer.experts):
        if off[e] < off[e + 1]:
            gate, up = (y[r.rows[off[e]:off[e + 1]].long()] @ gate_up[e].t()).chunk(2, dim=-1)
            z[off[e]:off[e + 1]] = (torch.nn.functional.silu(gate) * up) @ down[e].t()
    return (z[r.places.long()] * r.weights[..., None]).sum(1), h


def main():
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, value in dict(tokens=64, hidden=2048, inner=1024, experts=32, top=4, steps=20).items():
        p.add_argument("--" + name, type=int, default=value)
    p.add_argument("--format", choices=("fp8", "int8"), default="fp8")
    a = p.parse_args()
    layer, weights, draw = random_layer(a.hidden, a.inner, a.experts, a.top, ops=int8 if a.format == "int8" else block)
    x, residual = draw(a.tokens, a.hidden), draw(a.tokens, a.hidden, scale=4.0)
    out, h = layer(x, residual)
    want, want_h = float_layer(layer, weights, x, residual)
    rel = ((out.float() - want).norm() / want.norm()).item()
    print("relative error against the float layer: %.3f (residual %.1e)" % (rel, ((h.float() - want_h).norm() / want_h.norm()).item()))
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    for _ in range(a.steps):
        layer(x, residual)
    end.record()
    torch.cuda.synchronize()
    print("%d tokens, %d experts: %.1f us a step" % (a.tokens, a.experts, begin.elapsed_time(end) / a.steps * 1e3))


if __name__ == "__main__":
    main()
