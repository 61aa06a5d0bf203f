"""An expert layer on the library's operators: a training step in bfloat16, and
the same layer serving with 4-bit weights.

    python examples/expert_layer.py            # needs an MI355X (gfx950)

Every token goes through the `choices` experts that its router prefers; an
expert is a two-layer feed-forward network.  The forward pass is

    r    = route(x . w_router)                     tokens -> experts
    a    = x[token of each slot, slots by expert]
    u    = a_e . w1_e + b1_e,  h = gelu(u)         grouped products
    z    = h_e . w2_e
    y    = sum over a token's slots of weight * z

and ``ExpertLayer.step`` returns the gradients of all of it.  The rows of a,
u, h and z are sorted by expert; a slot without an expert (a masked token) has
no row, and its contribution is zero.
"""
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import dense_gemm_optimisation_fp32_amd as g  # noqa: E402


def gelu(x):
    return 0.5 * x * (1.0 + torch.erf(x * math.sqrt(0.5)))


def gelu_slope(x):
    return 0.5 * (1.0 + torch.erf(x * math.sqrt(0.5))) + x * torch.exp(-0.5 * x * x) / math.sqrt(2.0 * math.pi)


class ExpertLayer:
    def __init__(self, width, hidden, experts, choices, device="cuda", seed=0):
        gen = torch.Generator(device=device)
        gen.manual_seed(seed)

        def normal(*shape, scale):
            return (torch.randn(shape, generator=gen, device=device) * scale).bfloat16()

        self.choices = choices
        self.router = normal(width, experts, scale=width ** -0.5)
        self.w1 = normal(experts, width, hidden, scale=width ** -0.5)
        self.b1 = torch.zeros((experts, hidden), device=device)
        self.w2 = normal(experts, hidden, width, scale=hidden ** -0.5)

    def _route(self, logits):
        return g.route(logits, self.choices)

    def _route_grad(self, logits, r, grad):
        return g.route_grad(logits, r, grad)

    def _dispatch(self, x, masked=None):
        logits = g.matmul(x.float(), self.router.float())
        if masked is not None:                       # (tokens, experts): experts a token may not use
            logits = logits.masked_fill(masked, float("-inf"))
        r = self._route(logits)
        # Slots without an expert follow the last expert's; their rows are zeros.
        used = (r.order >= 0).unsqueeze(1)
        token = (r.order.clamp(min=0) // self.choices).long()
        a = torch.where(used, x[token], torch.zeros((), dtype=x.dtype, device=x.device))
        return logits, r, token, used, a

    def _combine(self, z, r, token, used):
        """(tokens, width) in 32 bits, and each row's weight."""
        weight = r.weights.reshape(-1)[r.order.clamp(min=0).long()].unsqueeze(1) * used
        y = torch.zeros((r.weights.shape[0], z.shape[1]), dtype=torch.float32, device=z.device)
        return y.index_add_(0, token, weight * z.float()), weight

    def forward(self, x, masked=None):
        _, r, token, used, a = self._dispatch(x, masked)
        h = g.grouped_linear(a, self.w1, r.offsets, bias=self.b1, activation="gelu")
        z = g.grouped_linear(h, self.w2, r.offsets)
        return self._combine(z, r, token, used)[0]

    def step(self, x, dy, masked=None):
        """y, and the gradients for dy (tokens, width): of x and the parameters."""
        logits, r, token, used, a = self._dispatch(x, masked)
        u = g.grouped_linear(a, self.w1, r.offsets, bias=self.b1)
        h = gelu(u.float()).to(x.dtype)
        z = g.grouped_linear(h, self.w2, r.offsets)
        y, weight = self._combine(z, r, token, used)

        dy_rows = dy.float()[token]
        dz = (weight * dy_rows).to(x.dtype)
        slot_grad = torch.zeros(r.weights.numel(), device=x.device)
        slot_grad.index_add_(0, r.order.clamp(min=0).long(), (dy_rows * z.float()).sum(1) * used.squeeze(1))
        dlogits = self._route_grad(logits, r, slot_grad.view_as(r.weights))

        dw2 = g.grouped_weight_grad(h, dz, r.offsets)
        dh = g.grouped_linear(dz, self.w2.transpose(1, 2), r.offsets)
        du = (dh.float() * gelu_slope(u.float())).to(x.dtype)
        dw1 = g.grouped_weight_grad(a, du, r.offsets)
        # A row of ones times du_e: the sum over each expert's rows, whose bounds stay on the device.
        db1 = g.grouped_weight_grad(torch.ones((du.shape[0], 1), device=x.device), du.float(), r.offsets).squeeze(1)
        da = g.grouped_linear(du, self.w1.transpose(1, 2), r.offsets)
        dx = g.matmul(dlogits, self.router.float().t())
        dx.index_add_(0, token, da.float() * used)
        drouter = g.matmul(x.float().t(), dlogits)
        return y, {"x": dx, "router": drouter, "w1": dw1, "b1": db1, "w2": dw2}

    def pack(self):
        """The layer's weights in 4 bits, as `serve` reads them: (n, k) an expert."""
        def packed(w):
            q = [g.mx4_quantize(w[e].t()) for e in range(w.shape[0])]
            return g.Mx4Tensor(torch.stack([t.codes for t in q]), torch.stack([t.scales for t in q]), w.shape[1])
        return packed(self.w1), packed(self.w2)

    def serve(self, x, weights, masked=None):
        q1, q2 = weights
        _, r, token, used, a = self._dispatch(x, masked)
        h = g.mx4_linear(a, q1, offsets=r.offsets, bias=self.b1, activation="gelu")
        z = g.mx4_linear(h, q2, offsets=r.offsets)
        return self._combine(z, r, token, used)[0]


def main():
    torch.manual_seed(0)
    layer = ExpertLayer(width=512, hidden=1024, experts=8, choices=2)
    x = torch.randn(300, 512, device="cuda").bfloat16()
    masked = torch.rand(300, 8, device="cuda") < 0.2
    masked[::50] = True                              # padded tokens
    y, grads = layer.step(x, torch.randn(300, 512, device="cuda"), masked)
    forward = layer.forward(x, masked)
    print(f"step: |y| {y.norm().item():.3f}, forward differs by {((forward - y).norm() / y.norm()).item():.2e}, "
          + ", ".join(f"|d{k}| {v.float().norm().item():.3f}" for k, v in grads.items()))
    served = layer.serve(x, layer.pack(), masked)
    print(f"4-bit serving differs from bfloat16 by {((served - y).norm() / y.norm()).item():.3f}")


if __name__ == "__main__":
    main()
