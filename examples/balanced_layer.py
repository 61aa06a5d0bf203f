"""The expert layer of expert_layer.py with balanced routing, orthogonalised updates
and serving with 8-bit weights.

    python examples/balanced_layer.py          # needs an MI355X (gfx950)

The router's scores are sigmoids; a bias for each expert, which has a part in the
choice alone, goes up for experts with fewer tokens than the mean and down for the
others after every step.  A token keeps half the sets of experts.  The experts'
matrices are updated by their gradients orthogonalised, all of a stack in one call.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from expert_layer import ExpertLayer, g  # noqa: E402


class BalancedLayer(ExpertLayer):
    def __init__(self, width, hidden, experts, choices, sets, device="cuda", seed=0):
        super().__init__(width, hidden, experts, choices, device, seed)
        self.sets = sets
        self.balance = torch.zeros(experts, device=device)

    def _route(self, logits):
        return g.route_balanced(logits, self.choices, bias=self.balance, sets=self.sets, kept_sets=(self.sets + 1) // 2, scale=2.5)

    def _route_grad(self, logits, r, grad):
        return g.route_balanced_grad(logits, r, grad)

    def update(self, x, dy, masked=None, rate=0.02, balance_rate=0.01):
        """A training step: y and the gradients, as `step`; the parameters change."""
        loads = self._dispatch(x, masked)[1].offsets.diff().float()
        y, grads = self.step(x, dy, masked)
        for name in ("w1", "w2"):
            w = getattr(self, name)
            # (As large as entries of an orthogonal matrix of that shape, whatever the shape.)
            scale = max(1.0, w.shape[2] / w.shape[1]) ** 0.5
            w -= g.orthogonalize(grads[name], scale=rate * scale)
        self.router -= (rate * grads["router"]).to(self.router.dtype)
        self.b1 -= rate * grads["b1"]
        self.balance += balance_rate * torch.sign(loads.mean() - loads)
        return y, grads

    def pack8(self):
        """The layer's weights in 8 bits, as `serve8` reads them: (n, k) an expert."""
        def packed(w):
            q = [g.int8_quantize(w[e].t()) for e in range(w.shape[0])]
            return g.Int8Tensor(torch.stack([t.codes for t in q]), torch.stack([t.scales for t in q]), w.shape[1])
        return packed(self.w1), packed(self.w2)

    def serve8(self, x, weights, masked=None):
        q1, q2 = weights
        _, r, token, used, a = self._dispatch(x, masked)
        h = g.int8_linear(a, q1, offsets=r.offsets, bias=self.b1, activation="gelu")
        z = g.int8_linear(h, q2, offsets=r.offsets)
        return self._combine(z, r, token, used)[0]


def main():
    torch.manual_seed(0)
    layer = BalancedLayer(width=512, hidden=1024, experts=16, choices=2, sets=4)
    x = torch.randn(600, 512, device="cuda").bfloat16()
    target = torch.randn(600, 512, device="cuda")
    for i in range(5):
        y = layer.forward(x)
        loads = layer._dispatch(x)[1].offsets.diff()
        print(f"step {i}: squares {(y - target).square().mean().item():.4f}, tokens an expert {loads.min().item()} to {loads.max().item()}")
        layer.update(x, 2.0 * (y - target) / y.numel())
    y = layer.forward(x)
    served = layer.serve8(x, layer.pack8())
    print(f"8-bit serving differs from bfloat16 by {((served - y).norm() / y.norm()).item():.4f}")


if __name__ == "__main__":
    main()
