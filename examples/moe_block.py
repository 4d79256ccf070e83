"""A mixture-of-experts block trained and then served with the library.

Training: layer norm -> router -> top-k gating -> route build -> permute ->
experts (torch products) -> weighted combine, gradients through all of it,
their global norm clipped before the update. Serving: the same weights, the
norm and the whole layer in one call for a few tokens, as a decode step does.

    python examples/moe_block.py
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import padded_permute_combine_gb300 as p  # noqa: E402
from padded_permute_combine_gb300 import autograd as ag  # noqa: E402


class MoeBlock(torch.nn.Module):
    """y = x + MoE(layer_norm(x)) with gated experts, softmax weights over all experts."""

    def __init__(self, hidden: int, ffn: int, experts: int, top_k: int, device, dtype=torch.float32):
        super().__init__()
        self.top_k = top_k
        new = lambda *shape: torch.nn.Parameter(  # noqa: E731
            (torch.randn(*shape, device=device) * shape[-1] ** -0.5).to(dtype))
        self.norm_weight = torch.nn.Parameter(torch.ones(hidden, device=device, dtype=dtype))
        self.norm_bias = torch.nn.Parameter(torch.zeros(hidden, device=device, dtype=dtype))
        self.router = new(experts, hidden)
        self.w_gate_up = new(experts, 2 * ffn, hidden)
        self.w_down = new(experts, hidden, ffn)

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        """Training: every expert's rows as one batch of products, capacity for all of them."""
        T, (E, K) = x.shape[0], (self.router.shape[0], self.top_k)
        h = ag.layer_norm(x, self.norm_weight, self.norm_bias)
        logits = (h @ self.router.t()).float()
        probs = torch.softmax(logits, 1)
        top, _ = p.moe_topk_gating(logits.detach(), K)
        chosen = torch.zeros(T, E, dtype=torch.bool, device=x.device).scatter(1, top.long(), True)
        weights, index = ag.routing_map_to_mok_inputs(probs, chosen, K)
        route = p.moe_route_build(index, E)
        xe = ag.permute(h, route, E, T, K)
        g, u = torch.bmm(xe, self.w_gate_up.transpose(1, 2)).chunk(2, dim=2)
        ye = torch.bmm(torch.nn.functional.silu(g) * u, self.w_down.transpose(1, 2))
        return x + ag.combine(ye, weights, route, T, K)

    @torch.no_grad()
    def decode(self, x: torch.Tensor) -> torch.Tensor:
        """Serving: a few tokens, each expert's weights read once."""
        h, _, _ = p.moe_layer_norm_fwd(x, self.norm_weight, self.norm_bias)
        y, _, _ = p.moe_layer(h, self.router, self.w_gate_up, self.w_down, self.top_k, "softmax", normalize=False)
        return x + y


def main(steps: int = 120, tokens: int = 256, hidden: int = 256, ffn: int = 512, experts: int = 8, top_k: int = 2,
         lr: float = 0.3, max_norm: float = 1.0, seed: int = 0) -> dict:
    torch.manual_seed(seed)
    dev = torch.device("cuda:0")
    block = MoeBlock(hidden, ffn, experts, top_k, dev)
    x = torch.randn(tokens, hidden, device=dev)
    target = torch.tanh(x @ torch.randn(hidden, hidden, device=dev) * hidden ** -0.5)
    params = list(block.parameters())
    for q in params:
        q.grad = torch.zeros_like(q)
    grads = p.moe_grad_set([q.grad for q in params])  # one handle: the gradients stay where they are
    losses, norms = [], []
    for _ in range(steps):
        for q in params:
            q.grad.zero_()
        loss = (block(x) - target).square().sum(1).mean()
        loss.backward()
        norms.append(p.moe_clip_grads(grads, max_norm).clone())
        with torch.no_grad():
            for q in params:
                q -= lr * q.grad
        losses.append(loss.detach())
    with torch.no_grad():
        trained = block(x)
    served = {n: float((block.decode(x[:n]) - trained[:n]).abs().max()) for n in (1, 7, 64)}
    return {"losses": torch.stack(losses).tolist(), "norms": torch.stack(norms).reshape(-1).tolist(),
            "clipped": float(torch.sqrt(sum(q.grad.double().square().sum() for q in params))), "served": served}


if __name__ == "__main__":
    r = main()
    print("loss %.4f -> %.4f, gradient norm %.3f -> %.3f" % (r["losses"][0], r["losses"][-1], r["norms"][0], r["norms"][-1]))
    print("decode against the training path, largest difference:", r["served"])
