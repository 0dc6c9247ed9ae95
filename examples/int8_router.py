"""Train the router of a routed layer whose experts are frozen in int8.

A layer's experts are quantised to int8, then its router weights are fitted so that the
layer's output follows that of another router over the same experts, while the balance loss
keeps the load even.  One step: logits = x Wr^T, the layer forward, dy of the squared error,
the logits' gradient through the layer and the loss, Wr's by a product.

    python examples/int8_router.py [--steps 30]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from routed_expert_decode_gb300 import int8  # noqa: E402

E, TOP_K, D, F, T, SEQUENCES = 64, 6, 1024, 512, 1024, 4


def quantised(weights: torch.Tensor) -> int8.Mat:
    """[E, N, K] floating weights as int8 codes with a scale per output channel."""
    q = torch.empty(weights.shape, dtype=torch.int8, device=weights.device)
    s = torch.empty(weights.shape[:2], device=weights.device)
    int8.quantize(weights.flatten(0, 1), q.flatten(0, 1), s.flatten())
    return int8.Mat(q, s)


def make_layer(g: torch.Generator) -> int8.Layer:
    def random(*shape):
        return torch.randn(shape, generator=g, device="cuda") * shape[-1] ** -0.5

    router = int8.make_router(E, TOP_K, n_group=8, topk_group=4, s=2.5)
    experts = [quantised(random(E, *s)) for s in ((F, D), (F, D), (D, F))]
    shared = [quantised(random(1, *s)) for s in ((F, D), (F, D), (D, F))]
    return int8.Layer(router, *experts, shared=shared)


def step(layer, w_router, x, target, seq, coef=0.01, rate=0.2):
    """One step in place; returns (squared error a token, balance loss, the router's gradient).
    The step's length is ``rate`` of the weights', against the gradient's direction."""
    logits = x.float() @ w_router.t()
    out = layer.forward(x, logits)
    diff = out.y.float() - target
    grads = layer.router_gradients(out, logits, 2.0 * diff / len(diff), coef=coef, seq=seq)
    dw_router = grads.dlogits.t() @ x.float()
    w_router.sub_(rate * w_router.norm() / dw_router.norm() * dw_router)
    return diff.square().sum(1).mean(), grads.loss[0], dw_router


def main() -> None:
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=30)
    a = ap.parse_args()
    g = torch.Generator(device="cuda").manual_seed(1)
    layer = make_layer(g)
    teacher, w_router = (torch.randn((E, D), generator=g, device="cuda") * D ** -0.5
                         for _ in range(2))
    seq = torch.linspace(0, T, SEQUENCES + 1).int().cuda()
    for i in range(a.steps):
        x = torch.randn((T, D), generator=g, device="cuda").bfloat16()
        target = layer.forward(x, x.float() @ teacher.t()).y.float()
        err, loss, _ = step(layer, w_router, x, target, seq)
        if i % 10 == 0 or i == a.steps - 1:
            print(f"step {i}: squared error {err:.1f}, balance loss {loss:.4f}")


if __name__ == "__main__":
    main()
