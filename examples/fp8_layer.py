"""A routed layer over block-scaled fp8 weights, end to end.

Quantises a layer of random bf16 weights to e4m3 with a scale per 128 x 128 block, runs
a decode step and a prefill chunk through fp8.Layer (router, quantiser, gate/up with
SwiGLU, down, shared expert, combine) and compares them with the layer in float32.

    python examples/fp8_layer.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from routed_expert_decode_gb300 import fp8  # noqa: E402

E, K, D, F = 64, 8, 1024, 512  # experts, picks a token, hidden and expert width


def quantize_weight(w):
    """fp8.Mat of [experts, N, K] weights whose sides are multiples of 128."""
    e, n, k = w.shape
    blocks = w.float().view(e, n // 128, 128, k // 128, 128)
    scale = blocks.abs().amax((2, 4)).clamp_min(1e-30) / 448.0
    q = (blocks / scale[:, :, None, :, None]).view(e, n, k).to(torch.float8_e4m3fn)
    return fp8.Mat(q, scale)


def plain_layer(x, idx, w, gate, up, down, shared):
    """The layer in float32 on the given routing."""
    def ffn(v, g, u, d):
        return (torch.nn.functional.silu(v @ g.T) * (v @ u.T)) @ d.T

    y = ffn(x, *(m[0] for m in shared))
    for e in range(gate.shape[0]):
        t, j = (idx == e).nonzero(as_tuple=True)
        if len(t):
            y[t] += w[t, j, None] * ffn(x[t], gate[e], up[e], down[e])
    return y


def run(tokens, seed=0):
    """Largest error of a layer call over `tokens` tokens, relative to its largest output."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std=1.0):
        v = std * torch.randn(shape, generator=g, device="cuda")
        return v.bfloat16()

    gate, up = normal(E, F, D, std=D ** -0.5), normal(E, F, D, std=D ** -0.5)
    down = normal(E, D, F, std=F ** -0.5)
    shared = (normal(1, F, D, std=D ** -0.5), normal(1, F, D, std=D ** -0.5),
              normal(1, D, F, std=F ** -0.5))
    router = fp8.make_router(E, K, n_group=8, topk_group=4, score=fp8.SCORE_SIGMOID, s=2.5)
    layer = fp8.Layer(router, quantize_weight(gate), quantize_weight(up), quantize_weight(down),
                      tuple(quantize_weight(m) for m in shared))
    x = normal(tokens, D)
    logits = normal(tokens, E)
    bias = 0.1 * torch.randn(E, generator=g, device="cuda")
    out = layer.forward(x, logits, bias)
    status = fp8.check_device_error(layer.buffers(tokens, x.dtype)["ws"])
    assert status == 0, status
    ref = plain_layer(x.float(), out.idx, out.w, gate.float(), up.float(), down.float(),
                      [m.float() for m in shared])
    return float(((out.y.float() - ref).abs().amax(1) / ref.abs().amax(1)).max()), out


if __name__ == "__main__":
    for n in (1, 512):
        print(f"{n} tokens: error against the float32 layer {run(n)[0]:.3f} of its largest output")
