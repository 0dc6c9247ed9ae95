"""GB300 routed Mixture-of-Experts layer: sigmoid+bias top-k routing, a stable
expert permutation, int8 block-quantised SwiGLU experts (Q8_0 or 2-bit) with a
shared expert, and an ordered combine -- all in the CUDA library ``libmoe.so``.

``routed_expert_decode_gb300.moe`` is the Python binding of its C ABI
(``include/moe.h``); ``routed_expert_decode_gb300.fp8`` that of the block-scaled
fp8 experts and their group-limited router (``include/moe_fp8.h``), ``.int8`` that
of experts in int8 with a scale per channel and token (``include/moe_int8.h``), and
``.router_grad`` that of the balance loss and the router's gradients
(``include/moe_router_grad.h``).
"""
from . import fp8, int8, moe, router_grad  # noqa: F401

__all__ = ["fp8", "int8", "moe", "router_grad"]
