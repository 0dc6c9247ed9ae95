"""Outputs of a layer's call whose buffers a later call has taken, without a GPU."""
import pytest
import torch

from routed_expert_decode_gb300 import fp8, router_grad


def output(call):
    return fp8.LayerOutput(*[torch.zeros(1)] * 12, call=call)


@pytest.mark.parametrize("kind", [0, 1])
def test_a_stale_output_is_refused(kind):
    """Plain calls and captured ones (1) count apart."""
    calls = [1, 1]
    out = output((calls, kind, 1))
    assert not out.stale and not output(None).stale
    calls[1 - kind] += 1
    assert not out.stale
    calls[kind] += 1
    assert out.stale
    with pytest.raises(ValueError, match="earlier call"):
        router_grad.layer_gradients(fp8.make_router(4, 2), out, torch.zeros((3, 4)),
                                    torch.zeros((3, 8)))
