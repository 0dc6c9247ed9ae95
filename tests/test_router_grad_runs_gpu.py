"""The logits' gradient where a warp has several batches of tokens: in place, and for each score,
number of picks and normalisation against calls of few tokens."""
import numpy as np
import pytest
import torch

from test_router_grad_gpu import dev, rg, router  # noqa: F401

pytestmark = pytest.mark.gpu


class Many:
    def __init__(self, E, k, dt):
        # more than four tokens a warp: 152 SMs hold at most 4 x 8 warps each of teams of 32
        # lanes, which take several tokens a warp for 20 and 64 experts
        self.T = 120007 if E < 128 else 30011
        self.E, self.k, S = E, k, 9
        g = torch.Generator("cuda").manual_seed(E + k)
        self.logits = torch.randn((self.T, E), generator=g, device="cuda").to(dt)
        self.idx = torch.randint(-1, E + 1, (self.T, k), generator=g, device="cuda",
                                 dtype=torch.int32)
        self.dw = torch.randn((self.T, k), generator=g, device="cuda")
        self.live = (torch.rand(self.T, generator=g, device="cuda") > 0.2).to(torch.uint8)
        cuts = np.random.default_rng(E).integers(0, self.T + 1, S + 1)
        self.seq = dev(np.sort(cuts).astype(np.int32))
        self.counts = torch.randint(0, 900, (S, E), generator=g, device="cuda", dtype=torch.int32)
        self.tokens = torch.randint(1, 9000, (S,), generator=g, device="cuda", dtype=torch.int32)

    def gradient(self, rg, r, out, a=0, n=None, logits=None):  # noqa: F811
        n = self.T if n is None else n
        logits = self.logits if logits is None else logits
        rg.route_backward(r, logits[a:a + n], self.idx[a:a + n], out, self.dw[a:a + n], self.counts,
                          self.tokens, seq=(self.seq - a).clamp(0, n), live=self.live[a:a + n],
                          coef=0.5)
        return out


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("fn", [0, 1, 2])
@pytest.mark.parametrize("E,k", [(20, 5), (64, 6), (64, 12), (256, 8), (256, 32), (384, 6),
                                 (1000, 12)])
def test_in_place_and_in_parts(rg, E, k, fn, dt):  # noqa: F811
    m = Many(E, k, dt)
    for renorm in (True, False):
        r = router(E, k, fn, renorm)
        whole = m.gradient(rg, r, torch.empty_like(m.logits))
        assert torch.isfinite(whole).all()
        same = m.logits.clone()
        m.gradient(rg, r, same, logits=same)
        assert torch.equal(same, whole)
        for a in range(0, m.T, m.T // 4):
            n = min(555, m.T - a)
            few = torch.empty((n, E), dtype=dt, device="cuda")
            assert torch.equal(whole[a:a + n], m.gradient(rg, r, few, a, n)), a
