"""int8 products whose sums pass 2^24 and are rounded on their way: odd codes of one sign, the
largest sums and lengths, on every kernel and tile.

The bar is int8_ref's: each addition of 16 products to an fp32 sum is off by less than one ulp of
a partial sum, all of which are below the last; whole numbers below 2^53 are exact in 64 bits."""
import numpy as np
import pytest
import torch

from test_int8_gpu import workspace

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24


@pytest.fixture(scope="module")
def int8(gpu):
    from routed_expert_decode_gb300 import int8 as m

    return m


class Odd:
    """Codes 91, 93 .. 127: every product odd and above 2^13."""

    def __init__(self, rows, N, K, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def codes(*shape):
            return (2 * torch.randint(45, 64, shape, generator=g, device="cuda",
                                      dtype=torch.int8) + 1)

        self.E, self.N, self.K, self.R = len(rows), N, K, sum(rows)
        self.off = [0, *np.cumsum(rows).tolist()]
        self.w, self.x = codes(self.E, N, K), codes(self.R, K)

    def product(self, int8):
        ones = torch.ones((self.E, self.N), device="cuda")
        out = torch.full((self.R, self.N), 7.0, device="cuda")
        ws = workspace(int8, self.R)
        off = torch.tensor(self.off, dtype=torch.int32, device="cuda") if self.E > 1 else None
        int8.product(int8.Mat(self.w, ones), self.x, torch.ones(self.R, device="cuda"), out, ws,
                     off=off)
        assert int8.check_device_error(ws) == 0
        return out

    def exact(self, n):
        """Of the last n channels."""
        return torch.cat([self.x[a:b].double() @ self.w[e, -n:].double().T
                          for e, (a, b) in enumerate(zip(self.off, self.off[1:]))])


@pytest.mark.parametrize("K", [4096, 8208, 131056])
@pytest.mark.parametrize("rows,N", [((20,), 70), ((64,), 19456), ((100,) * 15, 1280),
                                    ((2000,), 1040)], ids=["32", "64", "128", "pair"])
def test_sums_beyond_24_bits(int8, rows, N, K):
    c = Odd(rows, N, K, K + N)
    got, want = c.product(int8)[:, -70:].double(), c.exact(70)
    adds = -(-K // 16)
    assert want.min() > 2.0 ** 24
    rel = ((got - want) / want).abs().max().item()
    assert rel <= adds * 2 * U32 + U32, rel / U32 / adds


@pytest.mark.parametrize("rows,N", [((100,) * 15, 1280), ((2000,), 1040)], ids=["128", "pair"])
def test_sums_are_cut_off_towards_zero(int8, rows, N):
    """Sums of the other sign are those of the first, negated, and neither is above the exact
    one by more than the last rounding."""
    c = Odd(rows, N, 8208, 3)
    got, want = c.product(int8), c.exact(70)
    assert (got[:, -70:].double() <= want * (1 + U32)).all()
    c.w.neg_()
    assert torch.equal(c.product(int8), -got)


@pytest.mark.parametrize("rows,K", [((1,), 131056), ((3,), 60000), ((40,), 4099),
                                    ((300,), 131071)])
def test_the_other_kernels_sums_are_exact(int8, rows, K):
    """The kernels of few rows and of odd lengths: one rounding, that of the whole number."""
    c = Odd(rows, 70, K, 1)
    assert torch.equal(c.product(int8), c.exact(70).float())
