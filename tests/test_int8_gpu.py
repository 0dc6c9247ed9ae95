"""The int8 operators on a GPU against the 64-bit reference.

Bars, derived from the definitions (int8_ref): quantiser codes and scales bit for bit;
products within their bound, which is three fp32 roundings where the sums of codes are
exact; h within that bound carried through SwiGLU (fp8_ref)."""
import numpy as np
import pytest
import torch

import fp8_ref
import int8_ref as ref

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
HALF_ULP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TINY = {"f32": 2.0 ** -149, "bf16": 2.0 ** -133, "f16": 2.0 ** -24}


@pytest.fixture(scope="module")
def int8(gpu):
    from routed_expert_decode_gb300 import int8 as m

    return m


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def strided(t, pad):
    """The same rows at a larger row stride."""
    wide = torch.full((t.shape[0], t.shape[1] + pad), float("nan"), dtype=t.dtype, device=t.device)
    wide[:, :t.shape[1]] = t
    return wide[:, :t.shape[1]]


# ---------------------------------------------------------------- quantiser
def check_quantized(int8, x):
    T, d = x.shape
    q = torch.full((T, d), 77, dtype=torch.int8, device="cuda")
    s = torch.full((T,), -1.0, device="cuda")
    int8.quantize(x, q, s)
    rq, rs = ref.quantize(x.float().cpu().numpy())
    s = s.cpu().numpy()
    assert np.array_equal(np.isnan(s), np.isnan(rs))
    assert np.array_equal(s[~np.isnan(s)].view(np.uint32), rs[~np.isnan(s)].view(np.uint32))
    assert np.array_equal(q.cpu().numpy(), rq)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("T,d", [(1, 1), (1, 127), (3, 128), (7, 1024), (5, 1040), (2, 2001),
                                 (33, 6144), (3, 8192), (9, 8200), (2, 20003)])
def test_quantize(int8, dt, T, d):
    rng = np.random.default_rng(T * 1000 + d)
    x = rng.standard_normal((T, d)) * np.exp2(rng.integers(-12, 8, (T, 1)))
    x[:, rng.random(d) < 0.02] *= 50
    x = dev(x.astype(np.float32)).to(TYPES[dt])
    check_quantized(int8, x)
    check_quantized(int8, strided(x, 13))
    check_quantized(int8, strided(x, 8))


def test_quantize_special_values(int8):
    x = np.zeros((8, 256), np.float32)
    x[0] = np.linspace(-500, 500, 256)
    x[1, :] = 2.0 ** -140
    x[2, 3], x[2, 200] = np.nan, 1.0
    x[3, 7], x[3, 8] = np.inf, 1.0
    x[4, :] = 3.4e38
    x[5, :] = -0.0
    x[6, 255] = -np.inf
    x[7] = np.arange(256) - 127.5  # halves: ties to even
    check_quantized(int8, dev(x))
    check_quantized(int8, dev(x[:, :255].copy()))
    int8.quantize(dev(x)[:0], torch.empty((0, 256), dtype=torch.int8, device="cuda"),
                  torch.empty(0, device="cuda"))


# ---------------------------------------------------------------- products
class Case:
    """Weights, activation codes and the rows' experts of a product call."""

    def __init__(self, rows, N, K, seed=0, top_k=0, full=False):
        """rows: rows of each expert; top_k: with a permutation over the rows; full: codes
        over the whole range, -128 among them, so that sums pass 2^24."""
        rng = np.random.default_rng(seed)
        self.E, self.N, self.K, self.R = len(rows), N, K, int(sum(rows))
        self.off = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)

        def codes(*shape):
            if full:
                return rng.integers(-128, 128, shape).astype(np.int8)
            return np.clip(np.rint(rng.standard_normal(shape) * 32), -128, 127).astype(np.int8)

        self.w = [(codes(self.E, N, K), rng.uniform(0.5, 1.5, (self.E, N)).astype(np.float32) /
                   np.float32(32 * K ** 0.5)) for _ in range(2)]
        self.top_k = max(1, top_k)
        n = -(-self.R // self.top_k)
        self.xq = codes(n, K)
        self.xs = (rng.uniform(0.5, 1.5, n) / 32).astype(np.float32)
        self.perm = rng.permutation(n * top_k)[:self.R].astype(np.int32) if top_k else None
        self.row = np.arange(self.R) if self.perm is None else self.perm // self.top_k

    def expected(self, m=0):
        """(reference, bound) of all rows."""
        y, e = np.zeros((self.R, self.N)), np.zeros((self.R, self.N))
        for i in range(self.E):
            r = slice(self.off[i], self.off[i + 1])
            x = self.row[r]
            y[r], e[r] = ref.product(self.xq[x], self.xs[x], self.w[m][0][i], self.w[m][1][i])
        return y, e

    def mats(self, int8):
        return [int8.Mat(dev(q), dev(s)) for q, s in self.w]

    def rows(self):
        return dict(off=dev(self.off) if self.E > 1 else None,
                    perm=None if self.perm is None else dev(self.perm), top_k=self.top_k)


def workspace(int8, rows):
    return torch.zeros(int8.workspace_size(rows), dtype=torch.uint8, device="cuda")


def check(out, y, e, dt):
    got = out.double().cpu().numpy()
    err = np.abs(got - y)
    bar = e + (np.abs(y) + e) * HALF_ULP[dt] * (dt != "f32") + TINY[dt]
    bad = ~(err <= bar)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:3].tolist(),
                           float((err / bar)[bad].max()))


def run_product(int8, c, dt, pad=0, ws=None, stream=None):
    out = torch.full((c.R, c.N + pad), 7.0, dtype=TYPES[dt], device="cuda")
    ws = workspace(int8, c.R) if ws is None else ws
    int8.product(c.mats(int8)[0], dev(c.xq), dev(c.xs), out[:, :c.N], ws, stream=stream,
                 **c.rows())
    assert int8.check_device_error(ws, stream) == 0
    assert (out[:, c.N:] == 7.0).all()
    return out[:, :c.N]


def run_swiglu(int8, c, dt, pad=0):
    out = torch.full((c.R, c.N + pad), 7.0, dtype=TYPES[dt], device="cuda")
    ws = workspace(int8, c.R)
    int8.swiglu(*c.mats(int8), dev(c.xq), dev(c.xs), out[:, :c.N], ws, **c.rows())
    assert int8.check_device_error(ws) == 0
    assert (out[:, c.N:] == 7.0).all()
    return out[:, :c.N]


def check_both(int8, c, dt, pad=0):
    y, e = c.expected()
    check(run_product(int8, c, dt, pad), y, e, dt)
    u, eu = c.expected(1)
    h, eh = fp8_ref.swiglu(y, e, u, eu)
    check(run_swiglu(int8, c, dt, pad), h, eh, dt)


SHAPES = [
    # rows of each expert, N, K, top_k
    ((1,), 64, 64, 0), ((1,), 1, 16, 0), ((1,), 300, 1040, 0), ((3,), 128, 128, 0),
    ((16,), 96, 256, 0), ((17,), 65, 272, 0), ((33,), 200, 512, 0), ((64,), 128, 2048, 0),
    ((65,), 130, 144, 0), ((129,), 256, 640, 0), ((256,), 128, 256, 0), ((257,), 257, 400, 0),
    ((700,), 384, 1040, 0),
    ((1, 0, 2, 5), 100, 208, 2), ((0, 0, 0, 1), 128, 512, 1), ((40, 1, 0, 300), 144, 320, 3),
    ((0, 0), 64, 64, 0), ((31, 32, 33, 63, 64, 65), 192, 384, 4), ((600, 3), 70, 96, 2),
    # K that tensor copies cannot take
    ((5,), 33, 1, 0), ((40, 2), 65, 77, 2), ((3, 1), 130, 250, 0), ((70,), 129, 1000, 0),
]


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("rows,N,K,top_k", SHAPES)
def test_products(int8, rows, N, K, top_k, dt):
    check_both(int8, Case(rows, N, K, seed=sum(rows) + N + K, top_k=top_k), dt)


@pytest.mark.parametrize("rows,N,K", [((2,), 80, 6144), ((40, 3), 130, 6144), ((300,), 128, 4096)])
def test_codes_of_the_whole_range(int8, rows, N, K):
    check_both(int8, Case(rows, N, K, seed=5, full=True), "f32")


@pytest.mark.parametrize("rows,K", [((4,), 6144), ((100,), 2048), ((300,), 1024)])
def test_sums_are_exact(int8, rows, K):
    """With unit scales the output is the whole number itself."""
    c = Case(rows, 200, K, seed=9)
    c.xs[:] = 1
    c.w[0][1][:] = 1
    want = c.xq.astype(np.int64) @ c.w[0][0][0].astype(np.int64).T
    assert (np.abs(c.xq.astype(np.int64)) @ np.abs(c.w[0][0][0].astype(np.int64)).T).max() < 2 ** 24
    got = run_product(int8, c, "f32").cpu().numpy()
    assert np.array_equal(got.astype(np.int64), want)


@pytest.mark.parametrize("value", [127, -128])
@pytest.mark.parametrize("rows", [(3,), (200,)])
def test_largest_codes(int8, rows, value):
    """Every product of the largest magnitude: sums far beyond 2^24."""
    c = Case(rows, 70, 4096, seed=1)
    c.xq[:] = value
    c.w[0][0][:] = value
    y, e = c.expected()
    check(run_product(int8, c, "f32"), y, e, "f32")


@pytest.mark.parametrize("dt", TYPES)
def test_row_strides_and_offsets(int8, dt):
    check_both(int8, Case((20, 7, 130), 72, 160, seed=3, top_k=2), dt, pad=5)


def test_code_planes_off_16_bytes(int8):
    c = Case((9, 30), 100, 64, seed=4)
    w, x = torch.zeros(c.E * c.N * c.K + 16, dtype=torch.int8, device="cuda"), dev(c.xq)
    shifted = w[3:3 + c.E * c.N * c.K].view(c.E, c.N, c.K)
    shifted.copy_(dev(c.w[0][0]))
    xs = torch.zeros(x.numel() + 16, dtype=torch.int8, device="cuda")
    xv = xs[1:1 + x.numel()].view(x.shape)
    xv.copy_(x)
    out = torch.empty((c.R, c.N), device="cuda")
    ws = workspace(int8, c.R)
    int8.product(int8.Mat(shifted, dev(c.w[0][1])), xv, dev(c.xs), out, ws, **c.rows())
    y, e = c.expected()
    check(out, y, e, "f32")


def test_share_of_the_experts(int8):
    """off may start above 0 and end below R: rows outside are left as they are."""
    c = Case((10, 20, 5, 40), 96, 128, seed=6)
    out = torch.full((c.R, c.N), 7.0, device="cuda")
    ws = workspace(int8, c.R)
    w = int8.Mat(dev(c.w[0][0][1:3]), dev(c.w[0][1][1:3]))
    int8.product(w, dev(c.xq), dev(c.xs), out, ws, off=dev(c.off[1:4]))
    y, e = c.expected()
    a, b = c.off[1], c.off[3]
    check(out[a:b], y[a:b], e[a:b], "f32")
    assert (out[:a] == 7.0).all() and (out[b:] == 7.0).all()


@pytest.mark.parametrize("off", [(0, 5, 3, 12), (-1, 2, 4, 12), (0, 2, 4, 13)])
def test_bad_offsets_write_nothing(int8, off):
    c = Case((4, 4, 4), 64, 64, seed=7)
    out = torch.full((c.R, c.N), 7.0, device="cuda")
    ws = workspace(int8, c.R)
    int8.product(c.mats(int8)[0], dev(c.xq), dev(c.xs), out, ws,
                 off=dev(np.array(off, np.int32)))
    assert int8.check_device_error(ws) != 0
    assert (out == 7.0).all()
    assert int8.check_device_error(ws) == 0


@pytest.mark.parametrize("rows", [(6, 6), (6, 200)])
def test_bad_permutation_entries_spoil_their_rows_alone(int8, rows):
    c = Case(rows, 64, 64, seed=8, top_k=2)
    bad = [1, 7]
    perm = c.perm.copy()
    perm[bad] = [-5, 2 * len(c.xq) + 3]
    out = torch.empty((c.R, c.N), device="cuda")
    ws = workspace(int8, c.R)
    int8.product(c.mats(int8)[0], dev(c.xq), dev(c.xs), out, ws, off=dev(c.off), perm=dev(perm),
                 top_k=2)
    assert int8.check_device_error(ws) != 0
    y, e = c.expected()
    good = np.setdiff1d(np.arange(c.R), bad)
    check(out[dev(good)], y[good], e[good], "f32")


def test_nan_rows_stay_alone(int8):
    """What a row of NaN leaves: its own outputs NaN, the others' untouched."""
    c = Case((5, 40), 80, 128, seed=10)
    c.xs[[2, 20]] = np.nan
    y, e = c.expected()
    out = run_product(int8, c, "f32")
    bad = np.isin(np.arange(c.R), [2, 20])
    assert torch.isnan(out[dev(np.flatnonzero(bad))]).all()
    check(out[dev(np.flatnonzero(~bad))], y[~bad], e[~bad], "f32")


def test_repeats_bit_for_bit_and_workspaces_are_left_clean(int8):
    c = Case((3, 0, 50, 400), 200, 2048, seed=11, top_k=2)
    d = Case((2,), 64, 6144, seed=12)  # few tiles of a long K
    ws = workspace(int8, c.R)
    first = [run_product(int8, x, "f32", ws=ws).clone() for x in (c, d)]
    for _ in range(3):
        for x, f in zip((c, d), first):
            assert torch.equal(run_product(int8, x, "f32", ws=ws), f)


def test_stream_and_graph(int8):
    """Calls on another stream, and captured and replayed with new inputs."""
    c, c2 = Case((4, 90), 128, 512, seed=13), Case((4, 90), 128, 512, seed=14)
    y, e = c.expected()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        out = run_product(int8, c, "f32")
    s.synchronize()
    check(out, y, e, "f32")
    mat, off, ws = c.mats(int8)[0], dev(c.off), workspace(int8, c.R)
    xq, xs, out = dev(c.xq), dev(c.xs), torch.empty((c.R, c.N), device="cuda")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        int8.product(mat, xq, xs, out, ws, off=off)
    for k in (c, c2, c):
        xq.copy_(dev(k.xq))
        xs.copy_(dev(k.xs))
        g.replay()
        k.w = c.w
        y, e = k.expected()
        check(out, y, e, "f32")


@pytest.mark.parametrize("seed", range(6))
def test_drawn_shapes(int8, seed):
    rng = np.random.default_rng(100 + seed)
    E = int(rng.choice([1, 3, 8, 24]))
    rows = rng.poisson(rng.choice([0.5, 4, 20, 90]), E)
    N, K = int(rng.integers(1, 500)), int(rng.integers(1, 120)) * int(rng.choice([16, 16, 7]))
    check_both(int8, Case(rows, N, K, seed=seed, top_k=int(rng.integers(0, 4))),
               list(TYPES)[seed % 3])
