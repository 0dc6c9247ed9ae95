"""The int8 products where their kernels differ: shapes on each side of the rules that choose a
kernel or a tile, and places beyond 32-bit offsets."""
import numpy as np
import pytest
import torch

import int8_ref as ref
from test_int8_gpu import (HALF_ULP, TINY, TYPES, Case, check, check_both, dev, run_product,
                           workspace)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def int8(gpu):
    from routed_expert_decode_gb300 import int8 as m

    return m


def spread(E, **rows):
    """Rows of E experts, 0 but for the named ones."""
    r = [0] * E
    for e, n in rows.items():
        r[int(e[1:])] = n
    return tuple(r)


@pytest.mark.parametrize("rows,N,K,top_k", [
    # the stream for few rows: more rows of an expert than it takes at a time, odd channels
    (spread(64, e63=32), 130, 272, 3), (spread(64, e0=1, e5=7, e31=24), 65, 528, 1),
    ((1,) * 16, 6, 16, 2), ((4,), 1001, 2064, 0), (spread(9, e2=4), 3, 6160, 1),
    # one tile shared along K by several CTAs, rows on both sides of a tile's
    ((20,), 300, 6144, 0), ((33,), 130, 4112, 0), ((5, 0, 9), 200, 4096, 2), ((32,), 64, 8192, 1),
    # tiles of 64 and of 128 rows
    ((63, 64, 65, 1), 129, 144, 2), ((127, 128, 129), 200, 160, 0), ((120,) * 9, 96, 80, 2),
    # pairs of CTAs: last tiles of one row, odd channels, a share of the experts without rows
    ((513, 1, 0, 300), 257, 96, 2), ((257,) * 3, 131, 208, 0), ((1000, 0, 0), 384, 112, 4),
    ((2000,), 514, 80, 0), ((1500,), 640, 1040, 3),
])
def test_kernels(int8, rows, N, K, top_k):
    for dt in TYPES:
        check_both(int8, Case(rows, N, K, seed=N + K, top_k=top_k), dt, pad=len(rows) % 2)


@pytest.mark.parametrize("rows", [1, 4, 5, 16, 31, 40, 80, 130, 200, 300, 420, 700, 1100])
def test_rows_of_one_expert(int8, rows):
    c = Case((rows,), 192, 320, seed=rows, full=True)
    check_both(int8, c, "f32")


def test_workspace_of_two_graphs(int8):
    """Two captured calls that share a workspace, replayed in turn: counters of shared tiles are
    left as they were found."""
    cases = [Case((20,), 300, 6144, seed=1), Case((9, 12), 128, 4096, seed=2)]
    ws = workspace(int8, 64)
    graphs = []
    for c in cases:
        args = (c.mats(int8)[0], dev(c.xq), dev(c.xs), torch.empty((c.R, c.N), device="cuda"))
        rows = c.rows()
        int8.product(*args, ws, **rows)
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            int8.product(*args, ws, **rows)
        graphs.append((g, args, rows))
    for _ in range(3):
        for c, (g, args, _) in zip(cases, graphs):
            args[3].fill_(float("nan"))
            g.replay()
            y, e = c.expected()
            check(args[3], y, e, "f32")


def test_two_calls_at_once(int8):
    """Calls on two streams with workspaces of their own."""
    cases = [Case((700, 500), 300, 2048, seed=3), Case((3, 20), 500, 4096, seed=4)]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    outs = []
    for _ in range(4):
        outs = []
        for c, s in zip(cases, streams):
            with torch.cuda.stream(s):
                outs.append(run_product(int8, c, "f32"))
    torch.cuda.synchronize()
    for c, out in zip(cases, outs):
        y, e = c.expected()
        check(out, y, e, "f32")


# ---------------------------------------------------------------- beyond 32 bits
def codes(g, *shape):
    return torch.randint(-127, 128, shape, generator=g, device="cuda", dtype=torch.int8)


def check_exact(out, x, xs, w, ws):
    y, e = ref.product(*(t.cpu().numpy() for t in (x, xs, w, ws)))
    got = out.double().cpu().numpy()
    assert (np.abs(got - y) <= e + np.abs(y) * HALF_ULP["f32"] + TINY["f32"]).all()


@pytest.mark.parametrize("rows", [3, 30, 200, 2000])
def test_weights_beyond_32_bit_offsets(int8, rows):
    """The last of 34 experts of 128 MiB."""
    g = torch.Generator(device="cuda").manual_seed(rows)
    E, N, K = 34, 65536, 2048
    w = torch.zeros((E, N, K), dtype=torch.int8, device="cuda")
    w[-1] = codes(g, N, K)
    ws = torch.rand((E, N), generator=g, device="cuda") + 0.5
    x, xs = codes(g, rows, K), torch.rand(rows, generator=g, device="cuda") + 0.5
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[-1] = rows
    out = torch.empty((rows, N), device="cuda")
    int8.product(int8.Mat(w, ws), x, xs, out, workspace(int8, rows), off=off)
    n = slice(N - 300, N)
    r = slice(max(0, rows - 50), rows)
    check_exact(out[r, n], x[r], xs[r], w[-1, n], ws[-1, n])


@pytest.mark.parametrize("rows", [40, 900])
def test_rows_beyond_32_bit_offsets(int8, rows):
    """Activation rows past 4 GiB, and output rows 2 GiB apart."""
    g = torch.Generator(device="cuda").manual_seed(rows)
    n_x, N, K = 270000, 200, 16384
    x = torch.zeros((n_x, K), dtype=torch.int8, device="cuda")
    x[-rows:] = codes(g, rows, K)
    xs = torch.ones(n_x, device="cuda")
    w, ws = codes(g, 1, N, K), torch.rand((1, N), generator=g, device="cuda") / K
    perm = torch.arange(n_x - rows, n_x, dtype=torch.int32, device="cuda").flip(0).contiguous()
    wide = torch.empty((rows, 1 << 22 if rows > 100 else 1 << 26), dtype=torch.bfloat16,
                       device="cuda")
    out = wide[:, 7:7 + N]
    int8.product(int8.Mat(w, ws), x, xs, out, workspace(int8, rows),
                 off=torch.tensor([0, rows], dtype=torch.int32, device="cuda"), perm=perm)
    y, e = ref.product(x[-rows:].flip(0).cpu().numpy(), np.ones(rows, np.float32),
                       w[0].cpu().numpy(), ws[0].cpu().numpy())
    check(out, y, e, "bf16")


def test_quantiser_beyond_32_bit_offsets(int8):
    T, d = 270000, 16384
    x = torch.zeros((T, d), dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    x[-5:] = torch.randn((5, d), generator=g, device="cuda").bfloat16()
    q, s = torch.empty((T, d), dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
    int8.quantize(x, q, s)
    rq, rs = ref.quantize(x[-5:].float().cpu().numpy())
    assert np.array_equal(q[-5:].cpu().numpy(), rq) and np.array_equal(s[-5:].cpu().numpy(), rs)
    assert not q[:-5].any()
