"""The 64-bit reference of the fp8 operators against closed forms, and the argument
checks of their C ABI, without a GPU."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

import fp8_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_e4m3_values_and_encoding():
    torch = pytest.importorskip("torch")
    codes = np.arange(256, dtype=np.uint8)
    t = torch.from_numpy(codes.copy()).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(np.isnan(t), np.isnan(ref.VALUES))
    assert np.array_equal(t[~np.isnan(t)], ref.VALUES[~np.isnan(t)])
    fin = ~np.isnan(ref.VALUES)
    assert np.array_equal(ref.e4m3_encode(ref.VALUES[fin]), codes[fin])
    # halfway points go to the even code, beyond the range saturates
    pos = ref.VALUES[:127]
    mid = (pos[:-1] + pos[1:]) / 2
    even = np.where(np.arange(126) % 2 == 0, np.arange(126), np.arange(1, 127))
    assert np.array_equal(ref.e4m3_encode(mid), even)
    assert np.array_equal(ref.e4m3_encode([1e9, -1e9, np.inf]), [0x7E, 0xFE, 0x7E])


def test_quantize_closed_forms():
    x = np.zeros((3, 200), np.float32)
    x[0, 5], x[0, 130] = 448.0, -7.0
    x[1, :128] = 2.0 ** -149
    q, s, _ = ref.quantize(x)
    assert s[0, 0] == 1.0 and q[0, 5] == 0x7E
    assert q[0, 130] == 0xFE and s[0, 1] == np.float32(7.0) / np.float32(448.0)
    # below the smallest maximum, and empty blocks: code 0 under the smallest scale
    assert not q[1:].any() and (s[1:] == np.float32(2.0 ** -100) / np.float32(448.0)).all()


def test_route_reference_groups_and_ties():
    l = np.zeros((1, 8))
    idx, w, _ = ref.route(l, None, 3, 1, 1, 0, True, True, 2.5)
    assert idx.tolist() == [[0, 1, 2]] and np.allclose(w, 2.5 / 3)
    l = np.array([[0.0, 5.0, 0.0, 0.0, 4.0, 4.5, 0.0, 0.0]])
    assert ref.route(l, None, 2, 4, 1, 0, False, True, 1.0)[0].tolist() == [[1, 0]]
    assert ref.route(l, None, 2, 4, 1, 0, True, True, 1.0)[0].tolist() == [[5, 4]]
    w = ref.route(np.full((1, 4), -np.inf), None, 2, 1, 1, 2, False, True, 1.0)[1]
    assert (w == 0).all()


# ---------------------------------------------------------------- C ABI
@pytest.fixture(scope="module")
def fp8(cuda_built):
    from routed_expert_decode_gb300 import fp8 as m

    m.lib()
    return m


def test_struct_layouts_match_header(fp8, tmp_path):
    src = tmp_path / "layout.c"
    src.write_text(r'''
#include <stdio.h>
#include <stddef.h>
#include "moe_fp8.h"
int main(void) {
  printf("%zu %zu %zu %zu %zu\n", sizeof(moe_router), offsetof(moe_router, s),
         sizeof(moe_fp8_mat), sizeof(moe_fp8_rows), offsetof(moe_fp8_rows, top_k));
  return 0;
}
''')
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), str(src), "-o",
                    str(exe)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout
    assert [int(v) for v in out.split()] == [
        ctypes.sizeof(fp8.MoeRouter), fp8.MoeRouter.s.offset, ctypes.sizeof(fp8.Fp8Mat),
        ctypes.sizeof(fp8.Fp8Rows), fp8.Fp8Rows.top_k.offset]


FAKE = 1 << 22  # never dereferenced: every call below is refused on the host


@pytest.mark.parametrize("bad", [
    dict(n_expert=0), dict(n_expert=1025), dict(top_k=0), dict(top_k=33, n_expert=64),
    dict(top_k=300), dict(n_group=7), dict(n_group=0), dict(n_group=64),
    dict(topk_group=0), dict(n_group=8, topk_group=9), dict(n_group=64, n_expert=64),
    dict(n_expert=16, n_group=8, topk_group=2, top_k=5), dict(score=3),
    dict(group_score=2), dict(s=float("nan"))])
def test_router_refusals(fp8, bad):
    kw = dict(n_expert=256, top_k=8)
    kw.update(bad)
    r = fp8.make_router(**kw)
    assert fp8.group_route_workspace_size(r, 4) == 0
    st = fp8.lib().moe_group_route(ctypes.byref(r), FAKE, 0, 1024, None, 4, FAKE, FAKE, FAKE, FAKE,
                                   FAKE, FAKE, 1 << 30, None)
    assert st == 1


def test_router_argument_refusals(fp8):
    r = fp8.make_router(64, 4)
    need = fp8.group_route_workspace_size(r, 4)
    assert need > 0

    def call(**kw):
        a = dict(logits=FAKE, dt=0, ld=64, bias=FAKE, T=4, idx=FAKE, w=FAKE, off=FAKE, perm=FAKE,
                 pos=FAKE, ws=FAKE, n=need)
        a.update(kw)
        return fp8.lib().moe_group_route(ctypes.byref(r), a["logits"], a["dt"], a["ld"], a["bias"],
                                         a["T"], a["idx"], a["w"], a["off"], a["perm"], a["pos"],
                                         a["ws"], a["n"], None)

    for kw in (dict(logits=None), dict(logits=FAKE + 2), dict(dt=1, logits=FAKE + 1), dict(dt=3),
               dict(ld=63), dict(bias=FAKE + 1), dict(idx=None), dict(w=None), dict(off=None),
               dict(perm=None), dict(pos=FAKE + 2), dict(ws=None), dict(ws=FAKE + 128),
               dict(T=1 << 29)):
        assert call(**kw) == 1, kw
    assert call(n=need - 1) == 3


def test_quantize_and_combine_refusals(fp8):
    L = fp8.lib()
    q = [FAKE, 1, 128, 4, 128, FAKE, FAKE, None]
    for i, v in ((0, None), (0, FAKE + 1), (1, 5), (2, 127), (4, 0), (4, 1 << 25), (5, None),
                 (6, None), (6, FAKE + 2)):
        a = list(q)
        a[i] = v
        assert L.moe_fp8_quantize(*a) == 1, (i, v)
    c = [FAKE, 1, 128, 16, FAKE, FAKE, 4, 4, 128, FAKE, 128, FAKE, 1, 128, None]
    for i, v in ((0, None), (1, 3), (2, 100), (4, None), (5, None), (5, FAKE + 1), (7, 0), (7, 33),
                 (8, 0), (10, 1), (11, None), (11, FAKE + 1), (12, 9), (13, 127)):
        a = list(c)
        a[i] = v
        assert L.moe_fp8_combine(*a) == 1, (i, v)


def test_product_refusals(fp8):
    L = fp8.lib()
    need = fp8.workspace_size(8)

    def call(mat=(FAKE, FAKE), E=2, N=64, K=64, x=None, out=FAKE, dt=0, ld=64, ws=FAKE, n=need,
             swiglu=False):
        xs = dict(q=FAKE, scale=FAKE, n=8, rows=8, off=FAKE, perm=FAKE, top_k=2)
        xs.update(x or {})
        m, r = fp8.Fp8Mat(*mat), fp8.Fp8Rows(**xs)
        if swiglu:
            return L.moe_fp8_swiglu(ctypes.byref(m), ctypes.byref(m), E, N, K, ctypes.byref(r), out,
                                    FAKE if ld else None, ws, n, None)
        return L.moe_fp8_product(ctypes.byref(m), E, N, K, ctypes.byref(r), out, dt, ld, ws, n, None)

    for swiglu in (False, True):
        for kw in (dict(mat=(None, FAKE)), dict(mat=(FAKE, None)), dict(mat=(FAKE, FAKE + 2)),
                   dict(E=0), dict(E=1025), dict(N=0), dict(K=0), dict(x=dict(off=None)),
                   dict(x=dict(q=None)), dict(x=dict(scale=FAKE + 1)), dict(x=dict(off=FAKE + 1)),
                   dict(x=dict(perm=FAKE + 2)), dict(x=dict(top_k=0)),
                   dict(x=dict(perm=None, n=7)), dict(ws=None), dict(ws=FAKE + 8), dict(out=None),
                   dict(x=dict(rows=1 << 30), N=1 << 20)):
            assert call(swiglu=swiglu, **kw) == 1, kw
        assert call(swiglu=swiglu, n=need - 1) == 3
        # no rows: nothing to do, and nothing is touched
        assert call(swiglu=swiglu, x=dict(rows=0), ws=None) == 0
    assert call(dt=7) == 1 and call(ld=63) == 1 and call(out=FAKE + 2) == 1
    assert call(swiglu=True, ld=0) == 1


def test_workspace_grows_with_the_tiles(fp8):
    """A split tile's share holds 256 columns of fp32 for each row of its tile, two
    shares a CTA: the sizes behind the fixed head step with the tile rows."""
    ctas = (fp8.workspace_size(64) - fp8.workspace_size(1)) // (2 * 32 * 1024)
    assert ctas >= 1
    for rows, tile in ((1, 32), (24, 32), (25, 64), (64, 64), (65, 96), (96, 96), (97, 128),
                       (128, 128), (10 ** 6, 128)):
        assert fp8.workspace_size(rows) - fp8.workspace_size(1) == 2 * ctas * 1024 * (tile - 32)


def test_python_refusals(fp8):
    import torch

    cpu = torch.zeros((4, 64))
    with pytest.raises(ValueError):
        fp8.quantize(cpu, cpu, cpu)
    with pytest.raises(ValueError):
        fp8.Mat(torch.zeros((2, 64, 64), dtype=torch.uint8), torch.zeros((2, 1, 1)))
    with pytest.raises(ValueError):
        fp8.group_route(fp8.make_router(32, 2), cpu, None, cpu, cpu, cpu, cpu, cpu, cpu)
