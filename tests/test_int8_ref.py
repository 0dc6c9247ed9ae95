"""The int8 operators without a GPU: the reference's own pins and the refusals at the C ABI
and in the binding."""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

import int8_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 20  # an aligned address that nothing may touch


@pytest.fixture(scope="module")
def int8(cuda_built):
    from routed_expert_decode_gb300 import int8 as m

    m.lib()
    return m


def test_reference_quantiser():
    x = np.array([[0, 0, 0], [1, -127, 63.5], [2, np.nan, 1], [3, 1, -np.inf]], np.float32)
    q, s = ref.quantize(x)
    assert q.tolist() == [[0, 0, 0], [1, -127, 64], [0, 0, 0], [0, 0, 0]]  # 63.5: to even
    assert s[0] == np.float32(2.0 ** -100) / np.float32(127) and s[1] == 1
    assert np.isnan(s[2:]).all()
    # any finite row: the largest magnitude is 127, values come back within half a step
    rng = np.random.default_rng(0)
    x = (rng.standard_normal((50, 40)) * np.exp2(rng.integers(-90, 100, (50, 1)))).astype(np.float32)
    q, s = ref.quantize(x)
    assert (np.abs(q.astype(int)).max(1) == 127).all()
    assert (np.abs(q * s[:, None].astype(np.float64) - x) <= 0.5001 * s[:, None]).all()


def test_reference_bound_holds_for_plain_fp32():
    """A plain fp32 evaluation (in K order) stays inside the bound."""
    rng = np.random.default_rng(1)
    xq, wq = (rng.integers(-128, 128, (n, 4096)).astype(np.int8) for n in (5, 7))
    xs, ws = (rng.uniform(0.5, 2, n).astype(np.float32) for n in (5, 7))
    y, e = ref.product(xq, xs, wq, ws)
    acc = np.zeros((5, 7), np.float32)
    for k in range(0, 4096, 16):
        acc += (xq[:, k:k + 16].astype(np.int32) @ wq[:, k:k + 16].astype(np.int32).T)
    got = (acc * (xs[:, None] * ws[None, :])).astype(np.float32)
    assert (np.abs(got - y) <= e).all()


def test_struct_layouts_match_header(int8, tmp_path):
    src = tmp_path / "layout.c"
    src.write_text(r'''
#include <stdio.h>
#include <stddef.h>
#include "moe_int8.h"
int main(void) {
  printf("%zu %zu %zu %zu\n", sizeof(moe_int8_mat), sizeof(moe_int8_rows),
         offsetof(moe_int8_rows, off), offsetof(moe_int8_rows, top_k));
  return 0;
}
''')
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), str(src), "-o",
                    str(exe)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout
    assert [int(v) for v in out.split()] == [
        ctypes.sizeof(int8.Int8Mat), ctypes.sizeof(int8.Int8Rows), int8.Int8Rows.off.offset,
        int8.Int8Rows.top_k.offset]


def test_quantize_refusals(int8):
    L = int8.lib()
    ok = [FAKE, 1, 128, 4, 128, FAKE, FAKE, None]
    for i, v in ((0, None), (0, FAKE + 1), (1, 5), (2, 127), (4, 0), (4, 1 << 25), (5, None),
                 (6, None), (6, FAKE + 2), (3, (1 << 30) + 1)):
        a = list(ok)
        a[i] = v
        assert L.moe_int8_quantize(*a) == 1, (i, v)
    assert L.moe_int8_quantize(None, 1, 128, 0, 128, None, None, None) == 0  # no rows


def test_product_refusals(int8):
    L = int8.lib()
    need = int8.workspace_size(8)

    def call(mat=(FAKE, FAKE), E=2, N=64, K=64, x=None, out=FAKE, dt=0, ld=64, ws=FAKE, n=need,
             swiglu=False):
        xs = dict(q=FAKE, scale=FAKE, n=8, rows=8, off=FAKE, perm=FAKE, top_k=2)
        xs.update(x or {})
        m, r = int8.Int8Mat(*mat), int8.Int8Rows(**xs)
        mats = (ctypes.byref(m),) * (2 if swiglu else 1)
        f = L.moe_int8_swiglu if swiglu else L.moe_int8_product
        return f(*mats, E, N, K, ctypes.byref(r), out, dt, ld, ws, n, None)

    for swiglu in (False, True):
        for kw in (dict(mat=(None, FAKE)), dict(mat=(FAKE, None)), dict(mat=(FAKE, FAKE + 2)),
                   dict(E=0), dict(E=1025), dict(N=0), dict(K=0), dict(K=131072),
                   dict(x=dict(off=None)), dict(x=dict(q=None)), dict(x=dict(scale=FAKE + 1)),
                   dict(x=dict(off=FAKE + 1)), dict(x=dict(perm=FAKE + 2)), dict(x=dict(top_k=0)),
                   dict(x=dict(perm=None, n=7)), dict(x=dict(n=0)), dict(ws=None),
                   dict(ws=FAKE + 8), dict(out=None), dict(dt=7), dict(ld=63),
                   dict(out=FAKE + 2), dict(dt=1, out=FAKE + 1),
                   dict(x=dict(rows=1 << 30), N=1 << 20)):
            assert call(swiglu=swiglu, **kw) == 1, kw
        assert call(swiglu=swiglu, n=need - 1) == 3
        # no rows: nothing to do, and nothing is touched
        assert call(swiglu=swiglu, x=dict(rows=0), ws=None) == 0


def test_python_refusals(int8):
    cpu = torch.zeros((4, 64))
    with pytest.raises(ValueError):
        int8.quantize(cpu, cpu, cpu)
    with pytest.raises(ValueError):
        int8.Mat(torch.zeros((2, 64, 64), dtype=torch.int8), torch.zeros((2, 64)))
    with pytest.raises(ValueError):
        int8.product(None, cpu, cpu, cpu, cpu)
    with pytest.raises(ValueError):
        int8.swiglu(None, None, cpu, cpu, cpu, cpu)
