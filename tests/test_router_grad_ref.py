"""The router's gradients without a GPU: the reference against differences, and the refusals
at the C ABI and in the binding."""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

import fp8_ref
import router_grad_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 20  # an aligned address that nothing may touch


@pytest.fixture(scope="module")
def rg(cuda_built):
    from routed_expert_decode_gb300 import router_grad as m

    m.lib()
    return m


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("fn", [0, 1, 2])
def test_reference_gradient_against_differences(fn, renorm):
    """Central differences in 64 bits: step^2 of third derivatives below ten, and 2^-53 over
    the step of values around one."""
    T, E, k, S, s, coef, dloss, step = 14, 9, 3, 3, 2.5, 0.7, 1.3, 2.0 ** -13
    rng = np.random.default_rng(4)
    l = rng.standard_normal((T, E))
    idx = np.argsort(rng.random((T, E)), axis=1)[:, :k]
    idx[2, 1], idx[3, 2] = -1, idx[3, 0]
    seq, live = np.array([0, 5, 5, 12]), rng.random(T) > 0.3
    dw = rng.standard_normal((T, k))

    def value(l):
        _, p = fp8_ref.score(l, fn)
        ok = (idx >= 0) & (idx < E)
        pj = np.where(ok, np.take_along_axis(p, np.where(ok, idx, 0), 1), 0.0)
        w = s * pj / pj.sum(1, keepdims=True) if renorm else s * pj
        return (w * dw).sum() + dloss * ref.balance(l, idx, k, fn, S, seq, live, coef)[3]

    counts, tokens, *_ = ref.balance(l, idx, k, fn, S, seq, live, coef)
    assert counts[1].sum() == 0 and tokens[1] == 0
    g, bound = ref.route_backward(l, idx, k, fn, renorm, s, dw, counts, tokens, dloss, S, seq, live,
                                  coef)
    # below 300 roundings (3 * 70 + 66) of terms up to 2.5 * (2 * 3.5): 300 * 2^-24 * 18
    assert (bound <= 4e-4).all()
    for t in range(T):
        for e in range(E):
            up, down = l.copy(), l.copy()
            up[t, e] += step
            down[t, e] -= step
            d = (value(up) - value(down)) / (2 * step)
            assert abs(d - g[t, e]) <= 10 * step ** 2 + 1e-10, (t, e)


def test_reference_combine_gradient():
    rng = np.random.default_rng(5)
    T, k, R, d = 4, 3, 15, 6
    dy, o, w = rng.standard_normal((T, d)), rng.standard_normal((R, d)), rng.random((T, k))
    pos = rng.permutation(R)[:T * k].reshape(T, k)
    pos[1, 1] = -1
    dw, _, do, _ = ref.combine_backward(dy, o, w, pos)

    def value(o, w):
        return sum((dy[t] * w[t, j] * o[pos[t, j]]).sum() for t in range(T) for j in range(k)
                   if pos[t, j] >= 0)

    base = value(o, w)
    for t in range(T):
        for j in range(k):
            up = w.copy()
            up[t, j] += 1  # linear: a whole step is exact
            assert abs(value(o, up) - base - dw[t, j]) < 1e-12
    for r in range(R):
        for c in range(d):
            up = o.copy()
            up[r, c] += 1
            want = 0.0 if np.isnan(do[r, c]) else do[r, c]
            assert abs(value(up, w) - base - want) < 1e-12


def test_struct_layout_matches_header(rg, tmp_path):
    src = tmp_path / "layout.c"
    src.write_text(r'''
#include <stdio.h>
#include <stddef.h>
#include "moe_router_grad.h"
int main(void) {
  printf("%zu %zu %zu\n", sizeof(moe_tokens), offsetof(moe_tokens, seq), offsetof(moe_tokens, live));
  return 0;
}
''')
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), str(src), "-o",
                    str(exe)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout
    assert [int(v) for v in out.split()] == [ctypes.sizeof(rg.MoeTokens), rg.MoeTokens.seq.offset,
                                             rg.MoeTokens.live.offset]


def router(E=64, k=4, **kw):
    from routed_expert_decode_gb300 import fp8

    return fp8.make_router(E, k, **kw)


def test_balance_refusals(rg):
    r = router()
    need = rg.workspace_size(r, 10, 2)

    def call(r=r, logits=FAKE, dt=0, ld=64, idx=FAKE, tokens=None, count=FAKE, n=FAKE, prob=FAKE,
             loss=FAKE, ws=FAKE, size=need):
        t = dict(T=10, S=2, seq=FAKE, live=FAKE + 1)
        t.update(tokens or {})
        return rg.lib().moe_balance(ctypes.byref(r), logits, dt, ld, idx,
                                    ctypes.byref(rg.MoeTokens(**t)), 1.0, count, n, prob, loss, ws,
                                    size, None)

    for kw in (dict(r=router(64, 0)), dict(r=router(64, 65)), dict(logits=None),
               dict(logits=FAKE + 2), dict(dt=4), dict(ld=63), dict(idx=None), dict(idx=FAKE + 1),
               dict(tokens=dict(S=0)), dict(tokens=dict(S=65536)), dict(tokens=dict(seq=None)),
               dict(tokens=dict(seq=FAKE + 2)), dict(tokens=dict(T=1 << 29)), dict(count=None),
               dict(n=None), dict(prob=None), dict(loss=None), dict(loss=FAKE + 2), dict(ws=None),
               dict(ws=FAKE + 128)):
        assert call(**kw) == 1, kw
    assert call(size=need - 1) == 3
    assert rg.workspace_size(router(64, 65), 10) == 0


def test_route_backward_refusals(rg):
    def call(r=router(), logits=FAKE, dt=0, ld=64, idx=FAKE, dw=FAKE, tokens=None, count=FAKE,
             n=FAKE, dloss=FAKE, out=FAKE, odt=0, ldd=64):
        t = dict(T=10, S=2, seq=FAKE, live=FAKE + 1)
        t.update(tokens or {})
        return rg.lib().moe_route_backward(ctypes.byref(r), logits, dt, ld, idx, dw,
                                           ctypes.byref(rg.MoeTokens(**t)), count, n, dloss, 1.0,
                                           out, odt, ldd, None)

    for kw in (dict(r=router(64, 65)), dict(logits=None), dict(logits=FAKE + 2), dict(dt=4),
               dict(ld=63), dict(idx=None), dict(idx=FAKE + 1), dict(dw=FAKE + 2), dict(n=None),
               dict(count=FAKE + 1), dict(dloss=FAKE + 1), dict(out=None), dict(out=FAKE + 2),
               dict(odt=3), dict(ldd=63), dict(tokens=dict(S=0)), dict(tokens=dict(seq=None)),
               dict(tokens=dict(T=1 << 29)), dict(count=None, tokens=dict(T=1 << 29))):
        assert call(**kw) == 1, kw
    assert call(tokens=dict(T=0), logits=None, out=None) == 0


def test_combine_backward_refusals(rg):
    ok = [FAKE, 1, 128, FAKE, 1, 128, 16, FAKE, FAKE, 4, 4, 128, FAKE, FAKE, 128, None]
    for i, v in ((0, None), (0, FAKE + 1), (1, 3), (2, 127), (3, None), (4, 9), (5, 100),
                 (7, None), (7, FAKE + 2), (8, None), (8, FAKE + 1), (10, 0), (10, 33), (11, 0),
                 (12, FAKE + 2), (13, FAKE + 1), (14, 127), (9, 1 << 29)):
        a = list(ok)
        a[i] = v
        assert rg.lib().moe_combine_backward(*a) == 1, (i, v)
    for change in ({9: 0}, {12: None, 13: None}):
        a = list(ok)
        for i, v in change.items():
            a[i] = v
        assert rg.lib().moe_combine_backward(*a) == 0


def test_python_refusals(rg):
    cpu = torch.zeros((4, 64))
    with pytest.raises(ValueError):
        rg.balance(router(), cpu, cpu, cpu, cpu, cpu, cpu, cpu)
    with pytest.raises(ValueError):
        rg.route_backward(router(), cpu, cpu, cpu)
    with pytest.raises(ValueError):
        rg.combine_backward(cpu, cpu, cpu, cpu)
