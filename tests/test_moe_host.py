"""Refusals of the router, checkpoint and MXFP4 entry points, made on the host before any
CUDA call (fake addresses, never dereferenced), and the 64-bit reference's own identities."""
import numpy as np
import pytest

import scaling_aware_transpose_b200 as sat
from moe_reference import router, router_bwd, swiglu_bwd
from scaling_aware_transpose_b200 import build as lib_build

A, M8, M2 = 0x10000, 0x10008, 0x10002


@pytest.fixture(scope="module")
def L():
    lib_build.build()
    return sat.lib()


def test_router_refusals(L):
    def f(logits=A, T=4, E=32, flags=0, bias=None, mask=None, K=8, idx=A, w=A, counts=A, sums=A, loss=A, ws=A, n=1 << 20):
        return L.fp8q_router_topk(logits, T, E, flags, bias, mask, K, 1.0, 1.0, idx, w, counts, sums, loss, ws, n, None)

    for kw in (dict(E=0), dict(E=1025), dict(K=0), dict(K=33), dict(E=1024, K=65), dict(flags=8), dict(bias=A),
               dict(counts=None), dict(sums=None), dict(loss=None), dict(n=100)):
        assert f(**kw) == sat.FP8Q_ERR_ARG, kw
    for kw in (dict(T=-1), dict(T=1 << 40)):
        assert f(**kw) == sat.FP8Q_ERR_SHAPE, kw
    for kw in (dict(logits=None), dict(idx=None), dict(w=None), dict(ws=None)):
        assert f(**kw) == sat.FP8Q_ERR_NULL, kw
    for kw in (dict(logits=M8), dict(idx=M2), dict(w=M2), dict(counts=M2), dict(ws=M8), dict(flags=1, bias=M2)):
        assert f(**kw) == sat.FP8Q_ERR_ALIGN, kw
    assert f(T=0, logits=None, idx=None, w=None, counts=None, sums=None, loss=None, ws=None) == sat.FP8Q_OK
    assert sat.fp8q_router_workspace_bytes(-1, 8) == 0 and sat.fp8q_router_workspace_bytes(4, 2000) == 0
    assert sat.fp8q_router_workspace_bytes(0, 32) >= 32 * 8


def test_router_bwd_refusals(L):
    def f(logits=A, T=4, E=32, flags=0, K=8, idx=A, gw=A, rmap=None, rows=0, counts=A, gl=A, out=A):
        return L.fp8q_router_topk_bwd(logits, T, E, flags, None, K, 1.0, idx, gw, rmap, rows, counts, 1.0, gl, out, None)

    for kw in (dict(E=1025), dict(K=33), dict(flags=16), dict(gw=None, rmap=A), dict(rows=-1), dict(rows=1 << 31)):
        assert f(**kw) == sat.FP8Q_ERR_ARG, kw
    assert f(T=-1) == sat.FP8Q_ERR_SHAPE
    for kw in (dict(logits=None), dict(idx=None), dict(counts=None), dict(out=None)):
        assert f(**kw) == sat.FP8Q_ERR_NULL, kw
    for kw in (dict(logits=M8), dict(out=M8), dict(gw=M2), dict(rmap=M2, rows=9), dict(gl=M2)):
        assert f(**kw) == sat.FP8Q_ERR_ALIGN, kw
    assert f(T=0, logits=None, out=None) == sat.FP8Q_OK


def test_row_weights_refusals(L):
    f = L.fp8q_permute_row_weights
    assert f(A, A, -1, 8, A, None) == sat.FP8Q_ERR_SHAPE
    assert f(A, A, 8, 1 << 31, A, None) == sat.FP8Q_ERR_SHAPE
    assert f(None, A, 8, 8, A, None) == sat.FP8Q_ERR_NULL
    assert f(A, A, 8, 8, None, None) == sat.FP8Q_ERR_NULL
    assert f(M2, A, 8, 8, A, None) == sat.FP8Q_ERR_ALIGN
    assert f(None, None, 0, 0, None, None) == sat.FP8Q_OK


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
def test_reference_gradient_against_differences(sigmoid, renorm):
    """The 64-bit gradient the kernels are held to, against central differences."""
    rng = np.random.default_rng(3)
    T, E, K, h = 3, 7, 2, 1e-6
    l = rng.standard_normal((T, E))
    r = router(l, K, sigmoid, renorm, loss_coef=0.5)
    gw = rng.standard_normal((T, K))

    def value(x):
        q = router(x, K, sigmoid, renorm, loss_coef=0.5)
        pk = np.take_along_axis(q["p"], r["idx"], 1)
        w = pk / (pk.sum(1, keepdims=True) + 1e-20) if renorm else pk
        return (gw * w).sum() + 0.9 * r["coef"] * (r["counts"] * q["h"].sum(0)).sum()

    got, _ = router_bwd(l, r["idx"], gw, r["counts"], 0.9, sigmoid, renorm, loss_coef=0.5)
    for t in range(T):
        for e in range(E):
            a, b = l.copy(), l.copy()
            a[t, e] += h
            b[t, e] -= h
            assert abs((value(a) - value(b)) / (2 * h) - got[t, e]) < 1e-8


def test_swiglu_stash_refusals(L):
    def f(g=A, u=A, w=None, rows=128, cols=256, q=A, sf=A, qt=None, sft=None, gq=A, gsf=A, uq=A, usf=A):
        return L.fp8q_swiglu_quant_stash(g, u, w, rows, cols, q, sf, qt, sft, gq, gsf, uq, usf, None)

    for kw in (dict(rows=-1), dict(cols=100), dict(rows=1 << 31), dict(rows=100, qt=A, sft=A)):
        assert f(**kw) == sat.FP8Q_ERR_SHAPE, kw
    for kw in (dict(qt=A), dict(sft=A)):
        assert f(**kw) == sat.FP8Q_ERR_ARG, kw
    for k in ("g", "u", "q", "sf", "gq", "gsf", "uq", "usf"):
        assert f(**{k: None}) == sat.FP8Q_ERR_NULL, k
    for kw in (dict(g=M8), dict(u=M8), dict(gq=M8), dict(uq=M8), dict(q=M8), dict(w=M2), dict(qt=M2, sft=A)):
        assert f(**kw) == sat.FP8Q_ERR_ALIGN, kw
    assert f(rows=0, g=None) == sat.FP8Q_OK and f(cols=0, gq=None) == sat.FP8Q_OK


@pytest.mark.parametrize("quant", [False, True])
def test_swiglu_bwd_refusals(L, quant):
    def f(gq=A, gsf=A, uq=A, usf=A, w=None, dy=A, rows=4, cols=256, dw=None, yq=None, ysf=None, **o):
        dg, du, dgsf, dusf = (o.get(k, A) for k in ("dg", "du", "dgsf", "dusf"))
        if quant:
            return L.fp8q_swiglu_bwd_quant(gq, gsf, uq, usf, w, dy, rows, cols, dg, dgsf, du, dusf, yq, ysf, dw, None)
        return L.fp8q_swiglu_bwd(gq, gsf, uq, usf, w, dy, rows, cols, dg, du, dw, None)

    for kw in (dict(rows=-1), dict(cols=130), dict(cols=-128), dict(rows=1 << 31)):
        assert f(**kw) == sat.FP8Q_ERR_SHAPE, kw
    assert f(dw=A) == sat.FP8Q_ERR_ARG                       # a gradient of weights that were not given
    for k in ("gq", "gsf", "uq", "usf", "dy", "dg", "du") + (("dgsf", "dusf") if quant else ()):
        assert f(**{k: None}) == sat.FP8Q_ERR_NULL, k
    for k in ("gq", "uq", "dy", "dg", "du"):
        assert f(**{k: M8}) == sat.FP8Q_ERR_ALIGN, k
    assert f(w=M2) == sat.FP8Q_ERR_ALIGN
    if quant:
        assert f(yq=A) == sat.FP8Q_ERR_ARG and f(ysf=A) == sat.FP8Q_ERR_ARG
        assert f(yq=M8, ysf=A) == sat.FP8Q_ERR_ALIGN
    assert f(rows=0, gq=None) == sat.FP8Q_OK


def test_reference_swiglu_gradient_against_differences():
    rng = np.random.default_rng(5)
    g, u, dy, w = rng.standard_normal((3, 8)) * 3, rng.standard_normal((3, 8)), rng.standard_normal((3, 8)), rng.random(3)
    r = swiglu_bwd(g, u, dy, w)
    y = lambda g, u, w: g / (1 + np.exp(-g)) * u * w[:, None]  # noqa: E731
    h = 1e-6
    assert np.allclose((y(g + h, u, w) - y(g - h, u, w)) / (2 * h) * dy, r["dg"], atol=1e-8)
    assert np.allclose((y(g, u + h, w) - y(g, u - h, w)) / (2 * h) * dy, r["du"], atol=1e-8)
    assert np.allclose(((y(g, u, w + h) - y(g, u, w - h)) / (2 * h) * dy).sum(1), r["dw"], atol=1e-7)
