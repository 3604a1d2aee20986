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
               dict(counts=None), dict(sums=None), dict(loss=None), dict(n=10), dict(T=100000, n=100)):
        assert f(**kw) == sat.FP8Q_ERR_ARG, kw
    for kw in (dict(T=-1), dict(T=1 << 40)):
        assert f(**kw) == sat.FP8Q_ERR_SHAPE, kw
    for kw in (dict(logits=None), dict(idx=None), dict(w=None), dict(ws=None)):
        assert f(**kw) == sat.FP8Q_ERR_NULL, kw
    for kw in (dict(logits=M8), dict(idx=M2), dict(w=M2), dict(counts=M2), dict(ws=M8), dict(flags=1, bias=M2)):
        assert f(**kw) == sat.FP8Q_ERR_ALIGN, kw
    assert f(T=0, logits=None, idx=None, w=None, counts=None, sums=None, loss=None, ws=None) == sat.FP8Q_OK
    assert sat.fp8q_router_workspace_bytes(-1, 8) == 0 and sat.fp8q_router_workspace_bytes(4, 2000) == 0
    assert sat.fp8q_router_workspace_bytes(0, 32) >= 16 and sat.fp8q_router_workspace_bytes(1 << 20, 32) >= 32 * 8


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
    def f(g=A, u=A, w=None, rows=128, cols=256, q=A, sf=A, gq=A, gsf=A, uq=A, usf=A):
        return L.fp8q_swiglu_quant_stash(g, u, w, rows, cols, q, sf, gq, gsf, uq, usf, None)

    for kw in (dict(rows=-1), dict(cols=100), dict(rows=1 << 31)):
        assert f(**kw) == sat.FP8Q_ERR_SHAPE, kw
    for k in ("g", "u", "q", "sf", "gq", "gsf", "uq", "usf"):
        assert f(**{k: None}) == sat.FP8Q_ERR_NULL, k
    for kw in (dict(g=M8), dict(u=M8), dict(gq=M8), dict(uq=M8), dict(q=M8), dict(w=M2)):
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


def test_mxfp4_quantize_refusals(L):
    f = L.fp8q_quantize_rowwise_mxfp4
    assert f(A, 4, 96, A, A, None) == sat.FP8Q_ERR_SHAPE
    assert f(A, -1, 128, A, A, None) == sat.FP8Q_ERR_SHAPE
    assert f(None, 4, 128, A, A, None) == sat.FP8Q_ERR_NULL
    assert f(A, 4, 128, A, None, None) == sat.FP8Q_ERR_NULL
    assert f(M8, 4, 128, A, A, None) == sat.FP8Q_ERR_ALIGN
    assert f(A, 4, 128, A, M8, None) == sat.FP8Q_ERR_ALIGN
    assert f(None, 0, 128, None, None, None) == sat.FP8Q_OK
    assert sat.fp8q_mxfp4_sf_bytes(1, 128) == 512 and sat.fp8q_mxfp4_sf_bytes(129, 384) == 2 * 3 * 512
    assert sat.fp8q_mxfp4_sf_bytes(0, 128) == 0


def test_mxfp4_permute_refusals(L):
    def f(x=A, T=8, H=256, idx=A, K=2, E=4, align=128, q=A, sf=A, cap=1 << 20, off=A, rmap=A, ws=A, n=1 << 30):
        return L.fp8q_permute_pad_mxfp4(x, T, H, idx, K, E, align, q, sf, cap, off, rmap, ws, n, None)

    for kw in (dict(T=-1), dict(H=100), dict(T=1 << 40)):
        assert f(**kw) == sat.FP8Q_ERR_SHAPE, kw
    for kw in (dict(K=0), dict(K=65), dict(E=0), dict(E=5000), dict(align=0), dict(cap=100), dict(n=4)):
        assert f(**kw) == sat.FP8Q_ERR_ARG, kw
    for k in ("x", "idx", "q", "sf", "off", "rmap", "ws"):
        assert f(**{k: None}) == sat.FP8Q_ERR_NULL, k
    for k in ("x", "q", "sf", "ws"):
        assert f(**{k: M8}) == sat.FP8Q_ERR_ALIGN, k
    for k in ("idx", "off", "rmap"):
        assert f(**{k: M2}) == sat.FP8Q_ERR_ALIGN, k


def test_mxfp4_matmul_refusals(L):
    def f(aq=A, asf=A, m=4, bq=A, bsf=A, n=128, k=256, off=None, G=1, out=A):
        return L.fp8q_matmul_mxfp4(aq, asf, m, bq, bsf, n, k, off, G, out, None)

    for kw in (dict(m=-1), dict(n=-1), dict(k=100), dict(k=0), dict(k=(1 << 24) + 128), dict(m=1 << 31), dict(off=A, n=100),
               dict(off=A, n=1 << 24, G=200)):
        assert f(**kw) == sat.FP8Q_ERR_SHAPE, kw
    for kw in (dict(G=0), dict(G=2), dict(off=A, G=0)):
        assert f(**kw) == sat.FP8Q_ERR_ARG, kw
    for k in ("aq", "asf", "bq", "bsf", "out"):
        assert f(**{k: None}) == sat.FP8Q_ERR_NULL, k
        assert f(**{k: M8}) == sat.FP8Q_ERR_ALIGN, k
    assert f(off=M2) == sat.FP8Q_ERR_ALIGN
    assert f(m=0, aq=None) == sat.FP8Q_OK and f(n=0, out=None) == sat.FP8Q_OK


def test_reference_codes_round_trip():
    from moe_reference import E4M3, decode4, decode8, encode4, encode8, tile_scales
    rng = np.random.default_rng(1)
    q = rng.integers(0, 256, (5, 64), dtype=np.uint8)
    q[:, ::16] = 0x77  # the largest code in every tile: the scale is then the rule's own
    sf = rng.integers(60, 180, (5, 4)).astype(np.uint8)
    rq, rsf = encode4(decode4(q, sf))
    assert np.array_equal(rq, q) and np.array_equal(rsf, sf)
    c = rng.integers(0, 126, (3, 256), dtype=np.uint8)
    c[:, ::128] = 126
    s8 = rng.integers(60, 180, (3, 2)).astype(np.uint8)
    r8, rs8 = encode8(decode8(c, s8))
    assert np.array_equal(r8, c) and np.array_equal(rs8, s8) and E4M3[126] == 448
    assert sorted(tile_scales(np.arange(128 * 4, dtype=np.uint32).reshape(128, 4) % 251)) == sorted(np.arange(512) % 251)
    import torch
    t = torch.from_numpy(rng.integers(0, 255, (200, 12), dtype=np.uint8))
    assert np.array_equal(sat.mxfp4_tile_scales(t).numpy(), tile_scales(t.numpy()))
