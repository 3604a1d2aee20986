"""SwiGLU with 8-bit checkpoints and its backward: the forward byte for byte against the
library's own SwiGLU and quantizer, the backward against plain 64-bit formulas with error
bounds derived in moe_reference.swiglu_bwd (plus half a step of the output's type)."""
import numpy as np
import pytest
import torch

import scaling_aware_transpose_b200 as sat
from gpu_helpers import device_status_ok
from moe_reference import E4M3, U_BF16, decode8, encode8, swiglu_bwd

pytestmark = pytest.mark.gpu


def normal(rows, cols, seed, sigma=1.0, row_sigma=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((rows, cols), generator=g) * torch.exp(row_sigma * torch.randn((rows, 1), generator=g))
    return (x * sigma).to(torch.bfloat16)


@pytest.mark.parametrize("rows,cols", [(1, 128), (3, 384), (130, 640), (128, 2048), (256, 4224), (1000, 128)])
def test_forward_keeps_the_plain_results(rows, cols):
    gate, up = normal(rows, cols, rows + cols).cuda(), normal(rows, cols, rows + cols + 1).cuda()
    gate[0, :128] = 0
    q, sf, gq, gsf, uq, usf = sat.swiglu_quant_stash(gate, up)
    for got, want in zip((q, sf), sat.swiglu_quant(gate, up, transposed=False)):
        assert torch.equal(got, want)
    for got, want in zip((gq, gsf, uq, usf), (*sat.quantize_rowwise(gate), *sat.quantize_rowwise(up))):
        assert torch.equal(got, want)
    out = [torch.full((t.shape[0] + 3, t.shape[1]), 0xEE, dtype=torch.uint8, device="cuda") for t in (q, sf, q, sf, q, sf)]
    sat.fp8q_swiglu_quant_stash(gate, up, None, rows, cols, *out)
    assert all(torch.equal(a[:rows], b) and (a[rows:] == 0xEE).all() for a, b in zip(out, (q, sf, gq, gsf, uq, usf)))
    device_status_ok()


@pytest.mark.parametrize("rows,cols", [(1, 128), (37, 1408), (300, 2048)])
def test_forward_row_weights(rows, cols):
    """y is the library's fp32 silu(gate) * up, times the weight in fp32, then quantized."""
    gate, up = normal(rows, cols, 1).cuda(), normal(rows, cols, 2).cuda()
    w = torch.randn(rows, generator=torch.Generator().manual_seed(3)).cuda()
    w[0] = 0.0 if rows > 1 else w[0]
    q, sf, gq, _, _, usf = sat.swiglu_quant_stash(gate, up, row_weights=w)
    y = torch.empty((rows, cols), device="cuda")
    sat.fp8q_debug_swiglu_spec(gate.float(), up.float(), rows * cols, y)
    eq, esf = encode8((y * w[:, None]).double().cpu().numpy())
    assert np.array_equal(sf.cpu().numpy(), esf)
    assert np.array_equal(q.cpu().numpy(), eq)
    assert torch.equal(gq, sat.quantize_rowwise(gate)[0]) and torch.equal(usf, sat.quantize_rowwise(up)[1])


def near(got, want, tol, what):
    off = np.abs(np.asarray(got, np.float64) - want)
    bad = ~(off <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {np.nanmax(off)} at {np.argwhere(bad)[:3].tolist()}"


def near_pair(q, sf, want, tol, what):
    """A quantized pair: a scale the rule allows for some value within the tolerance, and
    codes within half a step of the values."""
    q, sf = q.cpu().numpy(), sf.cpu().numpy()
    rows, cols = q.shape
    e = sf.astype(np.float64) - 127
    t, s = np.abs(want).reshape(rows, -1, 128), tol.reshape(rows, -1, 128)
    top = 448 * 2.0 ** e
    assert ((np.maximum(t - s, 0) <= top[..., None]).all()), what + ": a scale too small"
    small = ((t + s).max(2) > top / 2) | (sf == 0) | ((t - s).max(2) <= 0)
    assert small.all(), what + ": a scale too large"
    step = np.repeat(2.0 ** e, 128, axis=1)
    near(E4M3[q] * step, want, tol * (1 + 2.0 ** -4) + np.abs(want) * 2.0 ** -4 + step * 2.0 ** -10, what)


def check(gq, gsf, uq, usf, dy, w):
    args = [t.cuda() for t in (gq, gsf, uq, usf, dy)]
    wd = None if w is None else w.cuda()
    r = swiglu_bwd(decode8(gq.numpy(), gsf.numpy()), decode8(uq.numpy(), usf.numpy()), dy.double().numpy(),
                   None if w is None else w.numpy())
    dg, du, dw = sat.swiglu_bwd(*args, row_weights=wd)
    for got, k in ((dg, "dg"), (du, "du")):
        near(got.double().cpu(), r[k], r["e_" + k] * 1.01 + np.abs(r[k]) * U_BF16 + 2.0 ** -134, k)
    pairs = sat.swiglu_bwd_quant(*args, row_weights=wd)
    for i, k in enumerate(("dg", "du", "y")):
        near_pair(pairs[2 * i], pairs[2 * i + 1], r[k], r["e_" + k] + np.abs(r[k]) * 2.0 ** -24, k + " codes")
    short = sat.swiglu_bwd_quant(*args, row_weights=wd, recompute=False)
    assert short[4] is None and all(torch.equal(a, b) for a, b in zip(short[:4], pairs[:4]))
    if w is None:
        assert dw is None and pairs[6] is None
    else:
        near(dw.double().cpu(), r["dw"], r["e_dw"] + 1e-38, "dw")
        assert torch.equal(dw, pairs[6])
    device_status_ok()
    return dg, du, dw


def stash(rows, cols, seed, sigma=1.0):
    out = []
    for i in range(2):
        out += [t.cpu() for t in sat.quantize_rowwise(normal(rows, cols, seed + i, sigma).cuda())]
    return out


@pytest.mark.parametrize("rows,cols", [(1, 128), (2, 256), (5, 384), (33, 640), (7, 1408), (17, 2048), (9, 4096),
                                       (3, 4224), (2, 8320), (4099, 128), (301, 1536)])
@pytest.mark.parametrize("weights", [False, True])
def test_backward(rows, cols, weights):
    w = torch.randn(rows, generator=torch.Generator().manual_seed(9)) if weights else None
    check(*stash(rows, cols, rows + cols), normal(rows, cols, 77, 1e-3), w)


def test_backward_at_the_edges():
    """Gates from -400 to 400, zero tiles, codes of every value, scales from 2^-127 to 2^40,
    zero and negative weights, zero gradients."""
    rows, cols = 64, 512
    gq, gsf, uq, usf = stash(rows, cols, 5)
    g = torch.Generator().manual_seed(6)
    codes = torch.tensor([c for c in range(256) if c & 127 != 127], dtype=torch.uint8)
    gq[:32] = codes[torch.randint(0, codes.numel(), (32, cols), generator=g)]
    uq[16:48] = codes[torch.randint(0, codes.numel(), (32, cols), generator=g)]
    gsf[:32] = torch.randint(118, 128, (32, cols // 128), generator=g).to(torch.uint8)
    gsf[32:40] = torch.randint(0, 168, (8, cols // 128), generator=g).to(torch.uint8)
    usf[40:48] = torch.randint(0, 150, (8, cols // 128), generator=g).to(torch.uint8)
    gq[50:52], gsf[50:52] = 0, 127
    uq[51:53], usf[51:53] = 0, 127
    w = torch.randn(rows, generator=g)
    w[3], w[4], w[60] = 0.0, -1.5, 1e-30
    dy = normal(rows, cols, 8, 1.0)
    dy[7] = 0
    check(gq, gsf, uq, usf, dy, w)


def test_largest_gates():
    """The largest BF16 gate: its code's value is 2^128, beyond fp32, yet sigmoid' there is 0 and
    the gate's gradient is dy * up (and 0 for the negative one)."""
    gate = torch.ones((2, 128), dtype=torch.bfloat16)
    gate[0, :64], gate[0, 64:] = torch.finfo(torch.bfloat16).max, torch.finfo(torch.bfloat16).min
    up, dy = torch.full_like(gate, 1.5), torch.full_like(gate, 0.5)
    _, _, *s = sat.swiglu_quant_stash(gate.cuda(), up.cuda())
    dg = sat.swiglu_bwd(*s, dy.cuda())[0]
    assert (dg[0, :64] == 0.75).all() and (dg[0, 64:] == 0).all()
    dgq, dgsf, *_ = sat.swiglu_bwd_quant(*s, dy.cuda(), recompute=False)
    assert np.array_equal(decode8(dgq.cpu().numpy(), dgsf.cpu().numpy())[0], [0.75] * 64 + [0.0] * 64)
    device_status_ok()


def test_no_rows_no_columns():
    u8 = lambda *s: torch.empty(s, dtype=torch.uint8, device="cuda")  # noqa: E731
    dg, _, dw = sat.swiglu_bwd(u8(0, 256), u8(0, 2), u8(0, 256), u8(0, 2),
                               torch.empty((0, 256), dtype=torch.bfloat16, device="cuda"),
                               row_weights=torch.empty(0, device="cuda"))
    assert dg.shape == (0, 256) and dw.shape == (0,)
    e = torch.empty((5, 0), dtype=torch.bfloat16, device="cuda")
    assert sat.swiglu_bwd(u8(5, 0), u8(5, 0), u8(5, 0), u8(5, 0), e, row_weights=torch.ones(5, device="cuda"))[2].tolist() == [0.0] * 5
    assert sat.swiglu_quant_stash(e, e)[0].shape == (5, 0)
    device_status_ok()


def test_only_the_rows_asked_for_are_written():
    rows, cols = 21, 640
    s = [t.cuda() for t in stash(rows, cols, 3)]
    dy = normal(rows, cols, 4).cuda()
    outs = [torch.full((rows + 4, cols), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    dw = torch.full((rows + 4,), 7.0, device="cuda")
    w = torch.ones(rows, device="cuda")
    sat.fp8q_swiglu_bwd(*s, w, dy, rows, cols, *outs, dw)
    want = sat.swiglu_bwd(*s, dy, row_weights=w)
    for got, ref in zip((*outs, dw), want):
        assert torch.equal(got[:rows], ref) and (got[rows:] == 7.0).all()


def test_same_bits_on_streams_and_under_capture():
    rows, cols = 777, 1408
    a, b = [[t.cuda() for t in (*stash(rows, cols, k), normal(rows, cols, k + 5, 1e-2))] for k in (10, 20)]
    w = torch.rand(rows, device="cuda")
    run = lambda t, **o: [*sat.swiglu_bwd(*t, row_weights=w, **o), *sat.swiglu_bwd_quant(*t, row_weights=w, **o)]  # noqa: E731
    want = {"a": run(a), "b": run(b)}
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(s1):
        r1 = run(a)
    r2 = run(b, stream=s2)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(r1, want["a"])) and all(torch.equal(x, y) for x, y in zip(r2, want["b"]))
    buf = [t.clone() for t in a]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = run(buf)
    for k, src in (("b", b), ("a", a)):
        for x, y in zip(buf, src):
            x.copy_(y)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(r, want[k]))


def test_wrong_tensors_are_refused():
    gq, gsf, uq, usf = [t.cuda() for t in stash(4, 256, 1)]
    dy = normal(4, 256, 2).cuda()
    for bad in (lambda: sat.swiglu_bwd(gq, gsf, uq, usf, dy.float()), lambda: sat.swiglu_bwd(gq, gsf[:2], uq, usf, dy),
                lambda: sat.swiglu_bwd(gq, gsf, uq[:, :128], usf, dy), lambda: sat.swiglu_bwd(gq, gsf, uq, usf, dy.cpu()),
                lambda: sat.swiglu_quant_stash(dy, dy[:2]), lambda: sat.swiglu_quant_stash(dy, dy, row_weights=torch.ones(3, device="cuda")),
                lambda: sat.swiglu_bwd(gq, gsf, uq, usf, dy, row_weights=torch.ones(4, device="cuda").double())):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(sat.Fp8qError):
        sat.swiglu_quant_stash(dy[:, :100].contiguous(), dy[:, :100].contiguous())
