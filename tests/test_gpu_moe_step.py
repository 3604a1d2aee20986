"""The new operators together with the old ones, as one MoE layer uses them.

Training step: router -> FP8 permute -> experts' first products (the test's own, in fp32)
-> SwiGLU with 8-bit checkpoints and the routing weight of each row -> second products ->
unweighted combine; back through the SwiGLU from the checkpoints (the row weights' gradient
among it) and into the logits, the balance loss included.  The logits' gradient is held to
64-bit formulas on the same checkpoints.

Serving pass: router -> 4-bit permute -> experts' 4-bit products -> SwiGLU -> FP8 combine,
held to the same pass in 64 bits with the roundings' bounds added up."""
import numpy as np
import pytest
import torch

import scaling_aware_transpose_b200 as sat
from gpu_helpers import device_status_ok
from moe_reference import U, U_BF16, decode4, decode8, encode4, router, router_bwd, router_units, swiglu_bwd

pytestmark = pytest.mark.gpu


def values8(q, sf):
    """fp32 values of a row-wise pair, on the device."""
    s = torch.exp2(sf.float() - 127).repeat_interleave(128, 1)
    return q.view(torch.float8_e4m3fn).float() * s


@pytest.mark.parametrize("T,E,K,H,I,sigmoid", [(200, 8, 2, 256, 384, False), (77, 12, 4, 128, 256, True), (1, 6, 2, 256, 128, False)])
def test_training_step(T, E, K, H, I, sigmoid):
    g = torch.Generator().manual_seed(T)
    rnd = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    x, logits = rnd(T, H).to(torch.bfloat16).cuda(), (rnd(T, E) * 1.5).cuda()
    bias = (rnd(E) * 0.1).cuda() if sigmoid else None
    wg, wu, w2 = [(rnd(E, a, b) / a ** 0.5).cuda() for a, b in ((H, I), (H, I), (I, H))]
    opt = dict(sigmoid=sigmoid, scale=1.5, loss_coef=0.02)

    # forward
    idx, w, counts, sums, loss = sat.router_topk(logits, K, bias=bias, **opt)
    q, sf, off, rmap = sat.permute_pad_quant(x, idx, E, 128)
    rows = int(off[-1])
    expert = torch.bucketize(torch.arange(rows, device="cuda"), off[1:].long(), right=True)
    xv = values8(q[:rows], sf[:rows])
    up_to = lambda m: torch.bmm(xv[:, None, :], m[expert])[:, 0].to(torch.bfloat16)  # noqa: E731
    gate, up = up_to(wg), up_to(wu)
    rw = sat.permute_row_weights(w, rmap, rows)
    y, ysf, gq, gsf, uq, usf = sat.swiglu_quant_stash(gate, up, row_weights=rw)
    z = torch.bmm(values8(y, ysf)[:, None, :], w2[expert])[:, 0].to(torch.bfloat16)
    out = sat.unpermute_unpad(z, rmap, K)

    # backward of sum(out * r) + 0.7 * loss
    r = rnd(T, H).to(torch.bfloat16).cuda()
    dz = torch.zeros((rows, H), device="cuda")
    dz[rmap.long()] = r.float().repeat_interleave(K, 0)     # the combine's backward, unweighted
    dy = torch.bmm(dz[:, None, :], w2[expert].transpose(1, 2))[:, 0].to(torch.bfloat16)
    dgate, dup, drw = sat.swiglu_bwd(gq, gsf, uq, usf, dy, row_weights=rw)
    dgq, dgsf, duq, dusf, y2, y2sf, drw2 = sat.swiglu_bwd_quant(gq, gsf, uq, usf, dy, row_weights=rw)
    assert torch.equal(drw, drw2)
    for q8, s8 in ((dgq, dgsf), (duq, dusf), (y2, y2sf)):   # ready for the weight gradients' products
        qt, sft = sat.direct_transpose(q8, s8, group_offsets=off)
        assert qt.numel() == rows * I and sft.numel() == rows * I // 128
    dlogits = sat.router_topk_bwd(logits, idx, drw, row_id_map=rmap, counts=counts,
                                  grad_loss=torch.tensor([0.7], device="cuda"), **opt)
    device_status_ok()

    # 64 bits, from the same checkpoints and dy
    ref = router(logits.cpu().numpy(), K, sigmoid, True, None if bias is None else bias.cpu().numpy(), None, 1.5, 0.02)
    assert np.array_equal(idx.cpu().numpy(), ref["idx"]) and np.array_equal(counts.cpu().numpy(), ref["counts"])
    host = lambda t: t.cpu().numpy()  # noqa: E731
    s = swiglu_bwd(decode8(host(gq), host(gsf)), decode8(host(uq), host(usf)), dy.double().cpu().numpy(), host(rw))
    at = host(rmap).reshape(T, K)
    gw, e_gw = s["dw"][at], s["e_dw"][at]
    want, mag = router_bwd(host(logits), ref["idx"], gw, ref["counts"], 0.7, sigmoid, True, None, 1.5, 0.02)
    _, mag_e = router_bwd(host(logits), ref["idx"], e_gw, ref["counts"], None, sigmoid, True, None, 1.5, 0.02)
    tol = 4 * router_units(host(logits)) * U * mag + 2 * mag_e + 1e-30
    assert (np.abs(host(dlogits) - want) <= tol).all()
    # padding rows: weight 0, so no value and no gradient; their zero checkpoints decode to zero
    pad = np.setdiff1d(np.arange(rows), host(rmap))
    for t in (values8(y, ysf), dgate.float(), dup.float(), values8(dgq, dgsf), values8(y2, y2sf)):
        assert (t[torch.from_numpy(pad).cuda()] == 0).all()
    # the combine of the weighted rows against 64 bits: z and out are rounded to BF16
    zz = z.double().cpu().numpy()[at].sum(1)
    assert (np.abs(out.double().cpu().numpy() - zz) <= U_BF16 * np.abs(zz) + K * U * np.abs(z.double().cpu().numpy()[at]).sum(1)).all()
    # the recomputed y is the forward's up to the checkpoints' and its own rounding
    gv, uv = gate.double().cpu().numpy(), up.double().cpu().numpy()
    eg, eu = np.abs(gv) * 2.0 ** -4 + 2.0 ** -10 * np.repeat(2.0 ** (host(gsf) - 127.0), 128, 1), np.abs(uv) * 2.0 ** -4 + 2.0 ** -10 * np.repeat(2.0 ** (host(usf) - 127.0), 128, 1)
    act = np.abs(gv / (1 + np.exp(-gv)))
    bound = host(rw)[:, None] * (1.1 * eg * (np.abs(uv) + eu) + act * eu)   # |silu'| <= 1.1
    ya, yb = values8(y, ysf).double().cpu().numpy(), values8(y2, y2sf).double().cpu().numpy()
    step = 2.0 ** -10 * (np.repeat(2.0 ** (host(ysf) - 127.0), 128, 1) + np.repeat(2.0 ** (host(y2sf) - 127.0), 128, 1))
    assert (np.abs(ya - yb) <= bound * 1.07 + 2.0 ** -3 * 1.07 * np.maximum(np.abs(ya), np.abs(yb)) + step).all()


@pytest.mark.parametrize("T,E,K,H,I", [(150, 8, 2, 512, 256), (1, 32, 8, 256, 128), (33, 5, 1, 384, 384)])
def test_serving_pass(T, E, K, H, I):
    g = torch.Generator().manual_seed(T + 1)
    rnd = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    x, logits = rnd(T, H).to(torch.bfloat16), rnd(T, E)
    wg, wu = (rnd(E * I, H) / H ** 0.5).to(torch.bfloat16), (rnd(E * I, H) / H ** 0.5).to(torch.bfloat16)
    qg, qu = sat.quantize_rowwise_mxfp4(wg.cuda()), sat.quantize_rowwise_mxfp4(wu.cuda())   # once, at load time

    idx, w, _, _, _ = sat.router_topk(logits.cuda(), K, balance=False)
    q, sf, off, rmap = sat.permute_pad_mxfp4(x.cuda(), idx, E, 128)
    gate = sat.matmul_mxfp4(q, sf, *qg, group_offsets=off, out=torch.zeros((q.shape[0], I), dtype=torch.bfloat16, device="cuda"))
    up = sat.matmul_mxfp4(q, sf, *qu, group_offsets=off, out=torch.zeros_like(gate))
    yq, ysf, _, _ = sat.swiglu_quant(gate, up, transposed=False)
    out = sat.unpermute_unpad(yq, rmap, K, weights=w, y_sf=ysf)
    device_status_ok()

    xv = decode4(*encode4(x.double().numpy()))
    gv, uv = (decode4(*encode4(m.double().numpy())).reshape(E, I, H) for m in (wg, wu))
    ref = router(logits.numpy(), K)
    total, bound = np.zeros((T, I)), np.zeros((T, I))
    scale = np.repeat(2.0 ** (ysf.cpu().numpy() - 127.0), 128, 1)[rmap.cpu().numpy()].reshape(T, K, I)
    for t in range(T):
        for s in range(K):
            e = ref["idx"][t, s]
            a, b = gv[e] @ xv[t], uv[e] @ xv[t]
            mag = (H / 64 + 1) * 2.0 ** -22
            ea = np.abs(a) * U_BF16 + mag * (np.abs(gv[e]) @ np.abs(xv[t]))   # a BF16 rounding, the products' sums
            eb = np.abs(b) * U_BF16 + mag * (np.abs(uv[e]) @ np.abs(xv[t]))
            act = a / (1 + np.exp(-a))
            y = act * b
            ey = 1.1 * ea * (np.abs(b) + eb) + np.abs(act) * eb
            ey = ey + 2.0 ** -4 * (np.abs(y) + ey) + 2.0 ** -10 * scale[t, s]   # E4M3
            total[t] += ref["weights"][t, s] * y
            bound[t] += ref["weights"][t, s] * ey + 1e-5 * np.abs(y)
    got = out.double().cpu().numpy()
    assert (np.abs(got - total) <= bound + U_BF16 * (np.abs(total) + bound)).all()


def test_training_step_captured():
    """Forward and backward of the new operators in one graph, replayed on new inputs."""
    T, E, K, I = 256, 8, 2, 256
    mk = lambda s: (torch.randn((T, E), generator=torch.Generator().manual_seed(s)).cuda(),  # noqa: E731
                    torch.randn((T * K + E * 127, I), generator=torch.Generator().manual_seed(s + 1)).to(torch.bfloat16).cuda())
    x = torch.randn((T, 128), device="cuda").to(torch.bfloat16)
    one = torch.ones(1, device="cuda")

    def step(logits, a):
        idx, w, counts, sums, loss = sat.router_topk(logits, K)
        q, sf, off, rmap = sat.permute_pad_mxfp4(x, idx, E, 128)
        rw = sat.permute_row_weights(w, rmap, a.shape[0])
        y, ysf, *stash = sat.swiglu_quant_stash(a, a, row_weights=rw)
        dg, du, drw = sat.swiglu_bwd(*stash, a, row_weights=rw)
        return [w, loss, off, y, dg, drw, sat.router_topk_bwd(logits, idx, drw, row_id_map=rmap, counts=counts, grad_loss=one)]

    ins = {k: mk(k) for k in (1, 5)}
    want = {k: step(*v) for k, v in ins.items()}
    buf = [t.clone() for t in ins[1]]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(*buf)
    for k in (5, 1, 5):
        for b, v in zip(buf, ins[k]):
            b.copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want[k]))
    device_status_ok()


@pytest.mark.parametrize("tokens,E,K", [(5, 8, 2), (100, 16, 4), (700, 32, 8)])
def test_shared_buffers_keep_stream_order(tokens, E, K):
    """Two inputs by turns through the same rows, offsets and products, with nothing in between
    but the stream: few pairs (one plain launch before the product) and many."""
    k, n = 512, 384
    cap = tokens * K + E * 127
    g = torch.Generator().manual_seed(tokens)
    inputs = []
    for _ in range(2):
        logits = torch.randn((tokens, E), generator=g).cuda()
        x = torch.randn((tokens, k), generator=g).to(torch.bfloat16).cuda()
        inputs.append((logits, x))
    w = sat.quantize_rowwise_mxfp4(torch.randn((E * n, k), generator=g).to(torch.bfloat16).cuda())
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda")  # noqa: E731
    idx = torch.empty((tokens, K), dtype=torch.int32, device="cuda")
    wt = torch.empty((tokens, K), device="cuda")
    q, sf, ws = u8(cap, k // 2), u8(sat.fp8q_mxfp4_sf_bytes(cap, k)), u8(sat.fp8q_permute_workspace_bytes(tokens, K, E))
    off, rmap = (torch.empty(s, dtype=torch.int32, device="cuda") for s in (E + 1, tokens * K))
    out = torch.zeros((cap, n), dtype=torch.bfloat16, device="cuda")

    def step(logits, x):
        sat.fp8q_router_topk(logits, tokens, E, sat.ROUTER_RENORM, None, None, K, 1.0, 1.0, idx, wt, None, None, None, None, 0)
        sat.fp8q_permute_pad_mxfp4(x, tokens, k, idx, K, E, 128, q, sf, cap, off, rmap, ws, ws.numel())
        sat.fp8q_matmul_mxfp4(q, sf, cap, *w, n, k, off, E, out)
        return out[rmap.long()], off.clone(), rmap.clone(), wt.clone()

    want = []
    for a in inputs:
        want.append(step(*a))
        torch.cuda.synchronize()
    got = [step(*inputs[i % 2]) for i in range(30)]
    torch.cuda.synchronize()
    for i, r in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(r, want[i % 2])), i
    # without the reads in between, the last step's results stand
    for i in range(31):
        sat.fp8q_router_topk(inputs[i % 2][0], tokens, E, sat.ROUTER_RENORM, None, None, K, 1.0, 1.0, idx, wt, None, None,
                             None, None, 0)
        sat.fp8q_permute_pad_mxfp4(inputs[i % 2][1], tokens, k, idx, K, E, 128, q, sf, cap, off, rmap, ws, ws.numel())
        sat.fp8q_matmul_mxfp4(q, sf, cap, *w, n, k, off, E, out)
    assert torch.equal(out[rmap.long()], want[0][0]) and torch.equal(off, want[0][1])
    device_status_ok()
