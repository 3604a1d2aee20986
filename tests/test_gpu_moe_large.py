"""The operators around the path past 2^31 elements: what lies there, and across the border,
has the same bits as a call on those rows alone (each row's results are its own), products are
held to 64-bit sums."""
import numpy as np
import pytest
import torch

import scaling_aware_transpose_b200 as sat
from gpu_helpers import device_status_ok
from moe_reference import decode4, matmul_bound

pytestmark = pytest.mark.gpu
BORDER = 1 << 31


def need(gib):
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < gib << 30:
        pytest.skip(f"needs {gib} GiB")


def random_bf16(rows, cols, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    out = torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda")
    for part in out.split(1 << 17):
        part.copy_(torch.randn(part.shape, generator=g, device="cuda") * scale)
    return out


def slices(rows, cols):
    """Row ranges at the start, across the border and at the end."""
    at = BORDER // cols
    return (slice(0, 70), slice(at - 40, at + 40), slice(rows - 77, rows))


def test_swiglu_checkpoints_and_backward():
    need(48)
    cols = 2048
    rows = BORDER // cols + 5003
    gate, up, dy = random_bf16(rows, cols, 1), random_bf16(rows, cols, 2), random_bf16(rows, cols, 3, 1e-2)
    w = torch.rand(rows, device="cuda")
    s = sat.swiglu_quant_stash(gate, up, row_weights=w)
    dg, du, dw = sat.swiglu_bwd(*s[2:], dy, row_weights=w)
    pairs = sat.swiglu_bwd_quant(*s[2:], dy, row_weights=w)
    device_status_ok()
    for r in slices(rows, cols):
        want = sat.swiglu_quant_stash(gate[r], up[r], row_weights=w[r])
        assert all(torch.equal(a[r], b) for a, b in zip(s, want)), r
        codes, d = [t[r].contiguous() for t in s[2:]], dy[r]
        assert all(torch.equal(a[r], b) for a, b in zip((dg, du, dw), sat.swiglu_bwd(*codes, d, row_weights=w[r]))), r
        assert all(torch.equal(a[r], b) for a, b in zip(pairs, sat.swiglu_bwd_quant(*codes, d, row_weights=w[r]))), r


def test_router():
    need(24)
    E, K = 256, 4
    T = BORDER // E + 100003
    l = random_bf16(T, E, 4)
    mask = (torch.arange(T, device="cuda") % 11 != 0).to(torch.uint8)
    bias = torch.linspace(-0.1, 0.1, E, device="cuda")
    gl, gw = torch.ones(1, device="cuda"), torch.randn((T, K), device="cuda")
    for o in (dict(sigmoid=True), dict()):
        b = bias if o else None
        idx, w, counts, sums, loss = sat.router_topk(l, K, bias=b, token_mask=mask, **o)
        grad = sat.router_topk_bwd(l, idx, gw, counts=counts, grad_loss=gl, token_mask=mask, **o)
        device_status_ok()
        live = int(mask.sum())
        assert int(counts.sum()) == live * K and abs(float(sums.double().sum()) / live - 1) < 1e-4
        assert torch.equal(counts.long(), torch.bincount(idx[mask != 0].reshape(-1).long(), minlength=E))
        for r in slices(T, E):
            i2, w2, *_ = sat.router_topk(l[r], K, bias=b, token_mask=mask[r], balance=False, **o)
            assert torch.equal(idx[r], i2) and torch.equal(w[r], w2), r
            g2 = sat.router_topk_bwd(l[r], i2, gw[r], counts=counts, grad_loss=gl, token_mask=mask[r], **o)
            assert torch.equal(grad[r], g2), r


def test_quantize_and_permute_mxfp4():
    need(32)
    cols = 7168
    rows = BORDER // cols + 301
    x = random_bf16(rows, cols, 5)
    q, sf = sat.quantize_rowwise_mxfp4(x)
    at = BORDER // cols // 128 * 128
    for r in (slice(0, 256), slice(at - 128, at + 128), slice(rows // 128 * 128 - 128, rows)):
        q2, sf2 = sat.quantize_rowwise_mxfp4(x[r])
        first = sat.fp8q_mxfp4_sf_bytes(r.start, cols)
        assert torch.equal(q[r], q2) and torch.equal(sf[first:first + sf2.numel()], sf2), r
    E, K = 8, 3
    g = torch.Generator(device="cuda").manual_seed(6)
    idx = torch.rand((rows, E), generator=g, device="cuda").topk(K, 1).indices.int()
    pq, psf, off, rmap = sat.permute_pad_mxfp4(x, idx, E, 128)
    device_status_ok()
    assert int(off[-1]) * (cols // 2) > BORDER
    for s in range(K):  # every row's codes, and its scales by their place
        to = rmap.view(rows, K)[:, s].long()
        for part in torch.arange(rows, device="cuda").split(1 << 16):
            assert torch.equal(pq[to[part]], q[part]), s
        r = torch.tensor([0, 1, at, rows // 2, rows - 1], device="cuda")
        words = lambda t, rr: t.view(-1, cols // 128, 32, 4, 4)[rr >> 7, :, rr & 31, rr >> 5 & 3]  # noqa: E731
        assert torch.equal(words(psf, to[r]), words(sf, r)), s


@pytest.mark.parametrize("m,n,k", [(1050001, 2064, 128), (4, 600064, 7296), (600064, 16, 7296), (600001, 3587, 128)])
def test_products(m, n, k):
    """Results, weights and rows past 2^31 elements."""
    need(24)
    assert max(m * n, n * k, m * k) > BORDER
    g = torch.Generator(device="cuda").manual_seed(m)

    def operand(rows):
        q = torch.randint(0, 256, (rows, k // 2), generator=g, device="cuda", dtype=torch.uint8)
        sf = torch.randint(125, 130, (rows, k // 32), generator=g, device="cuda", dtype=torch.uint8)
        return q, sf, sat.mxfp4_tile_scales(sf)

    (aq, asf, at), (bq, bsf, bt) = operand(m), operand(n)
    out = sat.matmul_mxfp4(aq, at, bq, bt)
    device_status_ok()
    pick = lambda rows: torch.tensor(sorted({0, rows // 3, rows // 2, rows * 9 // 10, *range(max(0, rows - 150), rows)}),  # noqa: E731
                                     device="cuda")
    r, c = pick(m), pick(n)
    a, b = (decode4(q[i].cpu().numpy(), sf[i].cpu().numpy()) for q, sf, i in ((aq, asf, r), (bq, bsf, c)))
    want, tol = matmul_bound(a, b)
    off = np.abs(out[r][:, c].double().cpu().numpy() - want)
    assert (off <= tol).all(), (off.max(), np.argwhere(off > tol)[:3])
