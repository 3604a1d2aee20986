"""MXFP4: quantization byte for byte against the definition (every BF16 value, ragged rows,
the fused permute), and the products against 64-bit sums with the bound of
moe_reference.matmul_bound: one row to many, odd sizes, odd k tiles, scales over a wide
range, expert groups with empty ones, rows past the last group."""
import numpy as np
import pytest
import torch

import scaling_aware_transpose_b200 as sat
from gpu_helpers import device_status_ok
from moe_reference import decode4, encode4, matmul_bound, tile_scales
from scaling_aware_transpose_b200 import synthetic

pytestmark = pytest.mark.gpu


def normal(rows, cols, seed, row_sigma=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((rows, cols), generator=g) * torch.exp(row_sigma * torch.randn((rows, 1), generator=g))
    return x.to(torch.bfloat16)


def quantized(x):
    q, sf = encode4(x.double().numpy())
    return q, sf, decode4(q, sf)


def near(got, want, tol, what):
    got = got.double().cpu().numpy()
    off = np.abs(got - want)
    bad = ~(off <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {np.nanmax(off)}, at {np.argwhere(bad)[:4].tolist()}"


# ------------------------------------------------------------------ quantization
@pytest.mark.parametrize("rows,cols", [(1, 128), (3, 384), (127, 128), (128, 256), (129, 640), (1000, 1408), (77, 7168)])
def test_quantize(rows, cols):
    x = normal(rows, cols, rows + cols)
    x[0, :64] = 0
    if rows > 2:
        x[2, 32:64] = -0.0
    q, sf = sat.quantize_rowwise_mxfp4(x.cuda())
    eq, esf, _ = quantized(x)
    assert np.array_equal(q.cpu().numpy(), eq)
    assert np.array_equal(sf.cpu().numpy(), tile_scales(esf))
    assert torch.equal(sat.mxfp4_tile_scales(torch.from_numpy(esf)), sf.cpu())
    device_status_ok()


def test_quantize_every_bf16_value():
    """Each finite BF16 value beside every amax position: as its tile's largest value, and
    below a larger one (16 binades up), so that every rounding border and scale is met."""
    bits = np.arange(65536, dtype=np.uint32)
    bits = bits[(bits & 0x7F80) != 0x7F80].astype(np.uint16)
    v = torch.from_numpy(bits.view(np.int16)).view(torch.bfloat16)
    n = v.numel() // 32 * 32
    rows = []
    for up in (0, 1, 2, 3):
        t = v[:n].view(-1, 32).clone()
        if up:
            t[:, 31] = (t[:, :31].float().abs().amax(1) * 2.0 ** (up - 1)).clamp_max(3.3e38).to(torch.bfloat16)
        rows.append(t)
    x = torch.cat(rows)
    x = x[: x.shape[0] // 4 * 4].reshape(-1, 128)
    q, sf = sat.quantize_rowwise_mxfp4(x.cuda())
    eq, esf, _ = quantized(x)
    assert np.array_equal(sf.cpu().numpy(), tile_scales(esf))
    assert np.array_equal(q.cpu().numpy(), eq)


def test_quantize_writes_its_rows_only():
    x = normal(130, 256, 1).cuda()
    q = torch.full((140, 128), 0xEE, dtype=torch.uint8, device="cuda")
    sf = torch.full((sat.fp8q_mxfp4_sf_bytes(130, 256) + 512,), 0xEE, dtype=torch.uint8, device="cuda")
    sat.fp8q_quantize_rowwise_mxfp4(x, 130, 256, q, sf)
    assert (q[130:] == 0xEE).all() and (sf[-512:] == 0xEE).all() and not (sf[:-512] == 0xEE).any()


@pytest.mark.parametrize("tokens,hidden,E,K,align", [(1, 128, 4, 2, 128), (300, 640, 8, 3, 128), (513, 256, 32, 8, 16),
                                                     (97, 384, 5, 1, 1), (64, 128, 600, 4, 128),
                                                     (128, 256, 32, 8, 128), (129, 256, 32, 8, 128),
                                                     (1024, 128, 128, 1, 4), (1024, 128, 129, 1, 4), (16, 128, 100, 64, 8), (7, 1408, 2, 1, 4096),
                                                     (33, 7168, 31, 3, 16)])
def test_permute(tokens, hidden, E, K, align):
    d = synthetic.moe(tokens=tokens, hidden=hidden, num_experts=E, topk=K, seed=tokens)
    x, idx = synthetic.to_torch_bf16(d["x"]), torch.from_numpy(d["topk_idx"])
    q, sf, off, rmap = sat.permute_pad_mxfp4(x.cuda(), idx.cuda(), E, align)
    _, _, off8, rmap8 = sat.permute_pad_quant(x.cuda(), idx.cuda(), E, align)
    assert torch.equal(off, off8) and torch.equal(rmap, rmap8)
    rows = int(off[-1])
    eq, esf, _ = quantized(x)
    wq, wsf = np.zeros((rows, hidden // 2), np.uint8), np.full((rows, hidden // 32), 127, np.uint8)
    at = rmap.cpu().numpy()
    wq[at], wsf[at] = np.repeat(eq, K, 0), np.repeat(esf, K, 0)
    assert np.array_equal(q[:rows].cpu().numpy(), wq)
    got = sf.cpu().numpy()
    mask = tile_scales(np.ones_like(wsf), 0) == 1
    assert np.array_equal(got[:mask.size][mask], tile_scales(wsf)[mask])
    device_status_ok()


@pytest.mark.parametrize("tokens,E,K", [(40, 6, 4), (128, 128, 8), (128, 256, 8), (300, 9, 4)])
def test_permute_of_repeated_and_bad_ids(tokens, E, K):
    """A token may name an expert twice; ids out of range are reported and get no row.  Few
    pairs (one launch) and many, as the E4M3 permute treats them."""
    g = torch.Generator().manual_seed(tokens)
    x = normal(tokens, 256, 3)
    idx = torch.randint(0, E, (tokens, K), generator=g).int()
    idx[:, 1] = idx[:, 0]
    idx[5, 2], idx[7, 0], idx[tokens - 1, K - 1] = E, -1, 1 << 30
    q, sf, off, rmap = sat.permute_pad_mxfp4(x.cuda(), idx.cuda(), E, 16)
    assert sat.fp8q_last_device_status() == sat.FP8Q_ERR_DEVICE
    _, _, off8, rmap8 = sat.permute_pad_quant(x.cuda(), idx.cuda(), E, 16)
    assert sat.fp8q_last_device_status() == sat.FP8Q_ERR_DEVICE
    assert torch.equal(off, off8) and torch.equal(rmap, rmap8)
    eq, _, _ = quantized(x)
    at = rmap.view(tokens, K).cpu().numpy()
    want = np.zeros((int(off[-1]), 128), np.uint8)
    for k in range(K):
        want[at[at[:, k] >= 0, k]] = eq[at[:, k] >= 0]
    assert np.array_equal(q[:int(off[-1])].cpu().numpy(), want)


def test_permute_leaves_rows_behind_the_last_expert():
    d = synthetic.moe(tokens=50, hidden=256, num_experts=4, topk=2, seed=3)
    x, idx = synthetic.to_torch_bf16(d["x"]).cuda(), torch.from_numpy(d["topk_idx"]).cuda()
    cap = sat.permute_max_rows(50, 2, 4, 128) + 128
    q = torch.full((cap, 128), 0xEE, dtype=torch.uint8, device="cuda")
    sf = torch.full((sat.fp8q_mxfp4_sf_bytes(cap, 256),), 0xEE, dtype=torch.uint8, device="cuda")
    off, rmap = torch.empty(5, dtype=torch.int32, device="cuda"), torch.empty(100, dtype=torch.int32, device="cuda")
    ws = torch.empty(sat.fp8q_permute_workspace_bytes(50, 2, 4), dtype=torch.uint8, device="cuda")
    sat.fp8q_permute_pad_mxfp4(x, 50, 256, idx, 2, 4, 128, q, sf, cap, off, rmap, ws, ws.numel())
    rows = int(off[-1])
    assert rows % 128 == 0 and rows < cap
    assert (q[rows:] == 0xEE).all() and (sf[sat.fp8q_mxfp4_sf_bytes(rows, 256):] == 0xEE).all()
    device_status_ok()


def test_permute_without_tokens():
    off = sat.permute_pad_mxfp4(torch.empty((0, 256), dtype=torch.bfloat16, device="cuda"),
                                torch.empty((0, 2), dtype=torch.int32, device="cuda"), 4, 128)[2]
    assert off.tolist() == [0] * 5


# ------------------------------------------------------------------ products
def operand(rows, k, seed, spread=0):
    """Random codes and scales: (codes, tiled scales, values)."""
    rng = np.random.default_rng(seed)
    q = rng.integers(0, 256, (rows, k // 2), dtype=np.uint8)
    sf = rng.integers(127 - spread, 128 + spread, (rows, k // 32)).astype(np.uint8)
    return torch.from_numpy(q).cuda(), torch.from_numpy(tile_scales(sf)).cuda(), decode4(q, sf)


def product(m, n, k, spread, seed=0):
    aq, asf, a = operand(m, k, seed, spread)
    bq, bsf, b = operand(n, k, seed + 1, spread)
    out = sat.matmul_mxfp4(aq, asf, bq, bsf)
    device_status_ok()
    want, tol = matmul_bound(a, b)
    near(out, want, tol, f"{m}x{n}x{k}")
    return out


def test_product_of_one_tile_without_scales():
    product(128, 128, 256, 0)


def test_product_of_one_tile():
    product(128, 128, 256, 4)


@pytest.mark.parametrize("k", [128, 256, 384, 512, 1408, 2304, 7168])
def test_product_k(k):
    product(128, 128, k, 3, k)


@pytest.mark.parametrize("m", [1, 2, 7, 8, 16, 17, 31, 64, 65, 127, 129, 200, 256, 300, 1000])
def test_product_m(m):
    product(m, 256, 512, 3, m)


@pytest.mark.parametrize("n", [1, 2, 7, 8, 31, 33, 64, 96, 100, 127, 128, 129, 160, 192, 255, 256, 257, 320, 384, 640, 1001])
def test_product_n(n):
    product(70, n, 384, 3, n)
    product(3, n, 640, 3, n)


@pytest.mark.parametrize("m,n,k", [(1, 4096, 7168), (5, 2050, 1408), (16, 7168, 2048), (33, 1000, 4096), (400, 2048, 2048),
                                   (1500, 1536, 640), (4096, 4096, 512), (2500, 5000, 256)])
def test_product_large(m, n, k):
    product(m, n, k, 2, m)


@pytest.mark.parametrize("m,n,k", [(2, 4821, 128), (130, 2048, 1152), (61, 2467, 3456), (40, 2560, 3456), (5, 67, 1664),
                                   (128, 200, 3200), (2, 10885, 384), (300, 5120, 640), (2, 5597, 3456), (7, 5600, 3456),
                                   (2, 2469, 1920), (100, 2472, 1920), (131, 9690, 640), (256, 9728, 896),
                                   (2, 9735, 4992), (90, 9736, 4992), (2, 4884, 2944), (128, 4888, 2944),
                                   (260, 9517, 640), (148, 9512, 640), (1, 10168, 6400), (3, 10016, 6400),
                                   (1, 6464, 2944), (79, 2720, 3584), (65, 2398, 3200), (1003, 2050, 640)])
def test_product_by_every_tile_width(m, n, k):
    """Sizes on either side of 16-byte rows for each tile width, alone and with k shared by two
    or four CTAs (odd numbers of scale tiles among them)."""
    product(m, n, k, 3, m + n)


@pytest.mark.parametrize("m,n,k", [(2048, 4096, 4096), (2001, 4001, 4224), (4096, 2050, 7168), (3300, 3584, 2176),
                                   (2561, 2560, 8192), (134, 10296, 4224)])
def test_product_by_pairs(m, n, k):
    """Sizes that CTA pairs take: whole 256 x 256 tiles, a second CTA without rows, ragged
    columns, an odd number of scale tiles."""
    product(m, n, k, 2, m)


@pytest.mark.parametrize("m,n,k", [(70, 96, 256), (300, 2048, 512), (300, 5120, 640), (260, 9520, 640), (4, 2048, 4096),
                                   (2048, 4096, 1024), (2000, 4104, 2048)])
def test_product_into_rows_on_16_bytes(m, n, k):
    """Rows that start on 16 bytes but not on 32, though n is a multiple of 16 (or of 8)."""
    aq, asf, a = operand(m, k, 1, 2)
    bq, bsf, b = operand(n, k, 2, 2)
    buf = torch.full((m * n + 16,), 7.0, dtype=torch.bfloat16, device="cuda")
    out = buf[8:8 + m * n].view(m, n)
    sat.matmul_mxfp4(aq, asf, bq, bsf, out=out)
    assert torch.equal(out, sat.matmul_mxfp4(aq, asf, bq, bsf)) and (buf[:8] == 7.0).all() and (buf[-8:] == 7.0).all()
    device_status_ok()


def test_product_wide_scales_and_nan():
    product(130, 140, 640, 20)
    aq, asf, a = operand(4, 256, 1)
    bq, bsf, b = operand(128, 256, 2)
    asf[16 * 2 + 3] = 255  # row 2, scale column 3
    out = sat.matmul_mxfp4(aq, asf, bq, bsf)
    assert torch.isnan(out[2]).all() and not torch.isnan(out[[0, 1, 3]]).any()


def test_product_of_quantized_rows():
    x, w = normal(77, 1408, 1), normal(300, 1408, 2)
    out = sat.matmul_mxfp4(*sat.quantize_rowwise_mxfp4(x.cuda()), *sat.quantize_rowwise_mxfp4(w.cuda()))
    want, tol = matmul_bound(quantized(x)[2], quantized(w)[2])
    near(out, want, tol, "quantized rows")


def test_rows_and_columns_past_the_end_are_not_written():
    aq, asf, a = operand(70, 256, 1)
    bq, bsf, b = operand(200, 256, 2)
    buf = torch.full((90 * 200,), 7.0, dtype=torch.bfloat16, device="cuda")
    sat.fp8q_matmul_mxfp4(aq, asf, 70, bq, bsf, 200, 256, None, 1, buf)
    want, tol = matmul_bound(a, b)
    near(buf[: 70 * 200].view(70, 200), want, tol, "rows")
    assert (buf[70 * 200:] == 7.0).all()


@pytest.mark.parametrize("sizes", [[128], [0, 128, 0], [256, 0, 384, 128], [0, 0], [128] * 40, [1024, 128, 0, 0, 640]])
@pytest.mark.parametrize("n", [128, 384])
def test_grouped(sizes, n):
    k, G = 384, len(sizes)
    rows = sum(sizes)
    cap = rows + 200
    aq, asf, a = operand(cap, k, rows, 2)
    bq, bsf, b = operand(G * n, k, rows + 1, 2)
    off = torch.tensor(np.cumsum([0, *sizes]), dtype=torch.int32, device="cuda")
    out = torch.full((cap, n), 7.0, dtype=torch.bfloat16, device="cuda")
    sat.matmul_mxfp4(aq, asf, bq, bsf, group_offsets=off, out=out)
    device_status_ok()
    at = 0
    for g, s in enumerate(sizes):
        if s:
            want, tol = matmul_bound(a[at:at + s], b[g * n:(g + 1) * n])
            near(out[at:at + s], want, tol, f"group {g}")
        at += s
    assert (out[rows:] == 7.0).all()


@pytest.mark.parametrize("sizes,n,k,more", [([1408, 0, 1152, 640], 2048, 2304, 300), ([128, 2048, 128, 1664], 1152, 4224, 300),
                                            ([1408, 0, 1152, 640], 2048, 7168, 300), ([128, 2048, 128, 1664], 1152, 7168, 300),
                                            ([2560, 0, 0], 2432, 3968, 300), ([0, 128, 128], 5120, 4736, 381),
                                            ([128, 128, 0], 512, 4608, 381), ([0, 128, 128], 128, 2944, 40),
                                            ([128, 128], 3328, 384, 254), ([128, 0, 0, 256], 384, 4736, 508),
                                            ([0, 0, 0, 256], 4864, 640, 508), ([256, 128, 128], 128, 128, 0)])
def test_grouped_by_every_kernel(sizes, n, k, more):
    """Pairs (groups whose last 256 rows are half full, empty and single-tile groups among large
    ones) and each tile width, alone and with k shared."""
    G, rows = len(sizes), sum(sizes)
    cap = rows + more
    aq, asf, a = operand(cap, k, rows, 2)
    bq, bsf, b = operand(G * n, k, rows + 1, 2)
    off = torch.tensor(np.cumsum([0, *sizes]), dtype=torch.int32, device="cuda")
    out = torch.full((cap, n), 7.0, dtype=torch.bfloat16, device="cuda")
    sat.matmul_mxfp4(aq, asf, bq, bsf, group_offsets=off, out=out)
    device_status_ok()
    at = 0
    for g, s in enumerate(sizes):
        if s:
            want, tol = matmul_bound(a[at:at + s], b[g * n:(g + 1) * n])
            near(out[at:at + s], want, tol, f"group {g}")
        at += s
    assert (out[rows:] == 7.0).all()
    for bad in ([0, 100, *off.tolist()[2:]], [128, *off.tolist()[1:]], [*off.tolist()[:-1], cap + 84]):
        sat.matmul_mxfp4(aq, asf, bq, bsf, group_offsets=torch.tensor(bad, dtype=torch.int32, device="cuda"), out=out)
        assert sat.fp8q_last_device_status() == sat.FP8Q_ERR_SHAPE, bad


def test_bad_groups_are_reported_and_skipped():
    aq, asf, _ = operand(512, 256, 1)
    bq, bsf, _ = operand(3 * 128, 256, 2)
    for bad in ([0, 100, 256, 512], [128, 128, 256, 512], [0, 256, 128, 512], [0, 128, 256, 640], [0, 128, 256, -128]):
        out = torch.full((512, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        sat.matmul_mxfp4(aq, asf, bq, bsf, group_offsets=torch.tensor(bad, dtype=torch.int32, device="cuda"), out=out)
        assert sat.fp8q_last_device_status() == sat.FP8Q_ERR_SHAPE, bad


def test_routed_tokens_through_the_experts():
    T, H, E, K, n = 333, 512, 6, 2, 256
    d = synthetic.moe(tokens=T, hidden=H, num_experts=E, topk=K, seed=9)
    x, idx = synthetic.to_torch_bf16(d["x"]), torch.from_numpy(d["topk_idx"])
    w = normal(E * n, H, 4)
    q, sf, off, rmap = sat.permute_pad_mxfp4(x.cuda(), idx.cuda(), E, 128)
    y = sat.matmul_mxfp4(q, sf, *sat.quantize_rowwise_mxfp4(w.cuda()), group_offsets=off)
    xv, wv = quantized(x)[2], quantized(w)[2]
    for s in range(K):
        rows = y[rmap.view(T, K)[:, s].long()]
        for e in range(E):
            pick = (idx[:, s] == e).numpy()
            if pick.any():
                want, tol = matmul_bound(xv[pick], wv[e * n:(e + 1) * n])
                near(rows[torch.from_numpy(pick).cuda()], want, tol, f"slot {s} expert {e}")
    device_status_ok()


def test_same_bits_on_streams_and_under_capture():
    a, b = [operand(300, 640, s, 2)[:2] for s in (1, 2)]
    w = operand(700, 640, 3, 2)[:2]
    x = normal(300, 640, 4).cuda()

    def run(t, **o):
        return [sat.matmul_mxfp4(*t, *w, **o), sat.matmul_mxfp4(*sat.quantize_rowwise_mxfp4(x, **o), *w, **o)]

    want = {"a": run(a), "b": run(b)}
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        with torch.cuda.stream(s1):
            r1 = run(a)
        r2 = run(b, stream=s2)
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(r1, want["a"]))
        assert all(torch.equal(u, v) for u, v in zip(r2, want["b"]))
    buf = [t.clone() for t in a]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = run(buf)
    for key, src in (("b", b), ("a", a)):
        for u, v in zip(buf, src):
            u.copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(r, want[key]))
    device_status_ok()


def test_wrong_tensors_are_refused():
    aq, asf, _ = operand(8, 256, 1)
    bq, bsf, _ = operand(16, 256, 2)
    off = torch.zeros(2, dtype=torch.int32, device="cuda")
    for bad in (lambda: sat.matmul_mxfp4(aq, asf[:100], bq, bsf), lambda: sat.matmul_mxfp4(aq, asf, bq[:, :64].contiguous(), bsf),
                lambda: sat.matmul_mxfp4(aq.cpu(), asf, bq, bsf), lambda: sat.matmul_mxfp4(aq, asf, bq, bsf, group_offsets=off.long()),
                lambda: sat.matmul_mxfp4(aq, asf, bq, bsf, out=torch.empty((8, 15), dtype=torch.bfloat16, device="cuda")),
                lambda: sat.quantize_rowwise_mxfp4(torch.ones((2, 128), device="cuda")),
                lambda: sat.mxfp4_tile_scales(torch.ones((2, 5), dtype=torch.uint8))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(sat.Fp8qError):  # groups need n % 128 == 0
        sat.matmul_mxfp4(aq, asf, bq, bsf, group_offsets=off)
