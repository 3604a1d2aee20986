"""The router and its gradient against plain 64-bit forms: odd expert counts, one to many
tokens, ties, switched-off experts, masked rows holding NaN, rows with nothing left,
selection biases closer than fp32 resolves, gradients against the formula and differences.

Tolerances count roundings: `router_units` half steps of fp32 for a probability (derived
there), doubled where two of them multiply; a BF16 result adds half a BF16 step."""
import numpy as np
import pytest
import torch

import scaling_aware_transpose_b200 as sat
from gpu_helpers import device_status_ok
from moe_reference import U, U_BF16, router, router_bwd, router_units

pytestmark = pytest.mark.gpu


def make(T, E, seed, dtype=torch.float32, spread=1.5):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((T, E), generator=g) * spread).to(dtype)


def near(got, want, tol, what):
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    off = np.abs(got - want)
    bad = ~(off <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {np.nanmax(off)}, at {np.argwhere(bad)[:3]}"


def check(logits, K, sigmoid=False, renorm=True, bias=None, mask=None, scale=1.0, coef=0.01, seed=0):
    T, E = logits.shape
    host = logits.float().numpy()
    ref = router(host, K, sigmoid, renorm, None if bias is None else bias.numpy(), None if mask is None else mask.numpy(),
                 scale, coef)
    cu = lambda t: None if t is None else t.cuda()  # noqa: E731
    opt = dict(sigmoid=sigmoid, renormalize=renorm, token_mask=cu(mask), scale=scale, loss_coef=coef)
    d = cu(logits)
    idx, w, counts, sums, loss = sat.router_topk(d, K, bias=cu(bias), **opt)
    idx2, w2, none, _, _ = sat.router_topk(d, K, bias=cu(bias), balance=False, **opt)
    assert none is None and torch.equal(idx, idx2) and torch.equal(w, w2)
    n = router_units(host)
    assert np.array_equal(idx.cpu().numpy(), ref["idx"]), "ids"
    assert np.array_equal(counts.cpu().numpy(), ref["counts"]), "counts"
    near(w.cpu(), ref["weights"], 2 * n * U * np.abs(ref["weights"]) + 1e-30, "weights")
    # a sum of shares: each off by 2n U, plus up to ceil(T / 4736) + 8 additions in fp32
    near(sums.cpu(), ref["sums"], (2 * n + T / 4736 + 9) * U * ref["sums"] + 1e-30, "prob_sums")
    near(loss.cpu(), ref["loss"], (2 * n + T / 4736 + 12) * U * abs(ref["loss"]), "loss")
    g = torch.Generator().manual_seed(seed + 1)
    gw = torch.randn((T, K), generator=g)
    gl = torch.tensor([1.3])
    bf = logits.dtype == torch.bfloat16
    for use_w, use_l in ((True, True), (True, False), (False, True), (False, False)):
        grad = sat.router_topk_bwd(d, idx, cu(gw) if use_w else None, counts=counts if use_l else None,
                                   grad_loss=cu(gl) if use_l else None, **opt)
        want, mag = router_bwd(host, ref["idx"], gw.numpy() if use_w else None, ref["counts"], 1.3 if use_l else None,
                               sigmoid, renorm, None if mask is None else mask.numpy(), scale, coef)
        assert grad.dtype == logits.dtype and torch.isfinite(grad).all()
        near(grad.float().cpu(), want, 4 * n * U * mag + 1e-30 + (U_BF16 * np.abs(want) * 1.01 if bf else 0), "gradient")
    device_status_ok()
    return idx, w, counts, sums, loss


@pytest.mark.parametrize("E,K", [(1, 1), (2, 2), (8, 3), (31, 31), (32, 8), (33, 8), (60, 6), (64, 64), (100, 40),
                                 (256, 8), (257, 5), (512, 64), (1000, 33), (1024, 8)])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_expert_counts(E, K, sigmoid):
    check(make(37, E, E + K), K, sigmoid=sigmoid)
    check(make(19, E, E + K + 1, torch.bfloat16), K, sigmoid=sigmoid, renorm=False, scale=2.5)


@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 1000, 5003, 40001])
def test_token_counts(T):
    check(make(T, 32, T, torch.bfloat16), 8)
    check(make(T, 72, T), 6, sigmoid=True, bias=torch.randn(72, generator=torch.Generator().manual_seed(3)) * 0.1)


@pytest.mark.parametrize("E", [100, 140, 300, 1024])
def test_ties_take_the_lowest_id(E):
    l = torch.zeros((5, E))
    l[1, ::2] = -0.0
    l[2, 50:] = 1.0
    l[3] = torch.arange(E).flip(0) // 10
    idx = check(l, 12)[0].cpu()
    assert idx[0].tolist() == list(range(12)) and idx[1].tolist() == list(range(12))
    assert idx[2].tolist() == list(range(50, 62))
    check(l, 12, sigmoid=True, bias=torch.zeros(E))


def test_bias_ties_below_fp32_resolution():
    """Scores that differ by 2^-40: the choice follows the double sums."""
    g = torch.Generator().manual_seed(5)
    E = 96
    l = torch.full((64, E), 0.25) + torch.randint(0, 2, (64, E), generator=g) * 2.0 ** -24
    bias = torch.randint(-3, 4, (E,), generator=g).float() * 2.0 ** -40
    check(l, 8, sigmoid=True, bias=bias)
    # a bias alone decides where the scores are equal
    check(torch.zeros((3, E)), 9, sigmoid=True, bias=torch.randn(E, generator=g))


@pytest.mark.parametrize("E", [60, 128, 160, 320, 1000])
def test_switched_off_masked_and_empty_rows(E):
    T, K = 301, 6
    l = make(T, E, 11)
    l[:, 7] = -float("inf")
    l[5] = -float("inf")             # nothing left
    l[6, 3:] = -float("inf")         # fewer experts than slots
    l[8, 4] = float("inf")           # the largest finite value
    l[9] = -3.0e38                   # the lowest values of the type
    l[10, ::2] = -3.4028234663852886e38
    mask = (torch.arange(T) % 7 != 0).to(torch.uint8)
    mask[5:11] = 1
    l[mask == 0] = float("nan")
    l[0, 3] = float("inf")
    for sigmoid in (False, True):
        for renorm in (False, True):
            idx, w, counts, sums, loss = check(l, K, sigmoid=sigmoid, renorm=renorm, mask=mask)
            assert idx[5].tolist() == list(range(K)) and (w[5] == 0).all()
            assert (w[mask.cuda() == 0] == 0).all()
    check(l, K, sigmoid=True, mask=mask, bias=torch.linspace(-0.1, 0.1, E))
    m = torch.zeros(T, dtype=torch.bool)
    _, w, counts, sums, loss = check(l, K, mask=m)      # every token masked
    assert float(loss) == 0.0 and int(counts.sum()) == 0 and (sums == 0).all() and (w == 0).all()


@pytest.mark.parametrize("E,K", [(40, 8), (128, 8), (256, 8), (256, 20), (320, 12), (1024, 16)])
def test_bias_that_is_not_finite(E, K):
    """A NaN bias counts as -inf, whole lanes of them (neighbours in fours) and all of them
    included; +inf puts an expert first."""
    l = make(50, E, E)
    nan = float("nan")
    for where in (slice(0, 4), slice(0, E, 3), slice(0, E - 1), slice(0, E)):
        bias = torch.linspace(-0.2, 0.2, E)
        bias[where] = nan
        check(l, K, sigmoid=True, bias=bias)
    groups = (torch.arange(E) // 4) % 32 < 6     # every expert of six lanes
    check(l, K, sigmoid=True, bias=torch.linspace(-0.2, 0.2, E).masked_fill(groups, nan))
    shifted = torch.linspace(-0.2, 0.2, E + 1).cuda()[1:]        # not on 16 bytes
    a = sat.router_topk(l.cuda(), K, sigmoid=True, bias=shifted, balance=False)
    b = sat.router_topk(l.cuda(), K, sigmoid=True, bias=shifted.clone(), balance=False)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    bias = torch.linspace(-0.2, 0.2, E)
    bias[E // 2], bias[E // 3], bias[7] = float("inf"), float("inf"), -float("inf")
    assert (check(l, K, sigmoid=True, bias=bias)[0][:, :2].cpu() == torch.tensor([E // 3, E // 2])).all()


def test_no_tokens():
    l = torch.empty((0, 32), device="cuda")
    idx, w, counts, sums, loss = sat.router_topk(l, 4)
    assert idx.shape == (0, 4) and int(counts.abs().sum()) == 0 and float(sums.sum()) == 0 and float(loss) == 0
    assert sat.router_topk_bwd(l, idx, w, counts=counts, grad_loss=loss).shape == (0, 32)
    device_status_ok()


@pytest.mark.parametrize("sigmoid,renorm", [(False, True), (False, False), (True, True), (True, False)])
def test_gradient_against_differences(sigmoid, renorm):
    """Central differences of sum(gw * weights) + gl * loss in 64 bits (ids and counts held,
    as they carry no gradient): their own error is below h^2 * 10 ~ 1e-9."""
    T, E, K, h = 4, 12, 3, 1e-5
    l = make(T, E, 21)
    l64 = l.double().numpy()
    g = np.random.default_rng(1)
    gw, gl = g.standard_normal((T, K)).astype(np.float32), 0.7
    idx, _, counts, _, _ = sat.router_topk(l.cuda(), K, sigmoid=sigmoid, renormalize=renorm, loss_coef=0.5)
    ids, cn = idx.cpu().numpy(), counts.cpu().numpy()

    def value(x):
        r = router(x, K, sigmoid, renorm, loss_coef=0.5)
        pk = np.take_along_axis(r["p"], ids, 1)
        w = pk / (pk.sum(1, keepdims=True) + 1e-20) if renorm else pk
        return (gw * w).sum() + gl * 0.5 * E * K / cn.sum() ** 2 * (cn * r["h"].sum(0)).sum()

    want = np.zeros((T, E))
    for t in range(T):
        for e in range(E):
            a, b = l64.copy(), l64.copy()
            a[t, e] += h
            b[t, e] -= h
            want[t, e] = (value(a) - value(b)) / (2 * h)
    got = sat.router_topk_bwd(l.cuda(), idx, torch.from_numpy(gw).cuda(), counts=counts,
                              grad_loss=torch.tensor([gl]).cuda(), sigmoid=sigmoid, renormalize=renorm, loss_coef=0.5)
    _, mag = router_bwd(l64, ids, gw, cn, gl, sigmoid, renorm, loss_coef=0.5)
    near(got.cpu(), want, 4 * router_units(l64) * U * mag + 1e-8, "gradient")


@pytest.mark.parametrize("E", [16, 48, 100, 200, 600])
def test_row_order_gradient_and_row_weights(E):
    T, K, align = 203, 4, 16
    l = make(T, E, 31)
    idx, w, counts, _, _ = sat.router_topk(l.cuda(), K)
    x = torch.randn((T, 128), device="cuda").to(torch.bfloat16)
    _, _, off, rmap = sat.permute_pad_quant(x, idx, E, align)
    rows = int(off[-1])
    rw = sat.permute_row_weights(w, rmap, rows)
    want = torch.zeros(rows, device="cuda")
    want[rmap.long()] = w.reshape(-1)
    assert torch.equal(rw, want)
    grows = torch.randn(rows, device="cuda")
    a = sat.router_topk_bwd(l.cuda(), idx, grows, row_id_map=rmap)
    b = sat.router_topk_bwd(l.cuda(), idx, grows[rmap.long()].view(T, K))
    assert torch.equal(a, b)
    device_status_ok()
    bad = rmap.clone()
    bad[5], bad[6] = rows, -1
    sat.router_topk_bwd(l.cuda(), idx, grows, row_id_map=bad)
    assert sat.fp8q_last_device_status() == sat.FP8Q_ERR_DEVICE
    out = sat.permute_row_weights(w, bad, rows)
    assert sat.fp8q_last_device_status() == sat.FP8Q_ERR_DEVICE
    want[rmap.long()[5:7]] = 0
    assert torch.equal(out, want)


@pytest.mark.parametrize("E,K", [(32, 8), (64, 8), (64, 40), (128, 33), (200, 8), (256, 40), (600, 40)])
def test_repeated_and_bad_ids_in_the_backward(E, K):
    """Ids that a caller made: a repeated one adds up, one out of range is skipped."""
    T = 9
    l = make(T, E, 41)
    idx = torch.stack([torch.randperm(E, generator=torch.Generator().manual_seed(t))[:K] for t in range(T)]).int()
    idx[0] = 5
    idx[1, 0] = idx[1, K - 1]
    gw = torch.randn((T, K), generator=torch.Generator().manual_seed(2))
    got = sat.router_topk_bwd(l.cuda(), idx.cuda(), gw.cuda())
    device_status_ok()
    want, mag = router_bwd(l.numpy(), idx.numpy().astype(np.int64), gw.numpy(), None, None)
    near(got.cpu(), want, 4 * (router_units(l.numpy()) + K) * U * mag + 1e-30, "gradient")
    idx[2, 1], idx[3, 2] = E, -1
    sat.router_topk_bwd(l.cuda(), idx.cuda(), gw.cuda())
    assert sat.fp8q_last_device_status() == sat.FP8Q_ERR_DEVICE


@pytest.mark.parametrize("E", [64, 256])
def test_same_bits_every_time_and_under_capture(E):
    """Two runs, two streams with their own workspaces, and a captured and replayed step on
    new inputs give the same bits."""
    T, K = 20011, 6
    a, b = make(T, E, 51).cuda(), make(T, E, 52).cuda()
    gl, gw = torch.ones(1, device="cuda"), torch.randn((T, K), device="cuda")

    def step(x, **o):
        r = sat.router_topk(x, K, **o)
        return [*r, sat.router_topk_bwd(x, r[0], gw, counts=r[2], grad_loss=gl, **o)]

    want = {k: step(x) for k, x in (("a", a), ("b", b))}
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(s1):
            r1 = step(a)
        with torch.cuda.stream(s2):
            r2 = step(b)
        r3 = step(a, stream=s1)  # a stream other than the current one
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(r1, want["a"]))
        assert all(torch.equal(x, y) for x, y in zip(r2, want["b"]))
        assert all(torch.equal(x, y) for x, y in zip(r3, want["a"]))
    x = a.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = step(x)
    for k, src in (("b", b), ("a", a)):
        x.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(r, want[k]))
    device_status_ok()


def test_wrong_tensors_are_refused():
    l = make(8, 32, 1).cuda()
    idx, w, counts, _, loss = sat.router_topk(l, 4)
    for bad in (lambda: sat.router_topk(l.double(), 4), lambda: sat.router_topk(l[:, ::2], 4),
                lambda: sat.router_topk(l.cpu(), 4), lambda: sat.router_topk(l, 4, token_mask=torch.ones(7, device="cuda")),
                lambda: sat.router_topk_bwd(l, idx, w[:4]), lambda: sat.router_topk_bwd(l, idx.long(), w),
                lambda: sat.router_topk_bwd(l, idx, w, row_id_map=idx[:2]), lambda: sat.permute_row_weights(w, idx[:3], 9)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(sat.Fp8qError):
        sat.router_topk(l, 33)
    with pytest.raises(sat.Fp8qError):
        sat.router_topk(l, 4, bias=torch.zeros(32, device="cuda"))  # a bias needs sigmoid scores


@pytest.mark.parametrize("E,K", [(72, 6), (256, 8), (500, 16), (1000, 3)])
def test_scores_apart_by_less_than_fp32_errors(E, K):
    """Clusters of scores 2^-24 to 2^-30 apart around the border of the choice, beside well
    separated rows: fp32 scores alone would order some of them wrongly."""
    g = torch.Generator().manual_seed(E)
    T = 700
    l = make(T, E, E + 1)
    near_l = 0.3 + torch.randint(0, 64, (T, E), generator=g).float() * 2.0 ** -25
    rows = torch.arange(T) % 3 != 0
    pick = torch.rand((T, E), generator=g) < 20.0 / E
    l = torch.where(rows[:, None] & pick, near_l, l.clamp_max(0.2))
    for scale in (0.0, 2.0 ** -26, 0.1):
        bias = torch.randn(E, generator=g) * scale
        check(l, K, sigmoid=True, bias=bias)
    check(l, K, sigmoid=True, bias=torch.full((E,), 3.0e4))   # sums that lose the low bits of the scores
    check(l, K, sigmoid=True)
    check(l, K)
