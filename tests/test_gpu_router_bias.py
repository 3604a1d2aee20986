"""The router's choice under a selection bias: experts that a logit of -inf (or NaN) switches
off come after every other, whatever their bias, in each of the kernels, on the fp32 scores'
way and on the exact one, with few and many slots; and scores are told apart down to the last
bit of their double sums.

The wanted ids are found here from the definition, by (off, -score, id) with the score
1 / (1 + exp(-l)) + bias in float64; the weights' bound is that of test_gpu_router."""
import numpy as np
import pytest
import torch

import scaling_aware_transpose_b200 as sat
from gpu_helpers import device_status_ok
from moe_reference import U, clean, router_units

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")
EXPERTS = [5, 32, 33, 64, 100, 128, 129, 200, 256, 300, 512, 600, 1024]


def chosen(l, bias, K):
    l = clean(l)
    with np.errstate(over="ignore"):
        score = 1.0 / (1.0 + np.exp(-l)) + np.asarray(bias, np.float64)
    score = np.where(np.isnan(score), -np.inf, score)
    return np.lexsort((-score, np.isneginf(l)), axis=1)[:, :K]


def make(T, E, seed):
    return torch.randn((T, E), generator=torch.Generator().manual_seed(seed)) * 1.5


def check(l, bias, K, mask=None, renorm=True):
    """The call with and without statistics: ids, counts and weights."""
    host = l.float().numpy()
    want = chosen(host, bias.numpy(), K)
    live = np.ones(len(host), bool) if mask is None else mask.numpy() != 0
    opt = dict(sigmoid=True, renormalize=renorm, bias=bias.cuda(), token_mask=None if mask is None else mask.cuda())
    idx, w, counts, sums, loss = sat.router_topk(l.cuda(), K, **opt)
    idx2, w2, *_ = sat.router_topk(l.cuda(), K, balance=False, **opt)
    device_status_ok()
    assert torch.equal(idx, idx2) and torch.equal(w, w2)
    bad = np.argwhere(idx.cpu().numpy() != want)
    assert not len(bad), f"ids at {bad[:4].tolist()}: {idx.cpu().numpy()[bad[0][0]]}, not {want[bad[0][0]]}"
    assert np.array_equal(counts.cpu().numpy(), np.bincount(want[live].reshape(-1), minlength=l.shape[1]))
    with np.errstate(over="ignore"):
        p = np.take_along_axis(1.0 / (1.0 + np.exp(-clean(host))), want, 1)
    ww = np.where(live[:, None], p / (p.sum(1, keepdims=True) + 1e-20) if renorm else p, 0.0)
    off = np.abs(w.double().cpu().numpy() - ww)
    assert (off <= 2 * router_units(host) * U * ww + 1e-30).all(), off.max()
    assert torch.isfinite(sums).all() and torch.isfinite(loss).all()
    return want


@pytest.mark.parametrize("E", EXPERTS)
@pytest.mark.parametrize("top", [0.5, 3.0e4, INF])
def test_a_large_bias_does_not_bring_an_expert_back(E, top):
    """Off experts with the largest biases of all, beside enough others: none is chosen, none
    is counted.  NaN logits switch off as -inf does."""
    T = 203
    l, g = make(T, E, E), torch.Generator().manual_seed(E + 1)
    bias = torch.randn(E, generator=g) * 0.1
    off = torch.randperm(E, generator=g)[:max(1, E // 3)]
    bias[off] = top
    l[:, off] = -INF
    l[::3, off] = NAN
    for K in {1, min(3, E - len(off)), min(8, E - len(off)), min(20, E - len(off))}:
        want = check(l, bias, K)
        assert not np.isin(want, off.numpy()).any()
    check(l.to(torch.bfloat16), bias, min(3, E - len(off)), renorm=False)


@pytest.mark.parametrize("E", EXPERTS)
def test_off_experts_fill_up_behind_all_others(E):
    """Fewer others than slots, rows with different numbers of them (none among these): the
    others first, by score, those with a bias of -inf or NaN too; then off experts, by bias.
    Masked rows of NaN lie between."""
    T, g = 181, torch.Generator().manual_seed(E + 2)
    l = make(T, E, E + 3)
    bias = torch.randn(E, generator=g) * 0.1
    bias[E // 2], bias[E - 1] = -INF, NAN
    left = torch.randint(0, 12, (T,), generator=g)
    for t in range(T):
        l[t, torch.randperm(E, generator=g)[int(left[t]):]] = -INF
    mask = (torch.arange(T) % 5 != 0).to(torch.uint8)
    l[mask == 0] = NAN
    for K in {min(5, E), min(8, E), min(24, E), min(64, E)}:
        check(l, bias, K, mask)
        check(l, torch.zeros(E), K, mask, renorm=False)


@pytest.mark.parametrize("E", EXPERTS)
def test_rows_with_nothing_left(E):
    """Every expert off: weights 0, ids by bias, the lowest first where biases are equal."""
    l = torch.full((9, E), -INF)
    l[2:4] = NAN
    K = min(6, E)
    bias = torch.zeros(E)
    assert (check(l, bias, K) == np.arange(K)).all()
    bias[E // 2], bias[E - 1] = 0.3, 0.01
    assert (check(l, bias, K)[:, :2] == [E // 2, E - 1]).all()
    check(l, torch.linspace(-0.1, 0.1, E).flip(0), K)
    assert (sat.router_topk(l.cuda(), K, sigmoid=True, bias=bias.cuda())[1] == 0).all()


def test_the_lowest_finite_logits_are_not_off():
    """The lowest values of the types are scores of 0, to which a bias may add."""
    for E in (32, 100, 256, 600):
        for low in (torch.finfo(torch.float32).min, torch.finfo(torch.bfloat16).min):
            l = make(50, E, 1)
            l[:, 3] = low
            l[:, 4] = -INF
            bias = torch.zeros(E)
            bias[3:5] = 2.0
            assert (check(l, bias, 3)[:, 0] == 3).all()


@pytest.mark.parametrize("E,K", [(60, 8), (128, 8), (200, 8), (256, 20), (500, 16), (1000, 33)])
def test_scores_one_bit_apart(E, K):
    """Equal logits and biases of whole multiples of 2^-52: p + bias is exact in double (p in
    [0.5, 1) has a last bit of 2^-53), so the multiples alone order the experts; equal ones by
    the lowest id.  The last row's p in [2^-3, 2^-2), where twice as much of the sum lies beyond
    a pair of fp32 values."""
    g = torch.Generator().manual_seed(E)
    steps = torch.randint(0, 8, (E,), generator=g)
    want = np.lexsort((-steps.numpy(),))[:K]
    bias = steps.double().mul(2.0 ** -52).float()
    for x in (0.405465, 0.1, 1.7, 3.3, -1.7):
        l = torch.full((6, E), x)
        assert (check(l, bias, K) == want).all()
        assert (sat.router_topk(l.cuda(), K, sigmoid=True, bias=bias.cuda())[0].cpu().numpy() == want).all()
