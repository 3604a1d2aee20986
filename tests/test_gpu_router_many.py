"""Balance statistics over millions of tokens with one share each, the worst there is for sums
in fp32: each addition of the same value to a sum in the same binade rounds the same way.

A lane adds at most 256 shares one after the other; 8 warps and 4 groups of lanes come on top,
each addition within half a step U of the sum, the rest is in double; a share is off by the
2 * 49 half steps of moe_reference.router_units for equal logits.  (n tokens a lane: 8 a CTA from
129 experts on, 592 CTAs up to 256 experts; 16 or 32 a CTA below.)"""
import numpy as np
import pytest
import torch

import scaling_aware_transpose_b200 as sat
from gpu_helpers import device_status_ok
from moe_reference import U

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("E,per_cta", [(5, 32), (51, 32), (127, 16), (160, 8), (255, 8)])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_sums_of_equal_shares(E, per_cta, sigmoid):
    n = 6000 if E <= 64 else 3000       # tokens a lane
    T = n * 592 * per_cta + 77
    free = torch.cuda.mem_get_info()[0]
    if free < T * (2 * E + 16) + (1 << 30):
        pytest.skip("too little memory")
    l = torch.zeros((T, E), dtype=torch.bfloat16, device="cuda")
    idx, w, counts, sums, loss = sat.router_topk(l, 1, sigmoid=sigmoid)
    device_status_ok()
    assert counts.tolist() == [T] + [0] * (E - 1)
    tol = (256 + 12 + 2 * 49) * U * T / E
    off = np.abs(sums.double().cpu().numpy() - T / E)
    assert (off <= tol).all(), (off.max() / (T / E), tol / (T / E))
    assert abs(float(loss) - 1.0) <= (256 + 14 + 2 * 49) * U  # E / T^2 * T * T / E
    mask = torch.zeros(T, dtype=torch.uint8, device="cuda")
    mask[::3] = 1
    live = int(mask.sum())
    sums = sat.router_topk(l, 1, sigmoid=sigmoid, token_mask=mask)[3]
    off = np.abs(sums.double().cpu().numpy() - live / E)
    assert (off <= (256 + 12 + 2 * 49) * U * live / E).all(), off.max() / (live / E)


def test_few_rounds_and_many_agree():
    """Sums over 300 rounds a lane (two launches) against those of its parts, and each token's own
    results."""
    E, T = 200, 592 * 8 * 300
    g = torch.Generator(device="cuda").manual_seed(1)
    l = torch.randn((T, E), generator=g, device="cuda").to(torch.bfloat16)
    idx, w, counts, sums, _ = sat.router_topk(l, 4)
    sums = sums.double()
    calls = [sat.router_topk(c, 4) for c in l.split(T // 20)]
    assert torch.equal(idx, torch.cat([c[0] for c in calls])) and torch.equal(w, torch.cat([c[1] for c in calls]))
    assert torch.equal(counts, sum(c[2] for c in calls))
    parts = sum(c[3].double() for c in calls)
    want = torch.softmax(l.double(), 1).sum(0)
    n = 2 * 75 + 256 + 14               # 2 * router_units at a span of logits below 26, and the additions
    assert ((sums - want).abs() <= n * U * want).all() and ((parts - want).abs() <= n * U * want).all()
    device_status_ok()


def test_several_launches_under_capture():
    """A call of two launches captured once and replayed on other logits gives the same bits."""
    E, K, T = 160, 2, 592 * 8 * 256 + 5000
    g = torch.Generator(device="cuda").manual_seed(2)
    a, b = (torch.randn((T, E), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    want = {k: [t.clone() for t in sat.router_topk(x, K)] for k, x in (("a", a), ("b", b))}
    buf = a.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = sat.router_topk(buf, K)
    for k, x in (("b", b), ("a", a)):
        buf.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(got, want[k])), k
    device_status_ok()
