"""Host side of the router: the workspace for few and very many tokens, the order of the reference."""
import numpy as np

import scaling_aware_transpose_b200 as sat
from moe_reference import router


def rows(tokens, experts):
    return (sat.fp8q_router_workspace_bytes(tokens, experts) - 16) / (8 * experts)


def test_workspace_of_launches_of_256_rounds():
    """A row per CTA: up to 592 (296 above 256 experts) a launch, a launch per 256 rounds of
    eight warps of one, two or four tokens."""
    for experts, most, per in ((32, 592, 32), (64, 592, 32), (128, 592, 16), (129, 592, 8), (256, 592, 8), (257, 296, 8),
                               (1024, 296, 8)):
        full = 256 * most * per
        assert rows(full, experts) == most
        assert rows(full + 1, experts) == most + 1
        assert rows(2 * full, experts) == 2 * most
        assert rows(2 * full + per * 5, experts) == 2 * most + 5
        assert rows(most * per * 3, experts) == most
        assert rows(per * 20, experts) == 20
        assert sat.fp8q_router_workspace_bytes(per * 16, experts) == 16  # one cluster, no rows


def test_reference_order_of_experts_that_are_off():
    """The 64-bit reference that the kernels are held to: off experts behind all others, whatever
    their bias; among themselves by the bias, then by the lowest id; a score of -inf before them."""
    inf, nan = np.inf, np.nan
    l = np.array([[0.1, -inf, 0.3, -inf, -2.0, nan], [-inf] * 6, [0.0, -inf, -inf, 1.0, -inf, -inf]])
    bias = np.array([0.0, 5.0, 0.0, 0.2, -0.1, 0.2])
    assert router(l, 6, sigmoid=True, bias=bias)["idx"].tolist() == [[2, 0, 4, 1, 3, 5], [1, 3, 5, 0, 2, 4], [3, 0, 1, 5, 2, 4]]
    bias[3], bias[0] = -inf, nan
    assert router(l[2:], 6, sigmoid=True, bias=bias)["idx"].tolist() == [[0, 3, 1, 5, 2, 4]]
    r = router(l[:1], 3, sigmoid=True, bias=bias)
    assert r["counts"].tolist() == [1, 0, 1, 0, 1, 0]
    assert router(l[1:2], 3, sigmoid=True, bias=np.zeros(6))["idx"].tolist() == [[0, 1, 2]]
    assert router(l[1:2], 3)["idx"].tolist() == [[0, 1, 2]]
