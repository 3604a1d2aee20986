"""Host side of the router's statistics: the workspace for few and very many tokens."""
import scaling_aware_transpose_b200 as sat


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
