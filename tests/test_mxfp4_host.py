"""Which kernel a 4-bit product takes (host only): that the sizes of the GPU tests reach the
kernels that they are there for, on the 148 SMs of a B200, and the refusals of the hook."""
import ctypes

import pytest

import scaling_aware_transpose_b200 as sat
import test_gpu_mxfp4
from mxfp4_sizes import DENSE_WALKS, EVERY, GROUPED


def variant(m, n, k, groups=0):
    return sat.fp8q_debug_mxfp4_variant(m, n, k, groups, 148)


def listed(test):
    return [m.args[1] for m in test.pytestmark if m.name == "parametrize"][0]


def tiles(m, n, columns):
    return (m + 127) // 128 * ((n + columns - 1) // columns)


@pytest.mark.parametrize("m,n,k,want", DENSE_WALKS)
def test_dense_walks(m, n, k, want):
    assert variant(m, n, k) == want and tiles(m, n, want[0]) > 148


@pytest.mark.parametrize("sizes,n,k,more,want", GROUPED)
def test_grouped(sizes, n, k, more, want):
    assert variant(sum(sizes) + more, n, k, len(sizes)) == want


def test_every_kernel_is_reached():
    dense = [*listed(test_gpu_mxfp4.test_product_by_every_tile_width), *listed(test_gpu_mxfp4.test_product_by_pairs)]
    assert {variant(*c) for c in dense} == EVERY
    old = {variant(sum(s) + more, n, k, len(s)) for s, n, k, more in listed(test_gpu_mxfp4.test_grouped_by_every_kernel)}
    assert old | {c[-1] for c in GROUPED} == EVERY
    walks = {c[-1] for c in GROUPED if c[-1][0] and c[-1][1] == 1 and tiles(sum(c[0]), c[1], c[-1][0]) > 148}
    assert walks == {(32, 1), (64, 1), (128, 1), (256, 1)}


def test_refusals():
    c, s = ctypes.c_int32(), ctypes.c_int32()
    f = sat.lib().fp8q_debug_mxfp4_variant
    for bad in ((0, 1, 128, 0, 148), (1, 0, 128, 0, 148), (1, 1, 100, 0, 148), (1, 1, 0, 0, 148), (1, 1, 128, -1, 148),
                (1, 1, 128, 0, 1)):
        assert f(*bad, c, s) == sat.FP8Q_ERR_ARG, bad
    assert f(1, 1, 128, 0, 148, None, s) == sat.FP8Q_ERR_NULL
