"""4-bit products where a CTA walks over several tiles, at every tile width, and the grouped
variants with shared k: against 64-bit sums with the bound of moe_reference.matmul_bound.  On a
GPU of 148 SMs the kernel that each size is there for is the one that runs."""
import numpy as np
import pytest
import torch

import scaling_aware_transpose_b200 as sat
from gpu_helpers import device_status_ok
from moe_reference import matmul_bound
from mxfp4_sizes import DENSE_WALKS, GROUPED
from test_gpu_mxfp4 import near, operand

pytestmark = pytest.mark.gpu


def takes(m, n, k, groups, want):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert sms != 148 or sat.fp8q_debug_mxfp4_variant(m, n, k, groups, sms) == want


@pytest.mark.parametrize("m,n,k,want", DENSE_WALKS)
def test_dense_walks(m, n, k, want):
    takes(m, n, k, 0, want)
    aq, asf, a = operand(m, k, m, 3)
    bq, bsf, b = operand(n, k, n, 3)
    buf = torch.full((m * n + 64,), 7.0, dtype=torch.bfloat16, device="cuda")
    out = sat.matmul_mxfp4(aq, asf, bq, bsf, out=buf[:m * n].view(m, n))
    device_status_ok()
    want, tol = matmul_bound(a, b)
    near(out, want, tol, f"{m}x{n}x{k}")
    assert (buf[m * n:] == 7.0).all()
    first = out.clone()
    for _ in range(3):
        assert torch.equal(sat.matmul_mxfp4(aq, asf, bq, bsf), first)


@pytest.mark.parametrize("sizes,n,k,more,want", GROUPED, ids=lambda v: f"{len(v)}groups" if isinstance(v, list) else str(v))
def test_grouped(sizes, n, k, more, want):
    G, rows = len(sizes), sum(sizes)
    cap = rows + more
    takes(cap, n, k, G, want)
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
    again = torch.full_like(out, 7.0)
    sat.matmul_mxfp4(aq, asf, bq, bsf, group_offsets=off, out=again)
    assert torch.equal(again, out)
