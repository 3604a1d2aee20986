"""The E4M3 form of the SwiGLU backward where a tile's values are tiny before their scales are
applied: saturated gates, gradients near the bottom of BF16, with factors (scale times row
weight) of 2 and more.  No code is a NaN and each pair is within test_gpu_swiglu_bwd's bounds
of the 64-bit formulas (its e_dg, e_du, e_y and half a step of E4M3)."""
import numpy as np
import pytest
import torch

import scaling_aware_transpose_b200 as sat
from gpu_helpers import device_status_ok
from moe_reference import decode8, swiglu_bwd
from test_gpu_swiglu_bwd import near_pair, normal, stash

pytestmark = pytest.mark.gpu


def check(gq, gsf, uq, usf, dy, w):
    wd = None if w is None else w.cuda()
    r = swiglu_bwd(decode8(gq.numpy(), gsf.numpy()), decode8(uq.numpy(), usf.numpy()), dy.double().numpy(),
                   None if w is None else w.numpy())
    p = sat.swiglu_bwd_quant(*[t.cuda() for t in (gq, gsf, uq, usf, dy)], row_weights=wd)
    device_status_ok()
    for i, k in enumerate(("dg", "du", "y")):
        assert (p[2 * i] & 0x7F != 0x7F).all(), f"{k}: {int((p[2 * i] & 0x7F == 0x7F).sum())} NaN codes"
        near_pair(p[2 * i], p[2 * i + 1], r[k], r["e_" + k] + np.abs(r[k]) * 2.0 ** -24, k)
    return p


@pytest.mark.parametrize("last", [-72.0, -80.0, -84.0, -88.0, -96.0])
@pytest.mark.parametrize("weight", [None, 0.25, 1.0, 3.0, -700.0])
def test_saturated_gates(last, weight):
    """Gates about -1000, one much nearer: s is 0 but there."""
    rows, cols = 3, 256
    gate = torch.full((rows, cols), -1000.0)
    gate[0, 5], gate[1, 200], gate[2, :128] = last, last, last
    gq, gsf = [t.cpu() for t in sat.quantize_rowwise(gate.to(torch.bfloat16).cuda())]
    uq, usf = [t.cpu() for t in sat.quantize_rowwise((normal(rows, cols, 1) * 300).cuda())]
    dy = normal(rows, cols, 2, 1e-3)
    dy[:, 3] = 0
    check(gq, gsf, uq, usf, dy, None if weight is None else torch.full((rows,), weight))


@pytest.mark.parametrize("size", [1e-33, 1e-36, 1e-37, 1e-38, 3e-39, 1e-39, 1e-40])
@pytest.mark.parametrize("weight", [None, 2.0, 1000.0, -5.0e5])
def test_gradients_at_the_bottom_of_the_range(size, weight):
    rows, cols = 9, 640
    gq, gsf, uq, usf = stash(rows, cols, 7)
    uq[4:], usf[4:] = [t[4:].cpu() for t in sat.quantize_rowwise((normal(rows, cols, 3) * 3000).cuda())]
    dy = (normal(rows, cols, 4, 1.0, 0.0).float() * size).to(torch.bfloat16)
    dy[:, 1::7] = 0
    dy[2, :128] = 0
    check(gq, gsf, uq, usf, dy, None if weight is None else torch.full((rows,), weight))


def test_largest_gate_with_large_up():
    """Scales whose product passes fp32 where the tile's values are 0: codes of 0."""
    rows, cols = 2, 128
    gate = torch.full((rows, cols), torch.finfo(torch.bfloat16).min, dtype=torch.bfloat16)
    up = torch.full((rows, cols), 3.0e6, dtype=torch.bfloat16)
    _, _, *s = sat.swiglu_quant_stash(gate.cuda(), up.cuda())
    p = sat.swiglu_bwd_quant(*s, torch.ones((rows, cols), dtype=torch.bfloat16, device="cuda"))
    device_status_ok()
    for q in (p[0], p[2], p[4]):
        assert (q & 0x7F == 0).all(), hex(int(q[0, 0]))
