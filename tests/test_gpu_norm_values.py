"""The group norm and its gradients where addresses and values are unusual, against float64
(oracle.served)."""
import numpy as np
import pytest
import torch

import mamba_ssd_scan_03_b200 as ssd
from oracle import served
from served_util import U, down, excess, store, up, up_rows
from test_gpu_norm import chain, fwd_bound, inputs

pytestmark = pytest.mark.gpu

UNSUPPORTED = 2


def flat(a, at):
    """The values `at` floats into a longer buffer, as parameters in one flat tensor lie."""
    big = torch.full((len(a) + at + 5,), 3.0, device="cuda")
    big[at:at + len(a)] = up(a)
    return big[at:at + len(a)]


# groups of every wide variant (lanes of a warp, a warp, a CTA), and of the largest narrow one
@pytest.mark.parametrize("rows,C,groups", [(5, 64, 1), (300, 64, 8), (7, 256, 1), (9, 768, 1),
                                           (9, 1024, 1), (33, 2048, 1), (40, 5120, 8),
                                           (3, 5120, 1), (2, 8192, 1)])
@pytest.mark.parametrize("at", [1, 2, 3, 4])
def test_weight_of_any_alignment(rows, C, groups, at):
    """Weight and bias `at` floats into a flat parameter buffer, rows on 16-byte boundaries."""
    g = inputs(rows, C, "f32", "bf16", seed=at)
    w, b = flat(g["w"], at), flat(g["b"], at)
    y, z = up_rows(g["y"]), up_rows(g["z"], "bf16")
    f = served.group_norm(g["y"], g["w"], g["b"], g["z"], groups)
    out = ssd.group_norm_gate(y, w, b, z, groups)
    assert excess(down(out), f["out"], fwd_bound(g, f, groups, True, "f32")) <= 0
    do = store(np.random.default_rng(2).standard_normal((rows, C)), "bf16")
    got = ssd.group_norm_gate_bwd(up(do, "bf16"), y, w, b, z, groups)
    ref = served.group_norm_backward(do, g["y"], g["w"], g["b"], g["z"], groups)
    # steps as in test_norm_gradients
    steps = 2 * chain(C, groups) + 32 + 4 * float(np.max(np.abs(down(z))))
    assert excess(down(got["y"]), ref["y"], steps * U * (ref["scale"] + 1e-30)) <= 0
    for k in ("weight", "bias"):
        assert excess(down(got[k]), ref[k], (steps + rows) * U * ref[k + "_scale"]) <= 0
    assert ssd.device_status() == 0


def test_wide_groups_need_an_aligned_weight():
    """Past 8192 channels a group asks for 16-byte addresses, the weight's among them."""
    g = inputs(2, 16384, "f32", "f32")
    y, z, do = up(g["y"]), up(g["z"]), up(g["y"])
    for at in (1, 2, 3):
        w = flat(g["w"], at)
        for call in (lambda: ssd.group_norm_gate(y, w, None, z),
                     lambda: ssd.group_norm_gate_bwd(do, y, w, None, z)):
            with pytest.raises(ssd.SSDError) as e:
                call()
            assert e.value.code == UNSUPPORTED
    w = flat(g["w"], 4)
    assert torch.equal(ssd.group_norm_gate(y, w, None, z),
                       ssd.group_norm_gate(y, up(g["w"]), None, z))
    assert ssd.device_status() == 0
