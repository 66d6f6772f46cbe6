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


def slope_bound(z):
    """silu' = sg + g (1 - sg), g = z sg, from sg = 1 / (1 + e), e = e^-z.  e is off by
    (2 |z| + 8) u of itself (its argument's two roundings, its own 2^-22), sg by ea = (1 - sg) that +
    4 u (the sum, the reciprocal's 2^-23), 1 - sg by sg ea + u (1 - sg), g by ea + u, the last step by
    u.  From z = 20 on the sum is 1, and so are sg and silu' for certain."""
    z = np.asarray(z, np.float64)
    sg = 1.0 / (1.0 + np.exp(np.minimum(-z, 700.0)))
    g = np.abs(z) * sg
    ea = (1 - sg) * (2 * np.abs(z) + 8) * U + 4 * U
    e = sg * ea + g * ((ea + U) * (1 - sg) + sg * ea + U * (1 - sg))
    e = np.where(z >= 20, 0.0, e)
    return e + U * np.abs(sg + z * sg * (1 - sg))


BIG_GATES = [-1e30, -3e7, -100.0, -90.0, -30.0, -12.0, -4.0, -1.3, -1.0, -0.1, 0.0, 0.5, 1.0, 4.0,
             8.0, 9.5, 11.0, 12.0, 16.0, 20.0, 25.0, 88.0, 1e3, 1.7e7, 3e7, 3e8, 1e30]


@pytest.mark.parametrize("C", [64, 37])
def test_slope_of_large_gates(C):
    """dz where the gate is far from zero: with an upstream gradient and a normalised value that are
    exactly known, dz is silu' itself.  One channel per group, centred: the value is its own mean, the
    output is the bias (1), and dz = dout silu'(z)."""
    z = np.resize(np.float32(BIG_GATES), (3, C))
    y = np.random.default_rng(0).standard_normal((3, C)).astype(np.float32)
    one = torch.ones(C, device="cuda")
    got = ssd.group_norm_gate_bwd(up(np.ones((3, C), np.float32)), up(y), one, one, up(z), C, 1e-5,
                                  True, False)
    zd = z.astype(np.float64)
    sg = 1.0 / (1.0 + np.exp(np.minimum(-zd, 700.0)))
    ref = sg * (1 + zd * (1 - sg))
    assert excess(down(got["z"]), ref, slope_bound(zd) + 2.0 ** -126 * (1 + np.abs(zd))) <= 0
    assert ssd.device_status() == 0


@pytest.mark.parametrize("C,groups", [(64, 1), (64, 8), (37, 1), (1024, 1)])
def test_gradients_of_a_saturated_gate(C, groups):
    """Gates of 2^24 and more ahead of the norm: silu is z, silu' is 1, and dz = dv y."""
    r = np.random.default_rng(3)
    z = np.exp(r.uniform(np.log(2.0 ** 24), np.log(2.0 ** 30), (5, C))).astype(np.float32)
    y = r.standard_normal((5, C)).astype(np.float32)
    do = r.standard_normal((5, C)).astype(np.float32)
    w = (1 + 0.2 * r.standard_normal(C)).astype(np.float32)
    got = ssd.group_norm_gate_bwd(up(do), up(y), up(w), None, up(z), groups)
    ref = served.group_norm_backward(do, y, w, None, z, groups)
    # as in test_norm_gradients, with silu and silu' exact: no steps of the gate's
    steps = 2 * chain(C, groups) + 32
    assert excess(down(got["y"]), ref["y"], steps * U * ref["scale"]) <= 0
    assert excess(down(got["z"]), ref["z"], steps * U * ref["mag"] * np.abs(y)) <= 0
    assert ssd.device_status() == 0
