"""GPU parity of the group norm with its SiLU gate and of its gradients against float64
(oracle.served), within bounds that count roundings (served_util)."""
import numpy as np
import pytest
import torch

import mamba_ssd_scan_03_b200 as ssd
from oracle import glue, served
from served_util import BF16, U, down, excess, store, up, up_rows

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
# rows, channels, groups: team of lanes, of a warp, of a CTA; odd widths; one row, one channel
SHAPES = [(5, 64, 1), (300, 64, 8), (7, 256, 1), (33, 512, 2), (9, 1024, 1), (3, 5120, 1),
          (40, 5120, 8), (2, 8192, 1), (1, 16384, 1), (6, 37, 1), (11, 111, 3), (4, 1537, 1),
          (3, 2600 * 2 + 2, 2), (2, 8191, 1), (17, 1, 1), (5, 6, 6), (150, 24, 1)]


def inputs(rows, C, y_io, z_io, seed=0, shift=0.0):
    r = np.random.default_rng(seed)
    return dict(y=store(r.standard_normal((rows, C)) + shift, y_io),
                z=None if z_io is None else store(2 * r.standard_normal((rows, C)), z_io),
                w=(1 + 0.2 * r.standard_normal(C)).astype(np.float32),
                b=r.standard_normal(C).astype(np.float32))


def chain(C, groups):
    """Roundings of a sum over a group: at most 32 terms one after another in a lane (16 units of
    ... channels), then 10 levels; 64 counts both."""
    return 64


def fwd_bound(g, f, groups, gate_first, o_io):
    """v (the gate's silu: |z| + 8 steps), its mean (the chain's error of the mean magnitude), the
    mean square (chain), rstd (4 steps), the products: relative to |v|, |mean| as they stand before
    they cancel."""
    z = None if g["z"] is None else np.abs(glue._f64(g["z"]))
    rows, C = f["v"].shape
    steps = chain(C, groups) + 16 + (0 if z is None else 2 * float(np.max(z)) + 16)
    grp = f["v"].reshape(rows, groups, -1)
    avg = np.broadcast_to(np.mean(np.abs(grp), -1, keepdims=True), grp.shape).reshape(rows, C)
    mag = (np.abs(f["v"]) + avg * (np.abs(f["mean"]) > 0) + np.abs(f["n"]) / f["rstd"]) \
        * f["rstd"] * np.abs(g["w"]) + np.abs(g["b"] if g["b"] is not None else 0)
    if z is not None and not gate_first:
        mag = mag * np.abs(glue.silu(glue._f64(g["z"])))
    b = steps * U * mag
    return b + BF16[o_io] * (np.abs(f["out"]) + b)


@pytest.mark.parametrize("rows,C,groups", SHAPES)
@pytest.mark.parametrize("y_io,z_io,o_io,center,gate_first,bias,pad,shift", [
    ("f32", "bf16", "bf16", False, True, False, 0, 0),
    ("f32", "f32", "f32", True, True, True, 8, 8),
    ("bf16", "bf16", "bf16", False, False, True, 1, 3),
    ("bf16", None, "f32", True, True, True, 0, 0)])
def test_norm(rows, C, groups, y_io, z_io, o_io, center, gate_first, bias, pad, shift):
    if C > 8192 and (pad or shift) % 8:
        pytest.skip("refused: groups past 8192 channels need aligned rows (test_norm_refuses)")
    g = inputs(rows, C, y_io, z_io, shift=0.5 if center else 0.0)
    if not bias:
        g["b"] = None
    out = up_rows(store(np.zeros((rows, C)), o_io), o_io, pad, shift)
    ssd.group_norm_gate(up_rows(g["y"], y_io, pad, shift), up(g["w"]),
                        None if g["b"] is None else up(g["b"]),
                        None if z_io is None else up_rows(g["z"], z_io, pad, shift), groups, 1e-5,
                        center, gate_first, out=out)
    f = served.group_norm(g["y"], g["w"], g["b"], g["z"], groups, 1e-5, center, gate_first)
    assert excess(down(out), f["out"], fwd_bound(g, f, groups, gate_first, o_io)) <= 0
    assert ssd.device_status() == 0


@pytest.mark.parametrize("rows,C,groups", SHAPES)
@pytest.mark.parametrize("y_io,z_io,d_io,center,gate_first,bias,pad,shift", [
    ("f32", "bf16", "bf16", False, True, False, 0, 0),
    ("f32", "f32", "f32", True, True, True, 8, 8),
    ("bf16", "bf16", "f32", False, False, True, 1, 3),
    ("bf16", None, "f32", True, True, True, 0, 0)])
def test_norm_gradients(rows, C, groups, y_io, z_io, d_io, center, gate_first, bias, pad, shift):
    if C > 8192 and (pad or shift) % 8:
        pytest.skip("refused: groups past 8192 channels need aligned rows (test_norm_refuses)")
    g = inputs(rows, C, y_io, z_io, seed=1, shift=0.5 if center else 0.0)
    if not bias:
        g["b"] = None
    do = store(np.random.default_rng(2).standard_normal((rows, C)), d_io)
    got = ssd.group_norm_gate_bwd(
        up_rows(do, d_io, pad, shift), up_rows(g["y"], y_io, pad, shift), up(g["w"]),
        None if g["b"] is None else up(g["b"]),
        None if z_io is None else up_rows(g["z"], z_io, pad, shift), groups, 1e-5, center,
        gate_first)
    ref = served.group_norm_backward(do, g["y"], g["w"], g["b"], g["z"], groups, 1e-5, center,
                                     gate_first)
    zmax = 0.0 if z_io is None else float(np.max(np.abs(glue._f64(g["z"]))))
    steps = 2 * chain(C, groups) + 32 + 4 * zmax
    # one channel per group: y is its own mean and everything cancels to eps; the bound's
    # magnitudes stand before that
    mag = steps * U * (ref["scale"] + 1e-30)
    assert excess(down(got["y"]), ref["y"], mag) <= 0
    if z_io is not None:
        yv = np.abs(glue._f64(g["y"]))
        f = served.group_norm(g["y"], g["w"], g["b"], g["z"], groups, 1e-5, center, gate_first)
        # silu' is at most 1.1 and carries |z| + 16 steps of its terms' magnitude 1 + |z|
        if gate_first:
            m = ref["mag"] * yv * (1.1 + np.abs(glue._f64(g["z"])))
        else:
            m = np.abs(glue._f64(do)) * ((np.abs(f["n"]) + np.abs(f["mean"]) * f["rstd"] + 1) *
                                         np.abs(g["w"]) +
                                         np.abs(0 if g["b"] is None else g["b"])) \
                * (1.1 + np.abs(glue._f64(g["z"])))
        bz = steps * U * m
        assert excess(down(got["z"]), ref["z"], bz + BF16[z_io] * (np.abs(ref["z"]) + bz)) <= 0
    else:
        assert got["z"] is None
    assert excess(down(got["weight"]), ref["weight"],
                  (steps + rows) * U * ref["weight_scale"]) <= 0
    if bias:
        assert excess(down(got["bias"]), ref["bias"], (steps + rows) * U * ref["bias_scale"]) <= 0
    else:
        assert got["bias"] is None
    assert ssd.device_status() == 0


@pytest.mark.parametrize("C,groups", [(64, 2), (5120, 1), (1000, 1)])
def test_norm_gradients_of_many_rows(C, groups):
    """More rows than CTAs, so that CTAs sum rows of their own; the sums repeat bit for bit."""
    g = inputs(3001, C, "f32", "bf16", seed=3)
    do = store(np.random.default_rng(4).standard_normal((3001, C)), "bf16")
    call = lambda: ssd.group_norm_gate_bwd(  # noqa: E731
        up(do, "bf16"), up(g["y"]), up(g["w"]), up(g["b"]), up(g["z"], "bf16"), groups)
    a, b = call(), call()
    ref = served.group_norm_backward(do, g["y"], g["w"], g["b"], g["z"], groups)
    for k in ("weight", "bias"):
        assert torch.equal(a[k], b[k])
        assert excess(down(a[k]), ref[k], (200 + 3001) * U * ref[k + "_scale"]) <= 0
    assert torch.equal(a["y"], b["y"]) and torch.equal(a["z"], b["z"])


def test_norm_gradients_against_differences():
    g = inputs(6, 48, "f32", "f32", seed=5)
    do = np.random.default_rng(6).standard_normal((6, 48))
    for center in (False, True):
        for first in (False, True):
            got = ssd.group_norm_gate_bwd(up(do.astype(np.float32)), up(g["y"]), up(g["w"]),
                                          up(g["b"]), up(g["z"]), 3, 1e-5, center, first)
            names = dict(y="y", z="z", weight="w", bias="b")
            for k, n in names.items():
                way = np.random.default_rng(7).standard_normal(g[n].shape)
                e = 1e-5
                at = lambda s: np.sum(do.astype(np.float32).astype(np.float64) * served.group_norm(  # noqa
                    **{m: (glue._f64(g[m]) + (s * e * way if m == n else 0)) for m in g},
                    ngroups=3, eps=1e-5, center=center, gate_first=first)["out"])
                diff = (at(1) - at(-1)) / (2 * e)
                mine = float(np.sum(down(got[k]) * way))
                # float32 gradients of unit scale, 288 terms: 200 u each
                assert abs(mine - diff) <= 300 * 200 * U * 4 + 1e-6 * abs(diff)


def test_norm_in_place_and_empty():
    g = inputs(20, 640, "f32", "bf16")
    y, w, z = up(g["y"]), up(g["w"]), up(g["z"], "bf16")
    ref = ssd.group_norm_gate(y, w, None, z, 2)
    assert ssd.group_norm_gate(y, w, None, z, 2, out=y) is y
    assert torch.equal(y, ref)
    e = torch.zeros(0, 640, device="cuda")
    assert ssd.group_norm_gate(e, w).shape == (0, 640)
    got = ssd.group_norm_gate_bwd(e, e, w, up(g["b"]), e)
    assert torch.all(got["weight"] == 0) and torch.all(got["bias"] == 0)


def test_norm_zero_rows_and_huge_values():
    """A row of zeros stays zero (eps); values whose squares overflow are not asked for, values
    whose squares underflow are."""
    y = torch.zeros(3, 64, device="cuda")
    y[1] = 1e18
    y[2] = 1e-22
    out = ssd.group_norm_gate(y, torch.ones(64, device="cuda"))
    assert torch.all(out[0] == 0)
    assert torch.allclose(out[1], torch.ones(64, device="cuda"), atol=1e-6)
    assert torch.allclose(out[2], y[2] / 1e-5 ** 0.5, rtol=1e-5, atol=0)


def test_norm_refuses():
    w = torch.ones(16392, device="cuda")
    y = torch.zeros(2, 16392, device="cuda")
    with pytest.raises(ssd.SSDError):  # one group of 16392 channels
        ssd.group_norm_gate(y, w)
    with pytest.raises(ssd.SSDError):
        ssd.group_norm_gate_bwd(y, y, w)
    y = torch.zeros(2, 8201, device="cuda")
    with pytest.raises(ssd.SSDError):  # odd and past 8192
        ssd.group_norm_gate(y, torch.ones(8201, device="cuda"))
    y = torch.zeros(4, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    with pytest.raises(ssd.SSDError):  # a narrower out in place of y
        ssd.group_norm_gate(y, w, out=y.view(torch.bfloat16)[:, :64])
    with pytest.raises(ssd.SSDError):  # groups that do not divide the channels
        ssd.group_norm_gate(y, w, ngroups=3)
    with pytest.raises(ssd.SSDError):
        ssd.group_norm_gate(y, w, eps=-1.0)
    with pytest.raises(ssd.SSDError):
        ssd.group_norm_gate(y, w, eps=float("nan"))
    with pytest.raises(ValueError):
        ssd.group_norm_gate(y, w[:63])
    with pytest.raises(ValueError):
        ssd.group_norm_gate(y.t(), torch.ones(4, device="cuda"))
    with pytest.raises(TypeError):
        ssd.group_norm_gate(y.half(), w)


@pytest.mark.parametrize("rows,C", [(700, 16384), (700, 8192), (1300, 4096), (2500, 640)])
def test_norm_rows_in_many_rounds(rows, C):
    """Rows that take the CTAs several rounds, through rings of one, two and three rows: the same
    values, bit for bit, as in calls of few rows, which need no ring."""
    g = inputs(rows, C, "f32", "f32", seed=8)
    do = torch.from_numpy(np.random.default_rng(9).standard_normal((rows, C)).astype(np.float32))
    y, z, w, b, do = up(g["y"]), up(g["z"]), up(g["w"]), up(g["b"]), do.cuda()
    out = ssd.group_norm_gate(y, w, b, z, 1)
    grads = ssd.group_norm_gate_bwd(do, y, w, b, z, 1)
    for lo in range(0, rows, 100):
        s = slice(lo, min(lo + 100, rows))
        assert torch.equal(out[s], ssd.group_norm_gate(y[s], w, b, z[s], 1))
        part = ssd.group_norm_gate_bwd(do[s], y[s], w, b, z[s], 1)
        assert torch.equal(grads["y"][s], part["y"]) and torch.equal(grads["z"][s], part["z"])
    assert ssd.device_status() == 0
