"""Packed prompts whose bounds fall or leave the rows: such sequences are left out and reported, the
rows and slots of all others are as in calls of their own (rows that two sequences name may hold
either's)."""
import numpy as np
import pytest
import torch

import mamba_ssd_scan_03_b200 as ssd
from oracle import served
from served_util import conv_bound, down, excess, scan_bound, up
from test_gpu_served import conv_inputs, flags, i32, scan_inputs

pytestmark = pytest.mark.gpu

INDEX = 6


def whole_sequences(cu, ntok):
    """The sequences to scan, and how many of them name each row."""
    ok = [i for i in range(len(cu) - 1) if 0 <= cu[i] <= cu[i + 1] <= ntok]
    named = np.zeros(ntok, int)
    for i in ok:
        named[cu[i]:cu[i + 1]] += 1
    return ok, named


def check_conv(cu, T, C, K, io="f32", seed=0):
    n = len(cu) - 1
    r = np.random.default_rng(seed)
    g = conv_inputs(T, C, K, n + 2, io, seed)
    slots = [int(s) for s in r.permutation(n + 2)[:n]]
    resume = [bool(v) for v in r.integers(0, 2, n)]
    st = up(g["state"], io)
    out = torch.full((T, C), 5.0, device="cuda", dtype=st.dtype)
    ssd.conv_silu_varlen(up(g["u"], io), up(g["w"]), i32(cu), up(g["bias"]), st, i32(slots),
                         flags(resume), out=out)
    status = ssd.device_status()
    ok, named = whole_sequences(cu, T)
    got, rst = down(out), down(up(g["state"], io))
    assert np.all(got[named == 0] == 5.0)
    for i in ok:
        one = ([cu[i], cu[i + 1]], g["state"], [slots[i]], [resume[i]])
        ref, state = served.conv_silu(g["u"], g["w"], g["bias"], *one)
        bound = conv_bound(g["u"], g["w"], g["bias"], *one, io)
        rows = [t for t in range(cu[i], cu[i + 1]) if named[t] == 1]
        worst = excess(got[rows], ref[rows], bound[rows])
        assert worst <= 0, (cu, i)
        rst[slots[i]] = state[slots[i]]
    assert [s for s in range(n + 2) if not np.array_equal(down(st)[s], rst[s])] == []
    assert status == (0 if len(ok) == n else INDEX)


def check_scan(cu, T, dim, N, hint=0, seed=0):
    n = len(cu) - 1
    r = np.random.default_rng(seed)
    g = scan_inputs(T, dim, N, 1, n + 2, "f32", seed=seed)
    slots = [int(s) for s in r.permutation(n + 2)[:n]]
    resume = [bool(v) for v in r.integers(0, 2, n)]
    t = {k: up(g[k]) for k in ("x", "dt", "A", "B", "C", "D", "z", "dt_bias", "state")}
    out = torch.full((T, dim), 5.0, device="cuda")
    ssd.selective_scan_varlen(t["x"], t["dt"], t["A"], t["B"], t["C"], i32(cu), t["D"], t["z"],
                              t["dt_bias"], True, t["state"], i32(slots), flags(resume), out=out,
                              max_seqlen=hint)
    status = ssd.device_status()
    ok, named = whole_sequences(cu, T)
    got, gst = down(out), down(t["state"])
    assert np.all(got[named == 0] == 5.0)
    for i in ok:
        one = dict(g, cu=[cu[i], cu[i + 1]], slots=[slots[i]], resume=[resume[i]])
        ref = served.selective_scan(**one)
        by, bh = scan_bound(one, ref, "f32")
        rows = [k for k in range(cu[i], cu[i + 1]) if named[k] == 1]
        worst = (excess(got[rows], ref[0][rows], by[rows]),
                 excess(gst[slots[i]], ref[1][slots[i]], bh[slots[i]]))
        assert max(worst) <= 0, (cu, i)
    left = [s for s in range(n + 2) if s not in [slots[i] for i in ok]]
    assert [s for s in left if not np.array_equal(gst[s], g["state"][s].astype(np.float64))] == []
    assert status == (0 if len(ok) == n else INDEX)


BIG = 2 ** 31 - 1
BOUNDS = [
    (100, [0, 200, 20, 30, 100]),             # past the rows, then back
    (300, [0, 100, 400, 200, 300]),
    (300, [0, 100, -5, 200, 300]),            # before the rows
    (300, [0, 250, 40, 290]),                 # rows named twice
    (300, [0, 120, 120, 300, 0, 0, 10]),      # and a start over
    (300, [0, BIG, -BIG - 1, 10, 300]),
    (300, [300, 0, 300]),
    (64, [70, 60, 50, 40, 30, 20, 10, 0]),    # nothing but falls
]


@pytest.mark.parametrize("T,cu", BOUNDS)
@pytest.mark.parametrize("C,K", [(40, 4), (33, 2), (8, 8)])
def test_conv_leaves_out_only_bad_sequences(T, cu, C, K):
    check_conv(cu, T, C, K, seed=len(cu))
    check_conv(cu, T, C, K, "bf16", seed=len(cu) + 1)


@pytest.mark.parametrize("T,cu", [(12, [0, 9, 13, 13]), (12, [-3, -3, 0, 12]), (12, [5, 5, 12, 12]),
                                  (12, [0, 12, 12, 13, 13, 12, 12])])
@pytest.mark.parametrize("C,K", [(40, 4), (33, 2)])
def test_conv_of_empty_sequences_off_the_rows(T, cu, C, K):
    """An empty fresh sequence clears its slot; not so where its bounds lie off the rows."""
    for seed in range(4):
        check_conv(cu, T, C, K, seed=seed)


@pytest.mark.parametrize("T,cu", BOUNDS)
def test_scan_leaves_out_only_bad_sequences(T, cu):
    check_scan(cu, T, 24, 16, seed=len(cu))


@pytest.mark.parametrize("T,cu", [
    (1000, [0, 5000, 3000, 300, 400, 1000]),  # bad sequences are not chunks
    (1000, [0, 1000, 0, 1000]),               # whole sequences twice
    (1000, [0, 900, 50, 950, 100, 1000]),
    (1000, [0, BIG, -BIG - 1, 10, 990]),
    (1000, [-1, 0, 995, 1001, 1001]),
    (1000, [0, 300, 300, 999])])              # in order
def test_scan_in_chunks_leaves_out_only_bad_sequences(T, cu):
    assert ssd.selective_varlen_workspace_size(T, len(cu) - 1, 24, 16, 1, 1000) > 0
    check_scan(cu, T, 24, 16, hint=1000, seed=len(cu))


def test_random_bounds():
    """Bounds in no order, on and around the rows; more of them than a warp has lanes."""
    r = np.random.default_rng(5)
    for k in range(24):
        n = int(r.integers(1, 12)) if k % 4 else int(r.integers(33, 70))
        T = int(r.integers(1, 260))
        cu = r.integers(-3, T + 4, n + 1)
        if k % 2:  # in order but for a few
            cu = np.sort(cu)
            at = r.integers(0, n + 1, 2)
            cu[at] = r.integers(-3, T + 4, 2)
        cu = [int(v) for v in cu]
        check_conv(cu, T, 12, 4, seed=k)
        check_scan(cu, T, 10, 8, seed=k)
    assert ssd.device_status() == 0
