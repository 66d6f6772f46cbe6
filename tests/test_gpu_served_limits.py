"""The served forms and the norm where callers reach their limits: offsets past 32 bits, refusals
that need device memory, calls captured, replayed, on two streams at once, and in place of their
workspace."""
import numpy as np
import pytest
import torch

import mamba_ssd_scan_03_b200 as ssd
from oracle import served
from served_util import conv_bound, down, excess, scan_bound, up
from test_gpu_served import conv_inputs, flags, i32, scan_inputs

pytestmark = pytest.mark.gpu

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3


def refused(code, call):
    with pytest.raises(ssd.SSDError) as e:
        call()
    assert e.value.code == code


def test_conv_rows_past_32_bits():
    """Rows whose element offsets pass 2^31, in u, out and the history."""
    T, C, K = 400_003, 5376, 4
    assert (T - 200) * C > 2 ** 31
    g = conv_inputs(150, C, K, 1, "bf16")
    lo = T - 150
    u = torch.zeros(T, C, device="cuda", dtype=torch.bfloat16)
    u[lo:] = up(g["u"], "bf16")
    nslots = 2 ** 31 // (C * (K - 1)) + 2
    hist = torch.empty(nslots, K - 1, C, device="cuda", dtype=torch.bfloat16)
    hist[nslots - 1] = up(g["state"], "bf16")[0]
    hist[3] = 0
    cu = [0, lo, T]
    out = ssd.conv_silu_varlen(u, up(g["w"]), i32(cu), up(g["bias"]), hist,
                               i32([3, nslots - 1]), flags([0, 1]))
    ref, rst = served.conv_silu(g["u"], g["w"], g["bias"], [0, 150], g["state"], None, [1])
    bound = conv_bound(g["u"], g["w"], g["bias"], [0, 150], g["state"], None, [1], "bf16")
    assert excess(down(out[lo:]), ref, bound) <= 0
    assert np.array_equal(down(hist[nslots - 1]), rst[0])
    one = ssd.conv_silu_step(hist, up(g["u"], "bf16")[:1].contiguous(), up(g["w"]),
                             up(g["bias"]), i32([nslots - 1]))
    ref, rst = served.conv_silu(g["u"][:1], g["w"], g["bias"], [0, 1], rst, None, [1])
    assert np.max(np.abs(down(one) - ref)) <= 2.0 ** -7 * (1 + np.max(np.abs(ref)))
    assert np.array_equal(down(hist[nslots - 1]), rst[0])
    assert ssd.device_status() == 0


def test_scan_state_past_32_bits():
    """A slot whose offset in the cache passes 2^31 floats, for prompts and tokens."""
    dim, N = 4096, 16
    nslots = 2 ** 31 // (dim * N) + 3
    state = torch.empty(nslots, dim, N, device="cuda")
    g = scan_inputs(6, dim, N, 1, 1)
    state[nslots - 1] = up(g["state"])[0]
    t = {k: up(g[k], "bf16") for k in ("x", "B", "C", "z")} | \
        {k: up(g[k]) for k in ("dt", "A", "D", "dt_bias")}
    y = ssd.selective_scan_varlen(t["x"], t["dt"], t["A"], t["B"], t["C"], i32([0, 6]), t["D"],
                                  t["z"], t["dt_bias"], True, state, i32([nslots - 1]),
                                  flags([1]))
    g.update(cu=[0, 6], slots=None, resume=[1])
    ref = served.selective_scan(**g)
    by, bh = scan_bound(g, ref, "f32")
    assert excess(down(y), ref[0], by) <= 0
    assert excess(down(state[nslots - 1:]), ref[1], bh) <= 0
    state[nslots - 1] = up(g["state"])[0]
    for i in range(6):
        row = {k: t[k][i:i + 1] for k in ("x", "dt", "B", "C", "z")}
        yi = ssd.selective_step(state, row["x"], row["dt"], t["A"], row["B"], row["C"], t["D"],
                                row["z"], t["dt_bias"], True, i32([nslots - 1]))
        assert excess(down(yi), ref[0][i:i + 1], by[i:i + 1]) <= 0
    assert excess(down(state[nslots - 1:]), ref[1], bh) <= 0
    assert ssd.device_status() == 0


def test_scan_rows_past_32_bits():
    """Rows of x, dt and y past 2^31 elements, in a strided view."""
    dim, N, T = 64, 16, 40
    stride = 2 ** 31 // (T - 8)
    g = scan_inputs(T, dim, N, 1, 1, gate=False)
    wide = torch.empty(T * stride, device="cuda", dtype=torch.bfloat16)
    x = wide.as_strided((T, dim), (stride, 1))
    x.copy_(up(g["x"], "bf16"))
    out = torch.empty(T * stride, device="cuda", dtype=torch.bfloat16).as_strided((T, dim),
                                                                                 (stride, 1))
    ssd.selective_scan_varlen(x, up(g["dt"]), up(g["A"]), up(g["B"], "bf16"), up(g["C"], "bf16"),
                              i32([0, T]), up(g["D"]), None, up(g["dt_bias"]), True, out=out)
    g.update(cu=[0, T], state=None)
    ref = served.selective_scan(**g)
    assert excess(down(out), ref[0], scan_bound(g, ref, "bf16")[0]) <= 0


def test_refusals_with_device_memory():
    u = torch.zeros(8, 16, device="cuda", dtype=torch.bfloat16)
    w = torch.zeros(16, 4, device="cuda")
    cu = i32([0, 8])
    cs = torch.zeros(2, 3, 16, device="cuda", dtype=torch.bfloat16)
    refused(INVALID, lambda: ssd.conv_silu_varlen(u, w, cu, out=u))           # in place
    refused(INVALID, lambda: ssd.conv_silu_varlen(u, w, cu, slots=i32([0])))  # slots, no cache
    refused(INVALID, lambda: ssd.conv_silu_varlen(u, w, cu, resume=flags([1])))
    refused(INVALID, lambda: ssd.conv_silu_varlen(u, w, i32([0, 1, 2, 8]), conv_state=cs))
    refused(INVALID, lambda: ssd.conv_silu_varlen(u, torch.zeros(16, 9, device="cuda"), cu))
    refused(INVALID, lambda: ssd.conv_silu_step(cs, u, w))                    # 8 rows, 2 slots
    refused(INVALID, lambda: ssd.conv_silu_step(None, u, w))
    refused(INVALID, lambda: ssd.conv_silu_step(cs[:0], u, w))                # a cache of no slots
    refused(INVALID, lambda: ssd.conv_silu_varlen(u, w, cu, conv_state=cs[:0]))
    refused(INVALID, lambda: ssd.conv_silu_step(torch.zeros(8, 0, 16, device="cuda",
                                                            dtype=torch.bfloat16), u, w[:, :1]
                                                .contiguous()))
    x = torch.zeros(8, 16, device="cuda")
    A, B = -torch.ones(16, 16, device="cuda"), torch.zeros(8, 1, 16, device="cuda")
    st = torch.zeros(2, 16, 16, device="cuda")
    refused(INVALID, lambda: ssd.selective_scan_varlen(x, x, A, B, B, cu, out=x))
    refused(INVALID, lambda: ssd.selective_scan_varlen(x, x, A, B, B, cu, resume=flags([1])))
    refused(INVALID, lambda: ssd.selective_scan_varlen(x, x, A, B, B, cu, max_seqlen=-1))
    refused(INVALID, lambda: ssd.selective_scan_varlen(x, x, A, B, B, cu, state=st[:0]))
    refused(INVALID, lambda: ssd.selective_step(st, x, x, A, B, B))           # 8 rows, 2 slots
    refused(INVALID, lambda: ssd.selective_step(None, x, x, A, B, B))
    refused(INVALID, lambda: ssd.selective_step(st[:0], x, x, A, B, B))
    wide = torch.zeros(16, 129, device="cuda")
    B129 = torch.zeros(8, 1, 129, device="cuda")
    refused(UNSUPPORTED, lambda: ssd.selective_scan_varlen(x, x, wide, B129, B129, cu))
    refused(UNSUPPORTED, lambda: ssd.selective_step(torch.zeros(8, 16, 129, device="cuda"), x, x,
                                                    wide, B129, B129))
    long = torch.zeros(2048, 16, device="cuda")
    BL = torch.zeros(2048, 1, 16, device="cuda")
    small = torch.zeros(16, device="cuda", dtype=torch.uint8)
    refused(WORKSPACE, lambda: ssd.selective_scan_varlen(long, long, A, BL, BL, i32([0, 2048]),
                                                         workspace=small))
    with pytest.raises(TypeError):
        ssd.selective_scan_varlen(x, x.bfloat16(), A, B, B, cu)   # dt neither f32 nor x's type
    with pytest.raises(TypeError):
        ssd.selective_scan_varlen(x, x, A, B, B, cu.long())
    with pytest.raises(TypeError):
        ssd.selective_scan_varlen(x, x, None, B, B, cu)
    with pytest.raises(TypeError):
        ssd.conv_silu_varlen(u.half(), w, cu)
    with pytest.raises(ValueError):
        ssd.selective_scan_varlen(x, x, A, B.cpu(), B, cu)
    with pytest.raises(ValueError):
        ssd.conv_silu_varlen(u[:1].expand(8, 16), w, cu)          # rows that overlap
    with pytest.raises(ValueError):
        ssd.conv_silu_varlen(u.t().contiguous().t(), w, cu)       # values that are not neighbours
    refused(INVALID, lambda: ssd.selective_scan_varlen(x, x, A, B, B, cu,
                                                       y_dtype=torch.bfloat16))  # f32 x, bf16 y
    assert ssd.device_status() == 0


def test_two_streams_at_once():
    """The chunked plan on two streams at the same time, each call with a workspace of its own."""
    g = scan_inputs(3000, 48, 16, 1, 1)
    t = {k: up(g[k], "bf16") for k in ("x", "B", "C", "z")} | \
        {k: up(g[k]) for k in ("dt", "A", "D", "dt_bias", "state")}
    assert ssd.selective_varlen_workspace_size(3000, 1, 48, 16, 1) > 0

    def call(st):
        return ssd.selective_scan_varlen(t["x"], t["dt"], t["A"], t["B"], t["C"], i32([0, 3000]),
                                         t["D"], t["z"], t["dt_bias"], True, st,
                                         resume=flags([1]))

    st0 = t["state"].clone()
    y0 = call(st0)
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    for k in range(6):
        s = streams[k % 2]
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            st = t["state"].clone()
            got.append((call(st), st))
    torch.cuda.synchronize()
    for y, st in got:
        assert torch.equal(y, y0) and torch.equal(st, st0)


def test_norm_and_chunks_captured():
    """The norm, its gradients and the chunked scan, captured, and replayed on new values; the norm
    with a ring past the default shared memory, where its first call may be the captured one."""
    g = scan_inputs(2000, 40, 16, 1, 1)
    t = {k: up(g[k], "bf16") for k in ("x", "B", "C")} | {k: up(g[k]) for k in ("dt", "A", "state")}
    y, z = torch.randn(2000, 2048, device="cuda"), torch.randn(2000, 2048, device="cuda")
    w, b = torch.randn(2048, device="cuda"), torch.randn(2048, device="cuda")
    cu = i32([0, 900, 2000])
    st = t["state"].repeat(2, 1, 1)

    def all_of(st):
        o = ssd.group_norm_gate(y, w, b, z, 2, center=True)
        d = ssd.group_norm_gate_bwd(o, y, w, b, z, 2, center=True)
        s = ssd.selective_scan_varlen(t["x"], t["dt"], t["A"], t["B"], t["C"], cu, softplus=True,
                                      state=st, resume=flags_)
        return [o, d["y"], d["z"], d["weight"], d["bias"], s]

    flags_ = flags([1, 0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = all_of(st)
    for seed in (1, 2):
        torch.manual_seed(seed)
        y.normal_(), z.normal_()
        cu.copy_(i32([[0, 900, 2000], [0, 1990, 1999]][seed - 1]))
        st0 = st.clone()
        got[-1].fill_(5.0)
        graph.replay()
        want = all_of(st0)
        n = int(cu[-1])
        for a, e in zip(got[:-1], want[:-1]):
            assert torch.equal(a, e)
        assert torch.equal(got[-1][:n], want[-1][:n]) and torch.all(got[-1][n:] == 5.0)
        assert torch.equal(st, st0)
    assert ssd.device_status() == 0


def test_infinities_outside_the_sequences():
    """NaN and infinities in rows that no sequence covers, and in slots that no sequence names, stay
    where they are."""
    g = scan_inputs(40, 24, 16, 1, 4, "f32", "f32")
    c = conv_inputs(40, 24, 4, 4, "f32")
    bad = [0, 1, 12, 13, 14, 38, 39]
    cu, slots = [2, 12, 12, 15, 38], [1, 0, -1, 3]
    dirty = {}
    for k, v in (("x", g["x"]), ("dt", g["dt"]), ("B", g["B"]), ("C", g["C"]), ("z", g["z"]),
                 ("u", c["u"])):
        v = v.copy()
        v[bad] = np.nan
        v[bad[::2]] = np.inf
        dirty[k] = up(v)
    st, cs = g["state"].copy(), c["state"].copy()
    st[2], cs[2] = np.nan, np.inf
    ts, tc = up(st), up(cs)
    y = ssd.selective_scan_varlen(dirty["x"], dirty["dt"], up(g["A"]), dirty["B"], dirty["C"],
                                  i32(cu), up(g["D"]), dirty["z"], up(g["dt_bias"]), True, ts,
                                  i32(slots), flags([1, 0, 1, 0]))
    o = ssd.conv_silu_varlen(dirty["u"], up(c["w"]), i32(cu), up(c["bias"]), tc, i32(slots),
                             flags([1, 0, 1, 0]))
    rows = list(range(2, 12)) + list(range(15, 38))
    assert torch.all(torch.isfinite(y[rows])) and torch.all(torch.isfinite(o[rows]))
    assert torch.all(torch.isfinite(ts[[0, 1, 3]])) and torch.all(torch.isfinite(tc[[0, 1, 3]]))
    assert torch.all(torch.isnan(ts[2])) and torch.all(torch.isinf(tc[2]))
    assert ssd.device_status() == 0


def test_bounds_past_the_rows_leave_their_sequence_out():
    """A last sequence that ends past the rows: none of its rows and not its slot; the others as
    usual."""
    g, c = scan_inputs(12, 16, 16, 1, 2), conv_inputs(12, 16, 4, 2, "bf16")
    st, cs = up(g["state"]), up(c["state"], "bf16")
    y = torch.full((12, 16), 5.0, device="cuda")
    ssd.selective_scan_varlen(up(g["x"], "bf16"), up(g["dt"]), up(g["A"]), up(g["B"], "bf16"),
                              up(g["C"], "bf16"), i32([0, 9, 13]), softplus=True, state=st, out=y)
    assert ssd.device_status() == 6
    assert torch.all(y[9:] == 5.0) and not torch.any(y[:9] == 5.0)
    assert np.array_equal(down(st)[1], g["state"][1].astype(np.float64))
    o = torch.full((12, 16), 5.0, device="cuda", dtype=torch.bfloat16)
    ssd.conv_silu_varlen(up(c["u"], "bf16"), up(c["w"]), i32([0, 9, 13]), conv_state=cs, out=o)
    assert ssd.device_status() == 6
    assert torch.all(o[9:] == 5.0) and not torch.any(o[:9] == 5.0)
    assert np.array_equal(down(cs)[1], down(up(c["state"], "bf16"))[1])


def test_many_sequences_longest_first():
    """More CTAs than the GPU holds at a time: sequences are taken by length, whatever their order
    and ties; more than 128 of them in their own order."""
    r = np.random.default_rng(11)
    for n, dim in ((100, 512), (128, 400), (140, 300)):
        lens = r.integers(0, 9, n)
        cu = [0] + [int(v) for v in np.cumsum(lens)]
        g = scan_inputs(cu[-1], dim, 16, 1, n, "bf16")
        resume = [bool(v) for v in r.integers(0, 2, n)]
        t = {k: up(g[k], "bf16") for k in ("x", "B", "C", "z")} | \
            {k: up(g[k]) for k in ("dt", "A", "D", "dt_bias", "state")}
        y = ssd.selective_scan_varlen(t["x"], t["dt"], t["A"], t["B"], t["C"], i32(cu), t["D"],
                                      t["z"], t["dt_bias"], True, t["state"], None, flags(resume))
        g.update(cu=cu, slots=None, resume=resume)
        ref = served.selective_scan(**g)
        by, bh = scan_bound(g, ref, "f32")
        assert excess(down(y), ref[0], by) <= 0
        assert excess(down(t["state"]), ref[1], bh) <= 0
    assert ssd.device_status() == 0
